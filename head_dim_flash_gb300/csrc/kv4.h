// The 4-bit K/V cache's part of the internal interface between the C-ABI host
// layer (api.cu) and the kernels.
#pragma once

#include "kernels.h"

namespace ffpa {

// Sites of a sequence that breaks the contract of a 4-bit cache, in the device status word.
enum : uint32_t { VS_KV4_WRITE = 0x78, VS_KV4_READ = 0x79, VS_KV4_DECODE = 0x7a };

// The paged 4-bit K/V cache (format in kv4.cuh) and its block table.
constexpr int kKv4Tile = 576;  // bytes of a tile of 16 tokens x 64 head dims
struct Kv4Cache {
    uint8_t* data;            // [num_pages][2][Hkv][page_size / 16][D / 64][kKv4Tile]
    int num_pages, page_size;
    const int* table;         // device [B rows, table_stride apart]: page of each block
    int max_blocks;
    long long table_stride;
};

// Writing the cache from, and reading it back to, a 16-bit tensor.
struct Kv4Io {
    Kv4Cache cache;
    int bf16;
    int B, Hkv, N, D;         // N: most tokens of one sequence
    void *k, *v;              // [B, Hkv, N, D] views, or packed [total, Hkv, D]
    View vk, vv;
    const int* start;         // device [B]: cache position of each sequence's first token (null: 0)
    const int* count;         // device [B]: tokens of each sequence (null: N); unused when packed
    const int* cu;            // device [B + 1]: packed token offsets, or null
    int total;
    int strips_per_cta;       // set by the launch
    int wide;                 // the same: every row of k begins on 32 bytes
    uint32_t* status;
};
cudaError_t launch_kv4_write(const Kv4Io& a, cudaStream_t s);
cudaError_t launch_kv4_read(const Kv4Io& a, cudaStream_t s);

// Decode / short-query forward over the cache.
struct Kv4Decode {
    Kv4Cache cache;
    const int* seq_lens;      // device [B]: cached tokens of each sequence
    FwdArgs f;                // k, v unused; pb.Nkv unused
};
size_t kv4_decode_workspace_bytes(const Problem& pb);
cudaError_t launch_decode_kv4(const Kv4Decode& a, void* workspace, cudaStream_t s);

}  // namespace ffpa
