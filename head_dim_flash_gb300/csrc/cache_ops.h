// Internal interface of the operators around a 16-bit K/V cache (rotary
// positions, decode over a shared prefix, decode that scores its cache,
// eviction) between the C-ABI host layer (api.cu) and the kernels.
#pragma once

#include "kernels.h"

namespace ffpa {

// Sites of a sequence whose length lies outside its cache, in the device status word.
enum : uint32_t { VS_LINE = 0x7b, VS_EVICT = 0x7c };

// Tokens that a cache and its prefix may hold, or an eviction keep: the kernels'
// indexes, up to a block of 4096 past the last token, stay within 31 bits.
constexpr int kMaxTokens = 0x7fffffff - 4096;

// Rotary positions of q and k (k absent: Hk = 0), or their inverse.
struct RopeArgs {
    int bf16;
    const void *q, *k;
    void *oq, *ok;
    View vq, vk, voq, vok;        // packed: one batch entry
    const unsigned long long* turns;  // device [rot / 2]: turns per position, in units of 2^-64
    int rot, interleaved;
    float mscale, sign;           // sign: -1 turns back (the gradient)
    int zero_rest;                // packed: rows of no sequence become zero, instead of staying as they are
    const int* start;             // device [B]: position of each sequence's first token (null: 0)
    const int* pos;               // device [B, N] / [total]: every position, or null
    const int* cu;                // device [B + 1]: packed token offsets, or null
    int B, Hq, Hk, N, total, D;
    // set by the launch
    int per_cta;                  // tokens per CTA
    int heads_per;                // heads per CTA
    int copy_q, copy_k;           // head dims past `rot` are copied (not in place)
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s);

// Cutting a cache to `keep` tokens per kv head.
struct EvictArgs {
    const void *k, *v;
    void *ok, *ov;
    View vk, vv, vok, vov;
    const float* weights;         // [B, Hkv, N]
    float* oweights;              // [B, Hkv, Nout]
    const int* lens;              // device [B]
    int* olens;
    int* kept;                    // [B, Hkv, keep]: where each kept token was, -1 behind the last
    int B, Hkv, N, Nout, D, keep, recent;
    int in_place;
    uint32_t* status;
};
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s);

// Decode forward over caches of different lengths; in the shared form also
// over a prefix of Np keys common to the batch, in the scoring form with the
// attention weights added to a score per token.
struct LineArgs {
    FwdArgs f;                    // pb.Nkv: tokens a sequence's cache can hold
    const int* lens;              // device [B] (null: all of pb.Nkv)
    // the shared prefix
    int shared, Np;
    const void *kp, *vp;          // [1, Hkv, Np, D]
    View vkp, vvp;
    // scoring
    const float* weights;         // [B, Hkv, N]
    float* oweights;
};
size_t line_workspace_bytes(const Problem& pb, bool shared, int Np);
bool line_fits(const Problem& pb, bool shared, int Np);  // its tiles can be numbered
// Launches nothing where the workspace is smaller than `need`, which it tells.
cudaError_t launch_line(const LineArgs& a, void* workspace, size_t workspace_bytes, size_t* need, cudaStream_t s);

}  // namespace ffpa
