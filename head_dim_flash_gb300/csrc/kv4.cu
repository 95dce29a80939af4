// Writing new tokens into the paged 4-bit K/V cache, and reading cached
// tokens back to 16 bits. The format is in kv4.cuh.
//
// Both are one pass over the data and bound by memory: a write reads 2 bytes
// and stores 9/16 of a byte per value, a read the reverse. A warp owns one
// tile of 16 tokens x 64 head dims, whose lanes hold it in the order in which
// the cache stores it: a whole tile is one 16-byte store per lane plus the
// scales, and the 16-bit side moves 128 contiguous bytes per token. A strip
// that a sequence covers in part (its first and last) is stored token by
// token, and the cells of other tokens are left as they were.
#include "kv4.cuh"

namespace ffpa {
namespace {

constexpr int kIoWarps = 8;  // at most; one CTA per (sequence, kv head, strip of 16 tokens)

template <bool BF16>
__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<BF16>(u[i]);
        x[2 * i] = f.x == f.x ? f.x : 0.f;  // the cache has no NaN: one is stored as zero
        x[2 * i + 1] = f.y == f.y ? f.y : 0.f;
    }
}

__device__ __forceinline__ float amax8(const float (&x)[8])
{
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    return m;
}

// Four fp16 pairs (exact cache values) in the element type.
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const uint32_t (&h)[4])
{
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u[i] = h[i];
        if constexpr (BF16) {
            const float2 f = unpack2<false>(h[i]);
            u[i] = pack2<true>(f.x, f.y);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// The strip of this CTA: false when the sequence does not reach it.
struct Strip {
    int b, h;
    int t0;          // its first cache position
    int p0, p1;      // the sequence's range of positions
    long long row0;  // row of position p0 in the 16-bit tensor
    uint8_t* base;   // first K tile
    size_t v_off;    // from a K tile to the V tile
};

__device__ __forceinline__ bool find_strip(const Kv4Io& a, uint32_t site, Strip& s)
{
    const long long u = unit_id();
    if (u >= static_cast<long long>(a.B) * a.Hkv) return false;
    s.b = static_cast<int>(u / a.Hkv);
    s.h = static_cast<int>(u % a.Hkv);
    int cnt;
    if (!kv4_range(a, s.b, site, s.p0, cnt, s.row0)) return false;
    s.p1 = s.p0 + cnt;
    const long long t0 = (static_cast<long long>(s.p0 >> 4) + blockIdx.x) << 4;
    if (t0 >= s.p1) return false;
    s.t0 = static_cast<int>(t0);
    const int block = s.t0 / a.cache.page_size;
    const int page = a.cache.table[s.b * a.cache.table_stride + block];
    if (page < 0 || page >= a.cache.num_pages) {
        if (threadIdx.x == 0) kv4_invalid(a.status, site, s.b);
        return false;
    }
    const int chunks = a.D >> 6;
    s.base = a.cache.data +
             kv4_strip_offset(a.cache, a.Hkv, chunks, page, 0, s.h, (s.t0 - block * a.cache.page_size) >> 4);
    s.v_off = static_cast<size_t>(a.Hkv) * (a.cache.page_size >> 4) * chunks * kKv4Tile;
    return true;
}

// Element offset of position p's row of this (sequence, head).
__device__ __forceinline__ long long row_offset(const Kv4Io& a, const Strip& s, const View& v, int p)
{
    return (a.cu ? 0 : s.b * v.sb) + s.h * v.sh + (s.row0 + (p - s.p0)) * v.sn;
}

template <bool BF16>
__global__ void __launch_bounds__(kIoWarps * 32) kv4_write_kernel(const Kv4Io a)
{
    Strip s;
    if (!find_strip(a, VS_KV4_WRITE, s)) return;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int chunks = a.D >> 6;
    for (int it = threadIdx.x >> 5; it < 2 * chunks; it += blockDim.x >> 5) {
        const int ch = it < chunks ? it : it - chunks;
        uint8_t* tile = s.base + static_cast<size_t>(ch) * kKv4Tile;
        if (it < chunks) {
            uint32_t code[4];
            uint32_t sc[2];
            bool in[2];
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const int p = s.t0 + g + 8 * hi;
                in[hi] = p >= s.p0 && p < s.p1;
                uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
                if (in[hi]) {
                    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.k) +
                                                                      row_offset(a, s, a.vk, p) + ch * 64 + t * 16);
                    w0 = src[0];
                    w1 = src[1];
                }
                float x0[8], x1[8];
                unpack8<BF16>(w0, x0);
                unpack8<BF16>(w1, x1);
                sc[hi] = kv4_scale_code(fmaxf(amax8(x0), amax8(x1)));
                const float f = kv4_scale_value(sc[hi]), rcp = f > 0.f ? 1.f / f : 0.f;
                code[2 * hi] = kv4_code8(x0, rcp);
                code[2 * hi + 1] = kv4_code8(x1, rcp);
            }
            if (in[0] && in[1]) {
                *reinterpret_cast<uint4*>(tile + lane * 16) = make_uint4(code[0], code[1], code[2], code[3]);
                *reinterpret_cast<uint16_t*>(tile + 512 + lane * 2) = static_cast<uint16_t>(sc[0] | (sc[1] << 8));
            } else {
#pragma unroll
                for (int hi = 0; hi < 2; ++hi)
                    if (in[hi]) {
                        *reinterpret_cast<uint2*>(tile + lane * 16 + 8 * hi) = make_uint2(code[2 * hi], code[2 * hi + 1]);
                        tile[512 + lane * 2 + hi] = static_cast<uint8_t>(sc[hi]);
                    }
            }
        } else {
            tile += s.v_off;
            uint32_t code[4], sc = 0;
            bool in[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int p = s.t0 + 2 * t + (j & 1) + 8 * (j >> 1);
                in[j] = p >= s.p0 && p < s.p1;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (in[j])
                    w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.v) + row_offset(a, s, a.vv, p) +
                                                        ch * 64 + g * 8);
                float x[8];
                unpack8<BF16>(w, x);
                float m = amax8(x);
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));  // the group's other half
                const uint32_t c = kv4_scale_code(m);
                const float f = kv4_scale_value(c), rcp = f > 0.f ? 1.f / f : 0.f;
                code[j] = kv4_code8(x, rcp);
                sc |= c << (8 * j);
            }
            uint8_t* scale = tile + 512 + ((g >> 1) * 4 + t) * 4;
            if (in[0] && in[1] && in[2] && in[3]) {
                *reinterpret_cast<uint4*>(tile + lane * 16) = make_uint4(code[0], code[1], code[2], code[3]);
                if (!(g & 1)) *reinterpret_cast<uint32_t*>(scale) = sc;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (in[j]) {
                        *reinterpret_cast<uint32_t*>(tile + lane * 16 + 4 * j) = code[j];
                        if (!(g & 1)) scale[j] = static_cast<uint8_t>(sc >> (8 * j));
                    }
            }
        }
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kIoWarps * 32) kv4_read_kernel(const Kv4Io a)
{
    Strip s;
    if (!find_strip(a, VS_KV4_READ, s)) return;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int chunks = a.D >> 6;
    for (int it = threadIdx.x >> 5; it < 2 * chunks; it += blockDim.x >> 5) {
        const int ch = it < chunks ? it : it - chunks;
        const uint8_t* tile = s.base + static_cast<size_t>(ch) * kKv4Tile + (it < chunks ? 0 : s.v_off);
        const uint4 w = *reinterpret_cast<const uint4*>(tile + lane * 16);
        const uint32_t code[4] = {w.x, w.y, w.z, w.w};
        if (it < chunks) {
            const uint32_t sc = *reinterpret_cast<const uint16_t*>(tile + 512 + lane * 2);
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const int p = s.t0 + g + 8 * hi;
                if (p < s.p0 || p >= s.p1) continue;
                uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k) + row_offset(a, s, a.vk, p) + ch * 64 +
                                                      t * 16);
                const uint32_t s2 = kv4_scale2(sc >> (8 * hi));
                uint32_t h[4];
                kv4_dequant8(code[2 * hi], s2, h);
                dst[0] = pack8<BF16>(h);
                kv4_dequant8(code[2 * hi + 1], s2, h);
                dst[1] = pack8<BF16>(h);
            }
        } else {
            const uint32_t sc = *reinterpret_cast<const uint32_t*>(tile + 512 + ((g >> 1) * 4 + t) * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int p = s.t0 + 2 * t + (j & 1) + 8 * (j >> 1);
                if (p < s.p0 || p >= s.p1) continue;
                uint32_t h[4];
                kv4_dequant8(code[j], kv4_scale2(sc >> (8 * j)), h);
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v) + row_offset(a, s, a.vv, p) + ch * 64 + g * 8) =
                    pack8<BF16>(h);
            }
        }
    }
}

// CTAs along x: the strips that N tokens can touch (one more when a start need not be a multiple of 16).
bool io_grid(const Kv4Io& a, dim3* grid, unsigned* threads)
{
    const long long strips = (static_cast<long long>(a.N) + (a.start ? 30 : 15)) >> 4;
    const int items = 2 * (a.D >> 6);
    *threads = 32u * static_cast<unsigned>(items < kIoWarps ? items : kIoWarps);
    return unit_grid(static_cast<unsigned>(strips), static_cast<long long>(a.B) * a.Hkv, grid);
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4Io& a, cudaStream_t s)
{
    dim3 grid;
    unsigned threads;
    if (!io_grid(a, &grid, &threads)) return cudaErrorInvalidConfiguration;
    if (a.bf16)
        kv4_write_kernel<true><<<grid, threads, 0, s>>>(a);
    else
        kv4_write_kernel<false><<<grid, threads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4Io& a, cudaStream_t s)
{
    dim3 grid;
    unsigned threads;
    if (!io_grid(a, &grid, &threads)) return cudaErrorInvalidConfiguration;
    if (a.bf16)
        kv4_read_kernel<true><<<grid, threads, 0, s>>>(a);
    else
        kv4_read_kernel<false><<<grid, threads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace ffpa
