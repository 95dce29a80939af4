// The 4-bit K/V cache: its format, and the device code that every kernel over
// it shares.
//
// A value is an e2m1 code times the scale of its group of 16 along the head
// dim. The scale byte holds five exponent bits (bias 15) and three bits of
// mantissa, that is, the eight bits behind the sign of a 16-bit float, so
// scale byte << 7 IS the scale as fp16. A code has two significant bits and a
// scale four: every cached value has at most six and is exact in fp16 and in
// bf16 (the largest, 6 x 10240, and the smallest, 2^-18, are fp16 numbers).
// The matrix products over the cache therefore run on exact operands.
//
// Layout: pages of page_size tokens (a multiple of 16), in each page
// [2 (K, V)][Hkv][page_size / 16][D / 64] tiles of 16 tokens x 64 head dims.
// A tile is 512 bytes of codes and 64 scale bytes, in the order in which the
// lanes of a warp hold the A operand of mma.m16n8k16, so that a lane's four
// matrix steps are one 16-byte load without any exchange. With lane =
// 4 g + t:
//   K (A rows = tokens, k = head dims): bytes 16 lane + 8 hi hold token
//     g + 8 hi, head dims 16 t .. 16 t + 15 (one group); its scale is byte
//     512 + 2 lane + hi;
//   V (A = V^T: rows = head dims, k = tokens): bytes 16 lane + 4 j hold token
//     2 t + (j & 1) + 8 (j >> 1), head dims 8 g .. 8 g + 7 (half a group); the
//     scale of head dims 16 p .. 16 p + 15 is byte 512 + 16 p + 4 t + j.
// The even head dim of a pair is in a byte's low nibble.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "kv4.h"
#include "ptx.cuh"
#include "tile_common.cuh"

namespace ffpa {

__device__ __forceinline__ void kv4_invalid(uint32_t* status, uint32_t site, int b)
{
    atomicCAS(status, 0u, DEV_INVALID | (site << 8) | ((static_cast<uint32_t>(b) & 0xffffu) << 16));
}

// The two values of a 16-bit pair. (A bf16 is the upper half of its float: one operation each, half of what the
// conversion takes.)
template <bool BF16>
__device__ __forceinline__ float2 kv4_unpack(uint32_t w)
{
    if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return unpack2<BF16>(w);
}

// Byte offset of the first tile of strip `strip` (16 tokens) of a page.
__device__ __forceinline__ size_t kv4_strip_offset(const Kv4Cache& c, int Hkv, int chunks, int page, int kv, int h,
                                                   int strip)
{
    const size_t strips = static_cast<size_t>(c.page_size >> 4);
    return (((static_cast<size_t>(page) * 2 + kv) * Hkv + h) * strips + strip) * (static_cast<size_t>(chunks) * kKv4Tile);
}

// Four bytes of codes -> four fp16 pairs, a byte's low nibble in the low half.
__device__ __forceinline__ void kv4_decode8(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n"
        " .reg .b8 a, b, c, d;\n"
        " mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, a;\n"
        " cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n"
        " cvt.rn.f16x2.e2m1x2 %3, d;\n"
        "}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A scale byte (the low byte of s) as a pair of fp16 scales.
__device__ __forceinline__ uint32_t kv4_scale2(uint32_t s)
{
    const uint32_t h = (s & 0xffu) << 7;
    return h | (h << 16);
}

// Eight codes (four bytes) times their scale, as four fp16 pairs (exact).
__device__ __forceinline__ void kv4_dequant8(uint32_t w, uint32_t scale2, uint32_t (&h)[4])
{
    kv4_decode8(w, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = hmul2_u32(h[i], scale2);
}

// Quotients that have to fall on a border between two codes exactly when the
// true quotient does. An input has at most 11 significant bits, a scale 4 and
// a border 5: a true quotient that is not a border is at least 2^-11 of itself
// away from one, and a product with an approximate reciprocal is 2^-22 of it
// off. Rounding the product to a coarser grid that holds the borders puts it
// back on a border that it belongs on and moves it across none, so the
// nearest-even rounding that follows decides as it would on the true quotient.

// Scale byte of a group whose largest magnitude is amax (not NaN; values past
// 61440 = 6 x 10240, infinity among them, count as 61440, so that every cached
// value is a finite fp16 number): amax / 6, here to 16 significant bits, rounded
// to nearest even to three bits of mantissa, steps of 2^-17 below 2^-14.
__device__ __forceinline__ uint32_t kv4_scale_code(float amax)
{
    const float v = __uint_as_float((__float_as_uint(fminf(amax, 61440.f) * (1.f / 6.f)) + 0x80u) & ~0xffu);
    const uint32_t u = __float_as_uint(v);
    const uint32_t normal = ((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - ((127u - 15u) << 3);
    const uint32_t small = __float_as_uint(v + 64.f) - __float_as_uint(64.f);  // 2^-17 is the last place of 64
    return v < 6.103515625e-05f ? small : normal;                              // 2^-14
}

// 1 / scale (0 for a scale of 0), to 2^-22.
__device__ __forceinline__ float kv4_scale_rcp(uint32_t code)
{
    const float f = __half2float(__ushort_as_half(static_cast<unsigned short>(code << 7)));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(f));
    return code ? r : 0.f;
}

// |x| / scale on a grid of 2^-15 (the unit in the last place of 384; the
// smallest border is 1/4, which a different quotient misses by 2^-13), with
// the sign of x.
__device__ __forceinline__ float kv4_quotient(float x, float rcp)
{
    const float q = fmaf(fabsf(x), rcp, 384.f) - 384.f;
    return __uint_as_float(__float_as_uint(q) | (__float_as_uint(x) & 0x80000000u));
}

// Codes of eight values (four bytes): nearest even, saturating.
__device__ __forceinline__ uint32_t kv4_code8(const float (&x)[8], float rcp)
{
    uint32_t r;
    asm("{\n"
        " .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
        " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n"
        "}\n"
        : "=r"(r)
        : "f"(kv4_quotient(x[0], rcp)), "f"(kv4_quotient(x[1], rcp)), "f"(kv4_quotient(x[2], rcp)),
          "f"(kv4_quotient(x[3], rcp)), "f"(kv4_quotient(x[4], rcp)), "f"(kv4_quotient(x[5], rcp)),
          "f"(kv4_quotient(x[6], rcp)), "f"(kv4_quotient(x[7], rcp)));
    return r;
}

// Launches a kernel of the 4-bit cache. It starts before the one before it in the stream has ended, and waits for that
// end (pdl_wait) before it touches memory; every CTA does, so that its own end follows from it.
template <typename... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t s,
                             const Args&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Sequence range [p0, p0 + cnt) of cache positions and its first row in the
// 16-bit tensor, from the device arrays. A range outside the cache's blocks or
// the tensor's rows records DEV_INVALID and is not processed.
__device__ __forceinline__ bool kv4_range(const Kv4Io& a, int b, uint32_t site, int& p0, int& cnt, long long& row0)
{
    long long s = a.start ? a.start[b] : 0, n, r = 0;
    bool ok;
    if (a.cu) {
        r = a.cu[b];
        n = static_cast<long long>(a.cu[b + 1]) - r;
        ok = r >= 0 && n >= 0 && n <= a.N && r + n <= a.total;
    } else {
        n = a.count ? a.count[b] : a.N;
        ok = n >= 0 && n <= a.N;
    }
    ok = ok && s >= 0 && s + n <= static_cast<long long>(a.cache.max_blocks) * a.cache.page_size && s + n <= 0x7fffffffLL;
    if (!ok) {
        if (threadIdx.x == 0) kv4_invalid(a.status, site, b);
        return false;
    }
    p0 = static_cast<int>(s);
    cnt = static_cast<int>(n);
    row0 = r;
    return true;
}

}  // namespace ffpa
