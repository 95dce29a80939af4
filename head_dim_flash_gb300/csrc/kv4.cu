// Writing new tokens into the paged 4-bit K/V cache, and reading cached
// tokens back to 16 bits. The format is in kv4.cuh.
//
// Both are one pass over the data and bound by memory: a write reads 2 bytes
// and stores 9/16 of a byte per value, a read the reverse. A warp owns a tile
// of 16 tokens x 64 head dims of K and the one of V, whose lanes hold it in the
// order in which the cache stores it: a whole tile is one 16-byte store per
// lane plus the scales, and the 16-bit side moves 128 contiguous bytes per
// token. A CTA takes one or two strips of 16 tokens of one (sequence, kv head),
// its warps the head-dim chunks; a K and a V tile are in flight per warp, 32
// warps per SM. (Loading the next tiles ahead costs a third of the warps and
// is slower.) A strip that a sequence covers in part (its first and last) is
// stored token by token, and the cells of other tokens are left as they were.
//
// Measured on a GB300, D = 512, bf16, 13900 tokens of 8 heads (a write reads
// 227 MB): write 50 us, 5.8 TB/s, where a copy runs at 6.8 and plain reading of
// as much at 5.2; bound by issue slots (70% busy, about 9 instructions a value)
// as much as by memory. Read 49 us, 5.9 TB/s: four fifths of it is writing,
// and a plain fill runs at 3.9 TB/s. One token: 2.5 to 4 us, a launch. Started
// as dependents of the kernel before them: a prompt written and read back 100.5
// -> 99.1 us, one token 7.8 -> 7.1.
#include <type_traits>

#include "kv4.cuh"

namespace ffpa {
namespace {

constexpr int kIoWarps = 8;  // at most

// The range of one (sequence, kv head), and its strips that this CTA takes.
struct Range {
    int b, h;
    int p0, p1;         // cache positions
    int first, last;    // strips [first, last)
    long long row0;     // row of position p0 in the 16-bit tensor
};

__device__ __forceinline__ bool find_range(const Kv4Io& a, uint32_t site, Range& s)
{
    const unsigned u = static_cast<unsigned>(unit_id());  // at most 65535^2 units: below 2^32
    if (u >= static_cast<unsigned long long>(a.B) * a.Hkv) return false;
    s.b = static_cast<int>(u / static_cast<unsigned>(a.Hkv));
    s.h = static_cast<int>(u - static_cast<unsigned>(s.b) * static_cast<unsigned>(a.Hkv));
    int cnt;
    if (!kv4_range(a, s.b, site, s.p0, cnt, s.row0)) return false;
    s.p1 = s.p0 + cnt;
    const long long first = (s.p0 >> 4) + static_cast<long long>(blockIdx.x) * a.strips_per_cta;
    const int end = cnt > 0 ? ((s.p1 - 1) >> 4) + 1 : 0;
    if (first >= end) return false;
    s.first = static_cast<int>(first);
    s.last = static_cast<int>(first + a.strips_per_cta < end ? first + a.strips_per_cta : end);
    return true;
}

// Element offset of this (sequence, head)'s row of position 16 `strip`, which may lie before the range.
__device__ __forceinline__ long long strip_row(const Kv4Io& a, const Range& s, const View& v, int strip)
{
    return (a.cu ? 0 : s.b * v.sb) + s.h * v.sh + (s.row0 + (16LL * strip - s.p0)) * v.sn;
}

// The K tiles of consecutive strips: null (and the status word) where the page is outside the cache.
struct Tiles {
    uint8_t* at;
    int in;          // place of the strip in its page
    const int* row;  // its entry in the block table
};

__device__ __forceinline__ void page_tiles(const Kv4Io& a, const Range& s, uint32_t site, Tiles& x)
{
    const int page = *x.row;
    x.at = nullptr;
    if (page >= 0 && page < a.cache.num_pages)
        x.at = a.cache.data + kv4_strip_offset(a.cache, a.Hkv, a.D >> 6, page, 0, s.h, x.in);
    else if (threadIdx.x == 0)
        kv4_invalid(a.status, site, s.b);
}

__device__ __forceinline__ Tiles first_tiles(const Kv4Io& a, const Range& s, uint32_t site)
{
    const unsigned spp = a.cache.page_size >> 4, block = static_cast<unsigned>(s.first) / spp;
    Tiles x{nullptr, static_cast<int>(s.first - block * spp), a.cache.table + s.b * a.cache.table_stride + block};
    page_tiles(a, s, site, x);
    return x;
}

__device__ __forceinline__ void next_tiles(const Kv4Io& a, const Range& s, uint32_t site, Tiles& x)
{
    if (++x.in < a.cache.page_size >> 4) {
        if (x.at) x.at += (a.D >> 6) * kKv4Tile;
        return;
    }
    x.in = 0;
    ++x.row;
    page_tiles(a, s, site, x);
}

// The tokens of a tile that a lane holds: of K two (hi = 0, 1), of V four (j = 0 .. 3).
__device__ __forceinline__ int k_token(int g, int hi) { return g + 8 * hi; }
__device__ __forceinline__ int v_token(int t, int j) { return 2 * t + (j & 1) + 8 * (j >> 1); }

// ---------------------------------------------------------------- write
template <bool BF16>
using Pair = typename std::conditional<BF16, __nv_bfloat162, __half2>::type;

// Largest magnitudes of the low and the high halves of four words of 16-bit values; NaN where there is one.
template <bool BF16>
__device__ __forceinline__ Pair<BF16> amax4(uint32_t (&w)[4])
{
    Pair<BF16> x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __habs2(*reinterpret_cast<Pair<BF16>*>(&w[i]));
    return __hmax2_nan(__hmax2_nan(x[0], x[1]), __hmax2_nan(x[2], x[3]));
}

// The larger half of a in the low half, that of b in the high half.
template <bool BF16>
__device__ __forceinline__ Pair<BF16> halves(Pair<BF16> a, Pair<BF16> b)
{
    const uint32_t x = *reinterpret_cast<uint32_t*>(&a), y = *reinterpret_cast<uint32_t*>(&b);
    uint32_t lo = __byte_perm(x, y, 0x5410), hi = __byte_perm(x, y, 0x7632);
    return __hmax2(*reinterpret_cast<Pair<BF16>*>(&lo), *reinterpret_cast<Pair<BF16>*>(&hi));
}

// The cache has no NaN, one is stored as zero.
template <bool BF16>
__device__ __forceinline__ void clear_nan(uint32_t (&w)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = kv4_unpack<BF16>(w[i]);
        if (v.x != v.x) w[i] &= 0xffff0000u;
        if (v.y != v.y) w[i] &= 0x0000ffffu;
    }
}

template <bool BF16>
__device__ __forceinline__ uint32_t codes(const uint32_t (&w)[4], float rcp)
{
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = kv4_unpack<BF16>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
    return kv4_code8(x, rcp);
}

__device__ __forceinline__ void load4(const uint16_t* p, uint32_t (&w)[4])
{
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
}

// 16 values, 32 bytes. In one access where every row is aligned to it: a lane's two halves of a sector then go out as
// one, which is worth 3% of a packed read (80.8 -> 78.7 us for 495 MB) and 2% of a write.
__device__ __forceinline__ void load8(const uint16_t* p, bool wide, uint32_t (&x)[4], uint32_t (&y)[4])
{
    if (wide) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                     : "l"(p));
    } else {
        load4(p, x);
        load4(p + 8, y);
    }
}

__device__ __forceinline__ void store8(uint16_t* p, bool wide, const uint4& x, const uint4& y)
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(x.x), "r"(x.y), "r"(x.z),
                     "r"(x.w), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "l"(p)
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = x;
        reinterpret_cast<uint4*>(p)[1] = y;
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kIoWarps * 32, 4) kv4_write_kernel(const Kv4Io a)
{
    pdl_wait();
    pdl_trigger();
    Range s;
    if (!find_range(a, VS_KV4_WRITE, s)) return;
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int chunks = a.D >> 6;
    const size_t v_off = static_cast<size_t>(a.Hkv) * (a.cache.page_size >> 4) * chunks * kKv4Tile;
    const uint16_t* k = static_cast<const uint16_t*>(a.k) + strip_row(a, s, a.vk, s.first) + g * a.vk.sn + t * 16;
    const uint16_t* v = static_cast<const uint16_t*>(a.v) + strip_row(a, s, a.vv, s.first) + 2 * t * a.vv.sn + g * 8;
    const long long k8 = 8 * a.vk.sn, v1 = a.vv.sn, v8 = 8 * a.vv.sn;

    // one tile of K (two tokens, 16 head dims of each per lane) and of V (four tokens, eight head dims)
    struct Data {
        uint32_t k[2][2][4], v[4][4];
    };
    const uint16_t *kr = k, *vr = v;  // the next strip's rows
    auto load = [&](int strip, Data& d) {
        const int lo = s.p0 - 16 * strip, hi = s.p1 - 16 * strip;  // tokens of the strip in the range
        if (lo <= 0 && hi >= 16) {
#pragma unroll
            for (int x = 0; x < 2; ++x) load8(kr + x * k8, a.wide, d.k[x][0], d.k[x][1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) load4(vr + (j & 1) * v1 + (j >> 1) * v8, d.v[j]);
        } else {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const bool in = k_token(g, x) >= lo && k_token(g, x) < hi;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) d.k[x][y][e] = 0;
                    if (in) load4(kr + x * k8 + 8 * y, d.k[x][y]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) d.v[j][e] = 0;
                if (v_token(t, j) >= lo && v_token(t, j) < hi) load4(vr + (j & 1) * v1 + (j >> 1) * v8, d.v[j]);
            }
        }
        kr += 2 * k8;
        vr += 2 * v8;
    };
    auto store = [&](int strip, int ch, Data& d, uint8_t* tiles) {
        // magnitudes stay 16-bit pairs (a maximum is exact) down to one per group
        Pair<BF16> mk[2], mv[4];
        for (;;) {
            mk[0] = __hmax2_nan(amax4<BF16>(d.k[0][0]), amax4<BF16>(d.k[0][1]));
            mk[1] = __hmax2_nan(amax4<BF16>(d.k[1][0]), amax4<BF16>(d.k[1][1]));
            Pair<BF16> all = __hmax2_nan(mk[0], mk[1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mv[j] = amax4<BF16>(d.v[j]);
                all = __hmax2_nan(all, mv[j]);
            }
            const float2 f = kv4_unpack<BF16>(*reinterpret_cast<uint32_t*>(&all));
            if (f.x == f.x && f.y == f.y) break;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                clear_nan<BF16>(d.k[x][0]);
                clear_nan<BF16>(d.k[x][1]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) clear_nan<BF16>(d.v[j]);
        }
        __syncwarp();
        uint32_t kc[4], ks[2], vc[4];
        Pair<BF16> m = halves<BF16>(mk[0], mk[1]);
        float2 f = kv4_unpack<BF16>(*reinterpret_cast<uint32_t*>(&m));
        ks[0] = kv4_scale_code(f.x);
        ks[1] = kv4_scale_code(f.y);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float rcp = kv4_scale_rcp(ks[x]);
            kc[2 * x] = codes<BF16>(d.k[x][0], rcp);
            kc[2 * x + 1] = codes<BF16>(d.k[x][1], rcp);
        }
        // a V group's halves are in lanes g and g ^ 1: the even one finds the scales of tokens 0 and 1, the odd one
        // those of 2 and 3
        const bool odd = g & 1;
        Pair<BF16> v01 = halves<BF16>(mv[0], mv[1]), v23 = halves<BF16>(mv[2], mv[3]);
        Pair<BF16> mine = odd ? v23 : v01, other = odd ? v01 : v23;
        uint32_t got = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t*>(&other), 4);
        m = __hmax2(mine, *reinterpret_cast<Pair<BF16>*>(&got));
        f = kv4_unpack<BF16>(*reinterpret_cast<uint32_t*>(&m));
        const uint32_t half = kv4_scale_code(f.x) | (kv4_scale_code(f.y) << 8);
        got = __shfl_xor_sync(0xffffffffu, half, 4);
        const uint32_t vs = odd ? got | (half << 16) : half | (got << 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) vc[j] = codes<BF16>(d.v[j], kv4_scale_rcp((vs >> (8 * j)) & 0xffu));
        if (!tiles) return;
        uint8_t* tile = tiles + ch * kKv4Tile;
        uint8_t* vtile = tile + v_off;
        uint8_t* scale = vtile + 512 + ((g >> 1) * 4 + t) * 4;
        const int lo = s.p0 - 16 * strip, hi = s.p1 - 16 * strip;
        if (lo <= 0 && hi >= 16) {
            *reinterpret_cast<uint4*>(tile + lane * 16) = make_uint4(kc[0], kc[1], kc[2], kc[3]);
            *reinterpret_cast<uint16_t*>(tile + 512 + lane * 2) = static_cast<uint16_t>(ks[0] | (ks[1] << 8));
            *reinterpret_cast<uint4*>(vtile + lane * 16) = make_uint4(vc[0], vc[1], vc[2], vc[3]);
            if (!(g & 1)) *reinterpret_cast<uint32_t*>(scale) = vs;
            return;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (k_token(g, x) >= lo && k_token(g, x) < hi) {
                *reinterpret_cast<uint2*>(tile + lane * 16 + 8 * x) = make_uint2(kc[2 * x], kc[2 * x + 1]);
                tile[512 + lane * 2 + x] = static_cast<uint8_t>(ks[x]);
            }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (v_token(t, j) >= lo && v_token(t, j) < hi) {
                *reinterpret_cast<uint32_t*>(vtile + lane * 16 + 4 * j) = vc[j];
                if (!(g & 1)) scale[j] = static_cast<uint8_t>(vs >> (8 * j));
            }
    };
    for (int ch = warp; ch < chunks; ch += warps) {
        kr = k + ch * 64;
        vr = v + ch * 64;
        Tiles tiles = first_tiles(a, s, VS_KV4_WRITE);
        for (int strip = s.first;;) {
            Data x;
            load(strip, x);
            store(strip, ch, x, tiles.at);
            if (++strip == s.last) break;
            next_tiles(a, s, VS_KV4_WRITE, tiles);
        }
    }
}

// ----------------------------------------------------------------- read
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

template <bool BF16>
__global__ void __launch_bounds__(kIoWarps * 32) kv4_read_kernel(const Kv4Io a)
{
    pdl_wait();
    pdl_trigger();
    Range s;
    if (!find_range(a, VS_KV4_READ, s)) return;
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int chunks = a.D >> 6;
    const size_t v_off = static_cast<size_t>(a.Hkv) * (a.cache.page_size >> 4) * chunks * kKv4Tile;
    uint16_t* k = static_cast<uint16_t*>(a.k) + strip_row(a, s, a.vk, s.first) + g * a.vk.sn + t * 16;
    uint16_t* v = static_cast<uint16_t*>(a.v) + strip_row(a, s, a.vv, s.first) + 2 * t * a.vv.sn + g * 8;
    const long long k8 = 8 * a.vk.sn, v1 = a.vv.sn, v8 = 8 * a.vv.sn;

    struct Data {
        uint4 k, v;
        uint32_t ks, vs;
    };
    uint16_t *kr = k, *vr = v;  // the next strip's rows
    auto load = [&](int ch, const uint8_t* tiles, Data& d) {
        if (!tiles) return;
        const uint8_t* tile = tiles + ch * kKv4Tile;
        d.k = __ldcs(reinterpret_cast<const uint4*>(tile + lane * 16));
        d.v = __ldcs(reinterpret_cast<const uint4*>(tile + v_off + lane * 16));
        d.ks = __ldcs(reinterpret_cast<const uint16_t*>(tile + 512 + lane * 2));
        d.vs = __ldcs(reinterpret_cast<const uint32_t*>(tile + v_off + 512 + ((g >> 1) * 4 + t) * 4));
    };
    auto store = [&](int strip, const Data& d) {
        const int lo = s.p0 - 16 * strip, hi = s.p1 - 16 * strip;  // tokens of the strip in the range
        const bool all = lo <= 0 && hi >= 16;
        const uint32_t kc[4] = {d.k.x, d.k.y, d.k.z, d.k.w}, vc[4] = {d.v.x, d.v.y, d.v.z, d.v.w};
        uint32_t h[4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (all || (k_token(g, x) >= lo && k_token(g, x) < hi)) {
                const uint32_t s2 = kv4_scale2(d.ks >> (8 * x));
                kv4_dequant8(kc[2 * x], s2, h);
                const uint4 lo8 = pack8<BF16>(h);
                kv4_dequant8(kc[2 * x + 1], s2, h);
                store8(kr + x * k8, a.wide, lo8, pack8<BF16>(h));
            }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (all || (v_token(t, j) >= lo && v_token(t, j) < hi)) {
                kv4_dequant8(vc[j], kv4_scale2(d.vs >> (8 * j)), h);
                *reinterpret_cast<uint4*>(vr + (j & 1) * v1 + (j >> 1) * v8) = pack8<BF16>(h);
            }
    };
    for (int ch = warp; ch < chunks; ch += warps) {
        kr = k + ch * 64;
        vr = v + ch * 64;
        Tiles tiles = first_tiles(a, s, VS_KV4_READ);
        for (int strip = s.first;;) {
            Data x;
            load(ch, tiles.at, x);
            if (tiles.at) store(strip, x);
            kr += 2 * k8;
            vr += 2 * v8;
            if (++strip == s.last) break;
            next_tiles(a, s, VS_KV4_READ, tiles);
        }
    }
}

// Completes the arguments. One warp per chunk, at most kIoWarps; CTAs along x cover the strips that N tokens can touch
// (one more when a start need not be a multiple of 16). A CTA takes two strips where there are enough to keep the SMs
// full: at D = 512 that is worth 6% of a prompt's write and 9% of a read against one; four cost 2 to 3% more than two.
bool io_grid(Kv4Io& a, dim3* grid, unsigned* threads)
{
    const long long strips = (static_cast<long long>(a.N) + (a.start ? 30 : 15)) >> 4;
    const long long units = static_cast<long long>(a.B) * a.Hkv, sms = num_sms() > 0 ? num_sms() : 152;
    a.strips_per_cta = strips * units >= 32 * sms ? 2 : 1;
    const int chunks = a.D >> 6;
    a.wide = ((reinterpret_cast<uintptr_t>(a.k) >> 1 | a.vk.sb | a.vk.sh | a.vk.sn) & 15) == 0;
    const int rounds = (chunks + kIoWarps - 1) / kIoWarps;
    *threads = 32u * static_cast<unsigned>((chunks + rounds - 1) / rounds);
    return unit_grid(static_cast<unsigned>((strips + a.strips_per_cta - 1) / a.strips_per_cta), units, grid);
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4Io& io, cudaStream_t s)
{
    Kv4Io a = io;
    dim3 grid;
    unsigned threads;
    if (!io_grid(a, &grid, &threads)) return cudaErrorInvalidConfiguration;
    return launch_dependent(a.bf16 ? kv4_write_kernel<true> : kv4_write_kernel<false>, grid, threads, 0, s, a);
}

cudaError_t launch_kv4_read(const Kv4Io& io, cudaStream_t s)
{
    Kv4Io a = io;
    dim3 grid;
    unsigned threads;
    if (!io_grid(a, &grid, &threads)) return cudaErrorInvalidConfiguration;
    return launch_dependent(a.bf16 ? kv4_read_kernel<true> : kv4_read_kernel<false>, grid, threads, 0, s, a);
}

}  // namespace ffpa
