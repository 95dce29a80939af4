// Cutting a K/V cache to `keep` tokens per kv head: the `recent` last ones
// stay, and of the others those with the largest scores; of equal scores the
// earlier token. Kept tokens stay in their order.
//
// Two kernels. The first has one CTA per (sequence, kv head). A score becomes a
// 32-bit key in the order of its value; three passes over the keys, each a
// histogram of 11, 11 and 10 bits of those that agree with what is already
// known, find the smallest key that stays and how many that equal it do. A last
// pass in index order writes where each kept token was, and its score. The keys
// are a 512th of the cache's bytes at D = 512 and are read from L2 after the
// first pass; what bounds the kernel is the latency of its passes: 16384 tokens
// 19 us, 900 tokens 8. (The keys in registers over the passes: 22; one addition per
// bin and warp, by matching lanes: 31.)
//
// The second moves the rows, each read and written once: bound by memory (64 kv
// heads cut from 16384 to 8192 tokens, D = 512, 2.1 GB: 312 us, 6.7 TB/s, a copy's
// rate). Out of place its CTAs take pieces of the kept tokens. In place a row moves
// to where an earlier one was: a CTA owns 64 to 256 head dims of one tensor's kv
// head and takes all its tokens in order. Sources ascend and none lies below its
// target, so a batch's targets may be sources of its own, and are no later batch's:
// a barrier stands between a batch's reads and its writes, and the next batch may
// already be on its way.
#include "cache_ops.h"
#include "kv4.cuh"

namespace ffpa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelEach = 4;       // keys per thread and tile of the ordered pass
constexpr int kBins = 2048;
constexpr int kCopies = 4;        // of the histogram: scores crowd a few bins
constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 8;     // 16-byte pieces that a thread has in flight

// Keys ordered as the scores are; both zeros are one, NaN lies below everything.
__device__ __forceinline__ uint32_t score_key(float w)
{
    if (isnan(w)) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ bool evict_len(const EvictArgs& a, int b, int& n)
{
    n = a.lens[b];
    if (n >= 0 && n <= a.N) return true;
    if (threadIdx.x == 0)
        atomicCAS(a.status, 0u, DEV_INVALID | (VS_EVICT << 8) | ((static_cast<uint32_t>(b) & 0xffffu) << 16));
    return false;
}

// Sum over the threads before me, and over all (32 warps).
__device__ __forceinline__ int2 block_scan(int x, int* warp_sum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    __syncthreads();  // the last call's sums have been read
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int w = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += o;
    }
    const int before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    return make_int2(before + incl - x, __shfl_sync(0xffffffffu, w, 31));
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictArgs a)
{
    pdl_wait();
    pdl_trigger();
    __shared__ int hist[kCopies][kBins];
    __shared__ int warp_sum[32];
    __shared__ int found[2];
    const unsigned unit = static_cast<unsigned>(unit_id());
    if (unit >= static_cast<unsigned>(a.B) * a.Hkv) return;
    const int b = static_cast<int>(unit / a.Hkv), tid = threadIdx.x;
    const float* w = a.weights + static_cast<size_t>(unit) * a.N;
    float* ow = a.oweights + static_cast<size_t>(unit) * a.Nout;
    int* kept = a.kept + static_cast<size_t>(unit) * a.keep;
    int n;
    if (!evict_len(a, b, n)) {
        for (int i = tid; i < a.keep; i += kSelThreads) kept[i] = -1;
        return;
    }
    const int m = min(n, a.keep);
    for (int i = m + tid; i < a.keep; i += kSelThreads) kept[i] = -1;
    if (n <= a.keep) {
        for (int i = tid; i < m; i += kSelThreads) {
            kept[i] = i;
            if (!a.in_place) ow[i] = w[i];
        }
        return;
    }
    const int early = n - a.recent;       // tokens that compete
    const int places = a.keep - a.recent; // for this many: fewer than `early`
    // the smallest key that stays, from its upper bits down, and how many that equal it do
    uint32_t known = 0, bits = 0;
    int left = places;
    if (places > 0) {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int width = pass < 2 ? 11 : 10, shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            for (int i = tid; i < kCopies * kBins; i += kSelThreads) hist[0][i] = 0;
            __syncthreads();
            int* mine = hist[(tid >> 5) & (kCopies - 1)];
            for (int i = tid; i < early; i += kSelThreads) {
                const uint32_t key = score_key(w[i]);
                if ((key & bits) == known) atomicAdd(&mine[(key >> shift) & ((1u << width) - 1)], 1);
            }
            __syncthreads();
            // bins from the largest down, two per thread
            const int hi = kBins - 1 - 2 * tid;
            int c0 = 0, c1 = 0;
#pragma unroll
            for (int c = 0; c < kCopies; ++c) {
                c0 += hist[c][hi];
                c1 += hist[c][hi - 1];
            }
            const int above = block_scan(c0 + c1, warp_sum).x;
            if (above < left && above + c0 + c1 >= left) {
                const bool first = above + c0 >= left;
                found[0] = first ? hi : hi - 1;
                found[1] = left - above - (first ? 0 : c0);
            }
            __syncthreads();
            known |= static_cast<uint32_t>(found[0]) << shift;
            bits |= ((1u << width) - 1) << shift;
            left = found[1];
            __syncthreads();
        }
    } else {
        known = 0xffffffffu;  // no key of a score: none stays
        left = 0;
    }
    // kept tokens in index order; the first `left` of those that equal the border
    int done = 0, equal = 0;
    const int warp = tid >> 5, lane = tid & 31;
    for (int base = 0; base < n; base += kSelThreads * kSelEach) {
        float x[kSelEach];
        uint32_t gt[kSelEach], eq[kSelEach];  // of the warp's 32 tokens of each round
        int count = 0;
#pragma unroll
        for (int j = 0; j < kSelEach; ++j) {
            const int i = base + warp * 32 * kSelEach + j * 32 + lane;
            x[j] = i < n ? w[i] : 0.f;
            const uint32_t key = score_key(x[j]);
            gt[j] = __ballot_sync(0xffffffffu, i < n && (i >= early || key > known));
            eq[j] = __ballot_sync(0xffffffffu, i < early && key == known);
            count += __popc(gt[j]) + (__popc(eq[j]) << 16);
        }
        // a tile has 4096 tokens: both counts fit 16 bits
        const int2 sum = block_scan(lane == 0 ? count : 0, warp_sum);  // its barriers: the tile has been read
        const int mine = __shfl_sync(0xffffffffu, sum.x, 0);
        int g = done + (mine & 0xffff), e = equal + (mine >> 16);
        const uint32_t lower = (1u << lane) - 1;
#pragma unroll
        for (int j = 0; j < kSelEach; ++j) {
            const int i = base + warp * 32 * kSelEach + j * 32 + lane;
            const int e_before = e + __popc(eq[j] & lower);
            const bool is_gt = gt[j] >> lane & 1, is_eq = (eq[j] >> lane & 1) && e_before < left;
            if (is_gt || is_eq) {
                const int at = g + __popc(gt[j] & lower) + min(e_before, left);
                kept[at] = i;
                ow[at] = x[j];
            }
            g += __popc(gt[j]);
            e += __popc(eq[j]);
        }
        done += sum.y & 0xffff;
        equal += sum.y >> 16;
    }
}

// Rows [first, first + rows) of a (K or V, sequence, kv head): source, target and list.
struct Move {
    const uint16_t* src;
    uint16_t* dst;
    long long sn, on;
    const int* kept;
};

__device__ __forceinline__ bool find_move(const EvictArgs& a, Move& m)
{
    const unsigned u = static_cast<unsigned>(unit_id());
    if (u >= 2u * a.B * a.Hkv) return false;
    const unsigned unit = u >> 1;
    const int b = static_cast<int>(unit / a.Hkv), h = static_cast<int>(unit - static_cast<unsigned>(b) * a.Hkv);
    const View& vi = u & 1 ? a.vv : a.vk;
    const View& vo = u & 1 ? a.vov : a.vok;
    m.src = static_cast<const uint16_t*>(u & 1 ? a.v : a.k) + b * vi.sb + h * vi.sh;
    m.dst = static_cast<uint16_t*>(u & 1 ? a.ov : a.ok) + b * vo.sb + h * vo.sh;
    m.sn = vi.sn;
    m.on = vo.sn;
    m.kept = a.kept + static_cast<size_t>(unit) * a.keep;
    // the new length: this CTA alone still reads the old one
    if (blockIdx.x == 0 && (u & 1) == 0 && h == 0 && threadIdx.x == 0) {
        const int n = a.lens[b];
        if (n >= 0 && n <= a.N) a.olens[b] = min(n, a.keep);
    }
    return true;
}

__global__ void __launch_bounds__(kMoveThreads) evict_copy_kernel(const EvictArgs a, const int most, const int rows)
{
    pdl_wait();
    pdl_trigger();
    Move m;
    if (!find_move(a, m)) return;
    const int nv = a.D >> 3;  // 16-byte pieces of a row
    const int r0 = blockIdx.x * rows, r1 = min(r0 + rows, most);
    const int total = (r1 - r0) * nv;
    for (int i0 = threadIdx.x; i0 < total; i0 += kMoveThreads * kMoveBatch) {
        uint4 x[kMoveBatch];
        int from[kMoveBatch];
#pragma unroll
        for (int j = 0; j < kMoveBatch; ++j) {
            const int i = i0 + j * kMoveThreads;
            from[j] = i < total ? __ldg(m.kept + r0 + i / nv) : -1;
        }
#pragma unroll
        for (int j = 0; j < kMoveBatch; ++j) {
            const int i = i0 + j * kMoveThreads;
            if (from[j] >= 0) x[j] = __ldcs(reinterpret_cast<const uint4*>(m.src + from[j] * m.sn + i % nv * 8));
        }
#pragma unroll
        for (int j = 0; j < kMoveBatch; ++j) {
            const int i = i0 + j * kMoveThreads;
            if (from[j] >= 0) __stcs(reinterpret_cast<uint4*>(m.dst + (r0 + i / nv) * m.on + i % nv * 8), x[j]);
        }
    }
}

// In place: COLS head dims (as many as D leaves), tokens in order.
template <int THREADS, int COLS>
__global__ void __launch_bounds__(THREADS) evict_shift_kernel(const EvictArgs a, const int most)
{
    pdl_wait();
    pdl_trigger();
    Move m;
    if (!find_move(a, m)) return;
    const int col = blockIdx.x * COLS + threadIdx.x % (COLS / 8) * 8;
    constexpr int kStep = THREADS / (COLS / 8), kRows = kStep * kMoveBatch;
    const bool mine = col < a.D;
    uint4 x[kMoveBatch];
    // my rows of a batch; a token that stays where it is does not move
    auto load = [&](int r0, uint4 (&v)[kMoveBatch], uint32_t& moves) {
        moves = 0;
#pragma unroll
        for (int j = 0; j < kMoveBatch; ++j) {
            const int r = r0 + j * kStep + threadIdx.x / (COLS / 8);
            const int from = r < most ? __ldg(m.kept + r) : -1;
            if (mine && from > r) {
                v[j] = __ldcs(reinterpret_cast<const uint4*>(m.src + from * m.sn + col));
                moves |= 1u << j;
            }
        }
    };
    auto store = [&](int r0, const uint4 (&v)[kMoveBatch], uint32_t moves) {
#pragma unroll
        for (int j = 0; j < kMoveBatch; ++j) {
            const int r = r0 + j * kStep + threadIdx.x / (COLS / 8);
            if (moves >> j & 1) __stcs(reinterpret_cast<uint4*>(m.dst + r * m.on + col), v[j]);
        }
    };
    // two batches in turn: a copy of one to the other would wait for its loads
    uint4 y[kMoveBatch];
    uint32_t mx, my;
    load(0, x, mx);
    for (int r0 = 0; r0 < most; r0 += 2 * kRows) {
        load(r0 + kRows, y, my);  // (nothing past the last row)
        __syncthreads();          // the first batch has been read
        store(r0, x, mx);
        load(r0 + 2 * kRows, x, mx);
        __syncthreads();
        store(r0 + kRows, y, my);
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s)
{
    const int most = a.keep < a.N ? a.keep : a.N;  // tokens that a kv head can keep
    dim3 grid;
    const long long units = static_cast<long long>(a.B) * a.Hkv;
    if (!unit_grid(1, units, &grid)) return cudaErrorInvalidConfiguration;
    cudaError_t e = launch_dependent(evict_select_kernel, grid, kSelThreads, 0, s, a);
    if (e != cudaSuccess) return e;
    if (a.in_place) {
        // As wide as leaves a CTA for most places on the SMs, two each (64 kv heads of 16384 tokens, D = 512: 256
        // head dims 477 us, 128 512, 64 628); what a narrow CTA has in flight is what its threads hold: 512 of them
        // where CTAs are few (8 kv heads of 131072: 756 us, 256 threads 1200).
        const long long sms = num_sms() > 0 ? num_sms() : 152;
        auto fits = [&](int c) { return a.D >= c && 2 * units * ((a.D + c - 1) / c) >= 3 * sms / 2; };
        const int cols = fits(256) ? 256 : fits(128) ? 128 : 64;
        const long long ctas = (a.D + cols - 1) / cols;
        if (!unit_grid(static_cast<unsigned>(ctas), 2 * units, &grid)) return cudaErrorInvalidConfiguration;
        const bool few = 2 * units * ctas <= sms;
        auto kern = cols == 256   ? evict_shift_kernel<kMoveThreads, 256>
                    : cols == 128 ? evict_shift_kernel<kMoveThreads, 128>
                    : few         ? evict_shift_kernel<2 * kMoveThreads, 64>
                                  : evict_shift_kernel<kMoveThreads, 64>;
        return launch_dependent(kern, grid, few ? 2 * kMoveThreads : kMoveThreads, 0, s, a, most);
    }
    // pieces of 64 KiB, smaller where that leaves SMs idle
    int rows = 32768 / a.D;
    const long long sms = num_sms() > 0 ? num_sms() : 152;
    while (rows > 4 && (most + rows - 1) / rows * 2 * units < 4 * sms) rows >>= 1;
    if (!unit_grid(most > 0 ? (most + rows - 1) / rows : 1, 2 * units, &grid)) return cudaErrorInvalidConfiguration;
    return launch_dependent(evict_copy_kernel, grid, kMoveThreads, 0, s, a, most, rows);
}

}  // namespace ffpa
