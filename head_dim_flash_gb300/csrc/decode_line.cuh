// Decode forward over 16-bit caches of different lengths: beside a prefix that
// the whole batch shares, or with every cached token's attention weight added
// to its score.
//
// With few query rows the work is reading K and V once. The key tiles of all
// units (sequence, kv head, block of rows) form one line, the shared prefix's
// units at its front, and the line is cut into equal ranges, one per group of
// warps: ragged lengths keep every SM busy to the end. Each unit takes two tiles
// more of the line than it has, for its start and end (a batch of short contexts
// behind a prefix would otherwise fall to a few ranges: 106 us against 68). The cut
// is made on the device, from the lengths there. A range's first and last unit may reach
// into its neighbours': such a piece leaves a normalised O (fp32) and the log2
// of its sum in the workspace, and a second kernel joins them:
//   L = log2 sum_s 2^L_s,  O = sum_s 2^(L_s - L) O_s.
//
// A group's warps own 64-wide head-dim chunks of K and V (two each above
// D = 512). TMA brings tiles into the group's ring; scores S = Q K^T are partial
// per warp (mma.m16n8k16 over its chunks) and summed through shared memory, a
// warp an eighth of the tile or so, which it also exponentiates; P goes back
// through shared memory, and O += P V stays with the chunks, in registers. P's
// reference is a row's maximum some tiles ago: it is renewed, and O rescaled, only
// when a score lies more than 2^8 above it, so most tiles need no agreement on a
// maximum. The scores of tile t + 1 are issued before the values of tile t.
//
// A tile is a chain of waits (data, sum, P), about 400 instructions a warp at six
// cycles each. A tile of 32 keys at D = 512 takes as long to arrive (64 KiB at the
// SM's share of HBM: 1.4 us). Head dims that divide into two groups of four warps
// run two (D = 256); the others run fifteen warps in groups of their chunks over
// tiles of 16 keys (16 ragged sequences at D = 320, 16 rows: 87 us against 102 with
// one group of five). Sixteen compute warps and a producer do not fit: the register
// file is dealt out to warps by fours. Two groups of eight at D = 512 whose own
// warps issued the loads took 343 us for 8 x 16384 tokens, one group and a producer
// 326.
//
// Measured on a GB300 (bf16, this kernel alone): 8 sequences of 16384 tokens, 8 kv
// heads of D = 512, 4 rows, 2.15 GB: 317 us, 6.8 TB/s with the scores' 17 MB; 16
// ragged ones of 1 to 8000, D = 320, 16 rows, 441 MB: 78 us, of which 10 until the
// first tile and from the last one.
//
// The scoring form also stores the scores (fp32, log2 units: 4 bytes per row
// and key beside 4 D of K and V), and the second kernel turns them into weights
// with the joined sums: w_j = sum_r 2^(s_rj - L_r), added in the order of the
// rows.
//
// Rows behind a sequence's length hold anything: their scores are replaced,
// not multiplied, and their V rows are zeroed in shared memory.
#pragma once

#include <atomic>
#include <type_traits>

#include "cache_ops.h"
#include "kv4.cuh"

namespace ffpa {
namespace line {

constexpr float kLn2 = 0.693147180559945309f;
constexpr int kUnitPlaces = 2;    // of a unit in the line besides its tiles
constexpr float kTau = 8.f;       // a score may lie 2^8 above its row's reference
constexpr int kMaxStages = 12;
constexpr int kMaxGroups = 15;
constexpr int kLens = 1024;     // lengths staged in shared memory; longer batches read them from L2
constexpr int kLineThreads = 288;  // warps 0..7 compute, warp 8 TMA producer
// Fifteen compute warps and the producer, 128 registers a thread.
constexpr int kLineThreadsMany = 512;
// The first with three idle warps: three warpgroups of 168 registers a thread, of
// which the two that compute take 232 and the producer's keeps 40.
constexpr int kLineThreadsWide = 384;
static_assert(2 * 232 + 40 == 3 * 168, "no more registers than the launch gives");
constexpr int kJoinThreads = 256;

enum LineSite : uint32_t { LS_PROD = 0x58, LS_FULL, LS_DRAIN };

struct LineGeo {
    int many;            // the variant with many warps
    int shift;           // keys of a tile: 1 << shift
    int chunks, warps, groups, stages, stage_bytes;
    int rows;            // query rows of a unit (16 or 32)
    int R, rblocks;      // rows of a kv head's group, their blocks
    int Rp, rblocks_p;   // the same for the shared prefix's units (rblocks_p = 0: not in the line)
    int tiles_p;         // tiles of one prefix unit
    int ranges;          // groups of the whole grid
    float *o_cut, *l_cut;      // [2 * ranges][rows][D], [2 * ranges][rows]
    float *o_whole, *l_whole;  // [B * Hq * Nq][D] (shared), [B * Hq * Nq]: units inside one range
    float *o_whole_p, *l_whole_p;  // [Hkv * Rp][D], [Hkv * Rp]
    int* before;         // [B + 1]: places of the line before each sequence's units; of the whole line
    float* scores;       // [B * Hq * Nq][pitch]
    int pitch;
    // many rows: the prefix is the tensor cores' (launch_xchg, split over the keys)
    int splits, split_keys;
    float *o_split, *l_split;  // [splits][Hkv][Rp][D], [splits][Hkv][Rp]
    uint16_t* q_rows;          // [Hkv][Rp][D]: the queries as its rows
};

// A place in the line.
struct Spot {
    int b;        // sequence, -1: the shared prefix
    int hk, rb;
    int tile, tiles;
    int keys;     // of the unit
};

struct __align__(1024) LineStatic {
    uint64_t full[kMaxGroups][kMaxStages], empty[kMaxGroups][kMaxStages];
    struct {
        Spot at;         // first tile of the group's range
        int from, to;    // tiles of the line before its first and behind its last
    } start[kMaxGroups];
    int abort_flag;
};
static_assert(sizeof(LineStatic) == 4096, "static shared block must be whole KiB");

constexpr int kLineSmem = kMaxSmem - static_cast<int>(sizeof(LineStatic)) - kLens * 4;  // dynamic

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// Length of sequence b; one outside its cache counts as 0 (and is recorded by stage_lens).
__device__ __forceinline__ int clamp_len(const LineArgs& a, int b)
{
    const int n = a.lens ? a.lens[b] : a.f.pb.Nkv;
    return n >= 0 && n <= a.f.pb.Nkv ? n : 0;
}

__device__ __forceinline__ int tiles_of(const LineGeo& g, int keys)
{
    return static_cast<int>((static_cast<unsigned>(keys) + (1u << g.shift) - 1) >> g.shift);
}

// Places that a unit of so many tiles takes in the line: its start's, then a tile each.
__device__ __forceinline__ int places_of(int tiles) { return tiles > 0 ? tiles + kUnitPlaces : 0; }

// Places of the whole line (below 2^31), and the units that have tiles (by whole warps).
__device__ __forceinline__ void line_sums(const LineArgs& a, const LineGeo& g, const int* staged, int& total, int& units)
{
    const Problem& pb = a.f.pb;
    int t = 0, u = 0;
#pragma unroll 4
    for (int i = threadIdx.x & 31; i < pb.B; i += 32) {
        const int n = places_of(tiles_of(g, staged ? staged[i] : clamp_len(a, i)));
        t += n;
        u += n > 0;
    }
    t = __reduce_add_sync(0xffffffffu, t);
    u = __reduce_add_sync(0xffffffffu, u);
    const int per = pb.Hkv * g.rblocks;
    total = pb.Hkv * g.rblocks_p * places_of(g.tiles_p) + t * per;
    units = pb.Hkv * g.rblocks_p + u * per;
}

// What the joining kernel asks of the line (by a whole warp).
__device__ __forceinline__ void store_befores(const LineArgs& a, const LineGeo& g, const int* staged)
{
    const Problem& pb = a.f.pb;
    const int lane = threadIdx.x & 31, per = pb.Hkv * g.rblocks;
    int run = 0;
    const int prefix = pb.Hkv * g.rblocks_p * places_of(g.tiles_p);
    for (int i0 = 0; i0 < pb.B; i0 += 32) {
        const int i = i0 + lane;
        const int n = i < pb.B ? places_of(tiles_of(g, staged ? staged[i] : clamp_len(a, i))) : 0;
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        if (i < pb.B) g.before[i] = prefix + (run + incl - n) * per;
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) g.before[pb.B] = prefix + run * per;
}

// The line cut into ranges, no more than it has places: the first `longer` hold
// one more than the others.
struct Cuts {
    int ranges, each, longer;
    __device__ Cuts(const LineGeo& g, int total)
    {
        ranges = min(g.ranges, total);
        each = ranges > 0 ? total / ranges : 0;
        longer = total - each * ranges;
    }
    __device__ int begin(int r) const { return r * each + min(r, longer); }
    __device__ int holding(int t) const  // the range that holds place t
    {
        const int head = longer * (each + 1);
        return t < head ? t / (each + 1) : longer + (t - head) / each;
    }
};

struct Line {
    const LineArgs& a;
    const LineGeo& g;
    const int* lens;  // staged, or null
    __device__ int len(int b) const { return lens ? lens[b] : clamp_len(a, b); }
    __device__ void enter(Spot& s) const  // the first unit with tiles at or behind sequence s.b
    {
        s.hk = s.rb = s.tile = 0;
        s.tiles = 0;
        while (s.b < a.f.pb.B) {
            s.keys = len(s.b);
            s.tiles = tiles_of(g, s.keys);
            if (s.tiles > 0) return;
            ++s.b;
        }
    }
    __device__ void next_unit(Spot& s) const
    {
        s.tile = 0;
        if (++s.rb < (s.b < 0 ? g.rblocks_p : g.rblocks)) return;
        s.rb = 0;
        if (++s.hk < a.f.pb.Hkv) return;
        s.hk = 0;
        ++s.b;
        enter(s);
    }
    // The first tile at or behind place t of the line, which lies before its end, and
    // how many tiles lie before it (called by whole warps).
    __device__ Spot find(int t, int& done) const
    {
        Spot s{};
        const int H = a.f.pb.Hkv;
        const int prefix_places = places_of(g.tiles_p), prefix = H * g.rblocks_p * prefix_places;
        if (t < prefix) {
            const int unit = t / prefix_places;
            s.b = -1;
            s.hk = unit / g.rblocks_p;
            s.rb = unit - s.hk * g.rblocks_p;
            s.tile = max(0, t - unit * prefix_places - kUnitPlaces);
            s.tiles = g.tiles_p;
            s.keys = a.Np;
            done = unit * g.tiles_p + s.tile;
            return s;
        }
        t -= prefix;
        done = H * g.rblocks_p * g.tiles_p;
        const int per = H * g.rblocks, lane = threadIdx.x & 31;
        s.b = a.f.pb.B;
        for (int i0 = 0, run = 0, units = 0; i0 < a.f.pb.B; i0 += 32) {
            const int tiles = i0 + lane < a.f.pb.B ? tiles_of(g, len(i0 + lane)) : 0, n = places_of(tiles);
            int incl = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += o;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, (run + incl) * per > t);
            const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
            if (past) {
                const int at = __ffs(past) - 1;
                const int first = run + __shfl_sync(0xffffffffu, incl - n, at);
                units += __popc(some & ((1u << at) - 1));
                s.b = i0 + at;
                s.tiles = __shfl_sync(0xffffffffu, tiles, at);
                const int rest = t - first * per, places = places_of(s.tiles);
                const int unit = rest / places;
                s.tile = max(0, rest - unit * places - kUnitPlaces);
                s.hk = unit / g.rblocks;
                s.rb = unit - s.hk * g.rblocks;
                s.keys = len(s.b);
                done += (first - units * kUnitPlaces) * per + unit * s.tiles + s.tile;
                return s;
            }
            run += __shfl_sync(0xffffffffu, incl, 31);
            units += __popc(some);
        }
        return s;
    }
};

// Row r of a unit: its (sequence, query head within the group, query).
__device__ __forceinline__ void row_of(int r, int b, int Nq, int R, int& bb, int& gg, int& i)
{
    bb = b;
    if (b < 0) {
        bb = r / R;
        r -= bb * R;
    }
    gg = r / Nq;
    i = r - gg * Nq;
}

// Shared memory of a group besides its ring: partial scores, P, maxima and sums.
__host__ __device__ constexpr int exchange_bytes(int warps, int mt, int nt)
{
    return warps * (mt * nt * 2) * 256 + mt * (nt / 2) * 512 + (mt * nt * 2) * 32 + warps * mt * 64;
}

// Keys of a tile: as many as the registers of a variant's rows and chunks leave room for.
template <int MT, int CC, bool MANY>
__host__ __device__ constexpr int tile_keys() { return CC == 1 && !MANY ? 32 : 16; }

template <int MT, int CC, bool MANY>
__host__ __device__ constexpr int line_threads()
{
    return MANY ? kLineThreadsMany : MT == 1 && CC == 1 ? kLineThreads : kLineThreadsWide;
}

// W: warps of a group where the variant has one number of them, else 0.
template <bool BF16, int MT, int CC, bool MANY, int W, bool SCORE>
__global__ void __launch_bounds__(line_threads<MT, CC, MANY>(), 1)
    line_kernel(const __grid_constant__ CUtensorMap tK, const __grid_constant__ CUtensorMap tV,
                const __grid_constant__ CUtensorMap tKp, const __grid_constant__ CUtensorMap tVp, const LineArgs a,
                const LineGeo g)
{
    constexpr int KT = tile_keys<MT, CC, MANY>(), NT = KT / 8, ROWS = 16 * MT;
    constexpr int SLOTS = MT * NT * 2;  // float2 a lane holds of a tile's scores
    const Problem& pb = a.f.pb;
    const int warps = W ? W : g.warps;
    __shared__ LineStatic sh;
    __shared__ int s_len[kLens];
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = g.stages, compute = g.groups * warps;  // warps behind these: idle, and the producer
    if (smem_u32(smem) & 1023u) {
        pdl_wait();
        if (threadIdx.x == 0) atomicCAS(a.f.ctl.status, 0u, 5u | (0xffu << 8));
        return;
    }
    if (threadIdx.x < g.groups * S) {
        mbar_init(&sh.full[threadIdx.x / S][threadIdx.x % S], 1);
        mbar_init(&sh.empty[threadIdx.x / S][threadIdx.x % S], warps);
    }
    if (threadIdx.x == 0) {
        sh.abort_flag = 0;
        prefetch_tmap(&tK);
        prefetch_tmap(&tV);
        if (g.rblocks_p) {
            prefetch_tmap(&tKp);
            prefetch_tmap(&tVp);
        }
    }
    fence_barrier_init();
    pdl_wait();  // from here on, what the kernel before wrote
    pdl_trigger();
    if (a.lens)
        for (int i = threadIdx.x; i < pb.B; i += blockDim.x) {
            const int n = a.lens[i];
            const bool good = n >= 0 && n <= pb.Nkv;
            if (!good && blockIdx.x == 0)
                atomicCAS(a.f.ctl.status, 0u, DEV_INVALID | (VS_LINE << 8) | ((static_cast<uint32_t>(i) & 0xffffu) << 16));
            if (pb.B <= kLens) s_len[i] = good ? n : 0;
        }
    __syncthreads();
    const Line line{a, g, a.lens && pb.B <= kLens ? s_len : nullptr};
    int total, units;
    line_sums(a, g, line.lens, total, units);
    const Cuts cuts(g, total);
    volatile int* abort_p = &sh.abort_flag;
    uint32_t* status = a.f.ctl.status;
    const uint64_t lim = a.f.ctl.limit_ns;
    const uint32_t half_bytes = static_cast<uint32_t>(g.stage_bytes / 2);
    // neighbouring ranges go to different SMs: a line of few tiles does not crowd a few of them
    auto range_of = [&](int group) { return group * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x); };
    auto ring_of = [&](int group) { return smem + static_cast<size_t>(group) * S * g.stage_bytes; };
    // where the groups' ranges begin and end: a warp for each
    for (int job = warp; job < 2 * g.groups; job += blockDim.x >> 5) {
        auto& start = sh.start[job >> 1];
        const int r = range_of(job >> 1) + (job & 1);
        int done = total - units * kUnitPlaces;
        Spot at{};
        if (r < cuts.ranges) at = line.find(cuts.begin(r), done);
        if (lane == 0) {
            if (job & 1) {
                start.to = done;
            } else {
                start.at = at;
                start.from = done;
            }
        }
    }
    __syncthreads();
    auto tiles_in = [&](int group) { return max(0, sh.start[group].to - sh.start[group].from); };  // 0: no range

    constexpr bool kWide = line_threads<MT, CC, MANY>() == kLineThreadsWide;
    constexpr int kProducer = MANY ? 15 : 8;
    if (warp >= kProducer) {
        // ------------------------------------------------------ producer
        if constexpr (kWide) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp > kProducer) return;
        // lane 2 i loads K of group i, lane 2 i + 1 its V; the groups take turns
        const int group = min(lane >> 1, g.groups - 1);
        const int mine = lane >> 1 < g.groups ? tiles_in(group) : 0;
        const int n_most = __reduce_max_sync(0xffffffffu, mine);
        Spot ahead = sh.start[group].at;
        uint64_t* const full = sh.full[group];
        uint8_t* const ring = ring_of(group) + (lane & 1) * half_bytes;
        int st = 0, issued = 0;
        uint32_t phase = 1;
        bool go = true;
        for (int t = 0; t < n_most; ++t) {
            if (t < mine && go) {
                go = mbar_wait(&sh.empty[group][st], phase, abort_p, status, lim, LS_PROD);
                if (go) {
                    if ((lane & 1) == 0) mbar_arrive_expect_tx(&full[st], g.stage_bytes);
                    const CUtensorMap* m = ahead.b < 0 ? (lane & 1 ? &tVp : &tKp) : (lane & 1 ? &tV : &tK);
                    tma_load_5d(ring + st * g.stage_bytes, m, &full[st], 0, ahead.tile * KT, 0, ahead.hk, max(ahead.b, 0));
                    ++issued;
                    if (++ahead.tile == ahead.tiles && t + 1 < mine) line.next_unit(ahead);
                }
            }
            if (++st == S) {
                st = 0;
                phase ^= 1u;
            }
        }
        // no copy in flight when the CTA leaves. K's and V's lanes may have stopped
        // apart when a wait ran out: a stage that lacks one of them is not waited for
        const int both = min(issued, __shfl_xor_sync(0xffffffffu, issued, 1));
        if ((lane & 1) == 0)
            for (int t = max(0, both - S); t < both; ++t) {
                int dummy = 0;
                if (!mbar_wait(&full[t % S], (t / S) & 1, &dummy, status, lim, LS_DRAIN, false)) break;
            }
        __syncwarp();
        if (blockIdx.x == 0) store_befores(a, g, line.lens);  // with nothing left to load
        return;
    }
    if constexpr (kWide) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int group = warp / warps, wg = warp - group * warps;
    const int range = range_of(group);
    const int n = warp < compute ? tiles_in(group) : 0;
    uint8_t* const ring = ring_of(group);
    float2* const part = reinterpret_cast<float2*>(smem + static_cast<size_t>(g.groups) * S * g.stage_bytes) +
                         group * exchange_bytes(warps, MT, NT) / 8;       // [warps][slot][lane] partial scores
    uint32_t* const p_s = reinterpret_cast<uint32_t*>(part + warps * SLOTS * 32);  // [mt][k16][lane][4]: P as A fragments
    float* const tops = reinterpret_cast<float*>(p_s + MT * (NT / 2) * 128);         // [slot][8 rows]: maxima
    float* const sums = tops + SLOTS * 8;                                            // [warps][ROWS]
    auto sync_group = [&] {
        if (warps > 1)
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(warps * 32) : "memory");
        else
            __syncwarp();
    };
    // the same, and whether x holds for any thread of the group
    auto any_group = [&](bool x) -> bool {
        if (warps == 1) {
            __syncwarp();
            return __any_sync(0xffffffffu, x);
        }
        uint32_t r;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\tbar.red.or.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(r)
            : "r"(1 + group), "r"(warps * 32), "r"(static_cast<uint32_t>(x))
            : "memory");
        return r != 0;
    };

    // (many rows) the queries as rows of the prefix' kernel, while the first tiles are on their way
    if (g.splits) {
        const int rows = pb.Hkv * g.Rp;
        for (int row = blockIdx.x * kProducer + warp; row < rows; row += gridDim.x * kProducer) {  // [Hkv][B][group][Nq]
            const int hk = row / g.Rp;
            int b, gg, i;
            row_of(row - hk * g.Rp, -1, pb.Nq, g.R, b, gg, i);
            const uint16_t* src = static_cast<const uint16_t*>(a.f.q) + b * pb.vq.sb +
                                  (hk * (pb.Hq / pb.Hkv) + gg) * pb.vq.sh + i * pb.vq.sn;
            uint16_t* dst = g.q_rows + static_cast<size_t>(row) * pb.D;
            for (int c = lane * 8; c < pb.D; c += 256)
                *reinterpret_cast<uint4*>(dst + c) = *reinterpret_cast<const uint4*>(src + c);
        }
    }
    if (n == 0) return;  // no barrier below spans groups
    // ------------------------------------------------------------ products
    const int my_chunks = CC == 1 ? 1 : (wg < g.chunks) + (wg + 8 < g.chunks);
    const int r_lo = lane >> 2, cpair = (lane & 3) * 2;
    const int R = g.R, G = pb.Hq / pb.Hkv;
    uint32_t qa[CC][4][MT][4];
    float o_acc[CC][8][MT][4];
    float m_run[MT][2], l_run[MT][2];  // references of my rows (every warp's alike), my share of their sums
    int jlim[MT][2];                // legal keys of the score rows: below this
    uint32_t pa[MT][NT / 2][4];
    float s[MT][NT][4];
    bool ok = true;
    Spot unit = sh.start[group].at;  // the unit whose scores are computed

    auto unit_rows = [&](const Spot& u) { return (u.b < 0 ? g.Rp : R) - u.rb * ROWS; };
    // queries and key limits of a unit
    auto enter_unit = [&](const Spot& u) {
        const int rows = unit_rows(u);
        const int total_keys = u.b < 0 ? 0 : (a.shared ? a.Np : 0) + u.keys;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const int r = mt * 16 + hi * 8 + r_lo;
                jlim[mt][hi] = 0;
                const uint16_t* q = nullptr;
                if (r < rows) {
                    int bb, gg, i;
                    row_of(u.rb * ROWS + r, u.b, pb.Nq, R, bb, gg, i);
                    q = static_cast<const uint16_t*>(a.f.q) + bb * pb.vq.sb + (u.hk * G + gg) * pb.vq.sh + i * pb.vq.sn;
                    int lim_j = u.keys;
                    if (pb.causal) {
                        // keys of the row's whole sequence, then of this unit
                        const int all = u.b < 0 ? a.Np + line.len(bb) : total_keys;
                        const int first = u.b < 0 ? 0 : all - u.keys;
                        lim_j = min(lim_j, all - pb.Nq + i + 1 - first);
                    }
                    jlim[mt][hi] = lim_j;
                }
#pragma unroll
                for (int cc = 0; cc < CC; ++cc)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                        for (int k8 = 0; k8 < 2; ++k8)
                            qa[cc][ks][mt][hi + 2 * k8] =
                                q && cc < my_chunks ? *reinterpret_cast<const uint32_t*>(
                                                          q + (wg + 8 * cc) * 64 + ks * 16 + k8 * 8 + cpair)
                                                    : 0u;
            }
    };
    // A unit's queries are wanted at once when it begins: they are called into L1
    // while the unit before it is at work (a row's 64 head dims are one line).
    auto touch_next = [&](Spot u) {
        line.next_unit(u);
        const int r = lane & 15;
        if (u.b >= pb.B || r >= unit_rows(u)) return;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (mt * 16 + r >= unit_rows(u)) break;
            int bb, gg, i;
            row_of(u.rb * ROWS + mt * 16 + r, u.b, pb.Nq, R, bb, gg, i);
            const uint16_t* q = static_cast<const uint16_t*>(a.f.q) + bb * pb.vq.sb + (u.hk * G + gg) * pb.vq.sh +
                                i * pb.vq.sn + (CC == 1 ? wg : wg + (lane >> 4) * 8) * 64;
            uint32_t x;
            if (CC == 1 || wg + (lane >> 4) * 8 < g.chunks)
                asm volatile("ld.global.ca.b32 %0, [%1];" : "=r"(x) : "l"(q));
        }
    };
    auto reset = [&] {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                m_run[mt][hi] = -INFINITY;
                l_run[mt][hi] = 0.f;
            }
#pragma unroll
            for (int cc = 0; cc < CC; ++cc)
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o_acc[cc][i][mt][e] = 0.f;
        }
    };
    int k_st = 0, v_st = 0;   // stages of the next scores and values
    uint32_t k_phase = 0;
    auto scores = [&] {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sh.full[group][k_st], k_phase, abort_p, status, lim, LS_FULL));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][i][e] = 0.f;
        const uint32_t kbase = smem_u32(ring + k_st * g.stage_bytes);
        if (++k_st == S) {
            k_st = 0;
            k_phase ^= 1u;
        }
        if (!ok) return;
#pragma unroll
        for (int cc = 0; cc < CC; ++cc) {
            if (cc >= my_chunks) break;
            const uint32_t blk = kbase + (wg + 8 * cc) * KT * 128;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int np = 0; np < NT / 2; ++np) {
                    uint32_t kb[4];
                    const int krow = np * 16 + (lane & 7) + ((lane >> 4) << 3);
                    ldsm4(blk + sw128_offset(krow, ks * 2 + ((lane >> 3) & 1)), kb);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma16816<BF16>(s[mt][np * 2], qa[cc][ks][mt], kb[0], kb[1]);
                        mma16816<BF16>(s[mt][np * 2 + 1], qa[cc][ks][mt], kb[2], kb[3]);
                    }
                }
        }
    };
    // Slot (mt, i, hi) of a tile: rows 16 mt + 8 hi + lane / 4, keys 8 i + 2 (lane % 4)
    // and the next; the warps take slots in turn.
    constexpr int kTurns = W ? (SLOTS + W - 1) / W : SLOTS;
    constexpr bool kEven = W != 0 && SLOTS % (W ? W : 1) == 0;
    auto slot_mt = [](int sl) { return MT == 1 ? 0 : sl / (NT * 2); };
    auto slot_i = [](int sl) { return (sl >> 1) & (NT - 1); };
    auto of_row = [&](const auto& v, int sl) { return MT == 1 || sl < NT * 2 ? (sl & 1 ? v[0][1] : v[0][0]) : (sl & 1 ? v[MT - 1][1] : v[MT - 1][0]); };
    // its scores: the sum over the group's warps, in log2 units, masked
    auto slot_scores = [&](int sl, const Spot& u) {
        float2 p[8];
        const float2* src = part + sl * 32 + lane;
        auto fetch = [&](int w) { p[w] = w < warps ? src[w * SLOTS * 32] : make_float2(0.f, 0.f); };
        fetch(0);
        fetch(1);
        float x = p[0].x + p[1].x, y = p[0].y + p[1].y;
        if (warps > 2) {
#pragma unroll
            for (int w = 2; w < 8; ++w) fetch(w);
            x += (p[2].x + p[3].x) + ((p[4].x + p[5].x) + (p[6].x + p[7].x));
            y += (p[2].y + p[3].y) + ((p[4].y + p[5].y) + (p[6].y + p[7].y));
        }
        const int j = (u.tile * KT) + slot_i(sl) * 8 + cpair, end = of_row(jlim, sl);
        return make_float2(j < end ? x * pb.scale_log2 : -INFINITY, j + 1 < end ? y * pb.scale_log2 : -INFINITY);
    };
    // A unit of up to eight rows leaves the matrix product's other eight idle: they
    // take the rows again with what P's rounding left over, so that P counts 16 bits
    // (bf16) or 22 and O's error is its own rounding's.
    auto is_fine = [&](const Spot& u) { return MT == 1 && unit_rows(u) <= 8; };
    // P of a tile in shared memory, from the references as they are, and its sums added
    // to `add`; true where a score lies too far above its reference
    auto exponentials = [&](const Spot& u, float (&add)[MT][2], bool first_try) {
        bool over = false;
        const bool fine = is_fine(u);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) add[mt][0] = add[mt][1] = 0.f;
#pragma unroll(W ? kTurns : 1)
        for (int j0 = 0; j0 < kTurns; ++j0) {
            const int sl = wg + j0 * warps;
            if (!kEven && sl >= SLOTS) break;
            if (fine && (sl & 1)) continue;
            const float2 x = slot_scores(sl, u);
            const int mt = slot_mt(sl), i = slot_i(sl), hi = sl & 1;
            if (SCORE && first_try) {
                const int r = u.rb * ROWS + mt * 16 + hi * 8 + r_lo, j = u.tile * KT + i * 8 + cpair;
                if (r < R && j < u.keys)
                    *reinterpret_cast<float2*>(g.scores + ((static_cast<size_t>(u.b) * pb.Hkv + u.hk) * R + r) * g.pitch + j) = x;
            }
            const float ref = of_row(m_run, sl), mu = ref == -INFINITY ? 0.f : ref;
            over = over || fmaxf(x.x, x.y) > ref + kTau;
            const float p0 = ex2_approx(x.x - mu), p1 = ex2_approx(x.y - mu);
#pragma unroll
            for (int m = 0; m < MT; ++m)
                if (m == mt) {
                    add[m][0] += hi ? 0.f : p0 + p1;
                    add[m][1] += hi ? p0 + p1 : 0.f;
                }
            uint32_t* to = p_s + ((mt * (NT / 2) + (i >> 1)) * 32 + lane) * 4 + (i & 1) * 2 + hi;
            const uint32_t packed = pack2<BF16>(p0, p1);
            *to = packed;
            if (fine) {
                const float2 back = unpack2<BF16>(packed);
                to[1] = pack2<BF16>(p0 - back.x, p1 - back.y);
            }
        }
        return over;
    };
    auto softmax = [&](const Spot& u) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                part[(wg * SLOTS + (mt * NT + i) * 2) * 32 + lane] = make_float2(s[mt][i][0], s[mt][i][1]);
                part[(wg * SLOTS + (mt * NT + i) * 2 + 1) * 32 + lane] = make_float2(s[mt][i][2], s[mt][i][3]);
            }
        sync_group();
        float add[MT][2];
        if (any_group(exponentials(u, add, true))) {
            // new references: the rows' maxima so far (a unit's first tile comes here)
            for (int sl = wg; sl < SLOTS; sl += warps) {
                const float2 x = slot_scores(sl, u);
                float top = fmaxf(x.x, x.y);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                if ((lane & 3) == 0) tops[sl * 8 + r_lo] = top;
            }
            sync_group();
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float alpha[2];
#pragma unroll
                for (int hi = 0; hi < 2; ++hi) {
                    float top = m_run[mt][hi];
#pragma unroll
                    for (int i = 0; i < NT; ++i) top = fmaxf(top, tops[((mt * NT + i) * 2 + hi) * 8 + r_lo]);
                    alpha[hi] = top == -INFINITY ? 1.f : ex2_approx(m_run[mt][hi] - top);
                    m_run[mt][hi] = top;
                    l_run[mt][hi] *= alpha[hi];
                }
                if (is_fine(u)) alpha[1] = alpha[0];
#pragma unroll
                for (int cc = 0; cc < CC; ++cc)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o_acc[cc][i][mt][e] *= alpha[e >> 1];
            }
            exponentials(u, add, false);
            sync_group();
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            l_run[mt][0] += add[mt][0];
            l_run[mt][1] += add[mt][1];
#pragma unroll
            for (int kp = 0; kp < NT / 2; ++kp) {
                const uint4 v = *reinterpret_cast<const uint4*>(p_s + ((mt * (NT / 2) + kp) * 32 + lane) * 4);
                pa[mt][kp][0] = v.x;
                pa[mt][kp][1] = v.y;
                pa[mt][kp][2] = v.z;
                pa[mt][kp][3] = v.w;
            }
        }
    };
    auto values = [&](const Spot& u) {
        const uint32_t vbase = smem_u32(ring + v_st * g.stage_bytes) + half_bytes;
        const int valid = u.keys - u.tile * KT;
#pragma unroll
        for (int cc = 0; cc < CC; ++cc) {
            if (cc >= my_chunks) break;
            if (!ok) break;
            const uint32_t blk = vbase + (wg + 8 * cc) * KT * 128;
            if (valid < KT) {
                // rows behind the last key: zero (what lies there may be NaN)
                for (int e = valid * 8 + lane; e < KT * 8; e += 32)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(blk + e * 16), "r"(0) : "memory");
                fence_proxy_async_smem();  // the slot is TMA's again after this tile
                __syncwarp();
            }
#pragma unroll
            for (int kp = 0; kp < NT / 2; ++kp)
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    uint32_t vb[4];
                    const int vrow = kp * 16 + (lane & 7) + (((lane >> 3) & 1) << 3);
                    ldsm4_trans(blk + sw128_offset(vrow, np * 2 + (lane >> 4)), vb);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma16816<BF16>(o_acc[cc][np * 2][mt], pa[mt][kp], vb[0], vb[1]);
                        mma16816<BF16>(o_acc[cc][np * 2 + 1][mt], pa[mt][kp], vb[2], vb[3]);
                    }
                }
        }
        // K and V of this stage have been read
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[group][v_st]);
        if (++v_st == S) v_st = 0;
    };
    // the piece of unit u that this range holds: its tiles [first, last)
    auto finish = [&](const Spot& u, int first, int last) {
        const bool whole = first == 0 && last == u.tiles;
        const int rows = unit_rows(u);
        const size_t cut = static_cast<size_t>(2 * range + (first == 0 ? 1 : 0)) * ROWS;
        // the rows' sums: four lanes of each warp hold a share
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                float l = l_run[mt][hi];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                if ((lane & 3) == 0) sums[wg * ROWS + mt * 16 + hi * 8 + r_lo] = l;
            }
        sync_group();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const int r = mt * 16 + hi * 8 + r_lo;
                if (r >= rows) continue;
                const bool fine = is_fine(u);
                float l = 0.f;
                for (int w = 0; w < warps; ++w) l += sums[w * ROWS + r];
                // (a row that is not a number stays one: its sum is neither above 0 nor 0)
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const float l2 = l == 0.f ? -INFINITY : m_run[mt][hi] + log2f(l);
                const int ur = u.rb * ROWS + r;  // row of the kv head's group
                const size_t row = (static_cast<size_t>(max(u.b, 0)) * pb.Hkv + u.hk) * (u.b < 0 ? g.Rp : R) + ur;
                float* dst = nullptr;
                uint16_t* out = nullptr;
                if (!whole) {
                    dst = g.o_cut + (cut + r) * pb.D;
                } else if (u.b < 0) {
                    dst = g.o_whole_p + row * pb.D;
                } else if (a.shared) {
                    dst = g.o_whole + row * pb.D;
                } else {
                    int bb, gg, i;
                    row_of(ur, u.b, pb.Nq, R, bb, gg, i);
                    out = static_cast<uint16_t*>(a.f.o) + bb * pb.vo.sb + (u.hk * G + gg) * pb.vo.sh + i * pb.vo.sn;
                }
#pragma unroll
                for (int cc = 0; cc < CC; ++cc) {
                    if (cc >= my_chunks) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int col = (wg + 8 * cc) * 64 + i * 8 + cpair;
                        float v0 = o_acc[cc][i][mt][2 * hi], v1 = o_acc[cc][i][mt][2 * hi + 1];
                        if (hi == 0 && fine) {
                            v0 += o_acc[cc][i][mt][2];
                            v1 += o_acc[cc][i][mt][3];
                        }
                        v0 *= inv;
                        v1 *= inv;
                        if (out)
                            *reinterpret_cast<uint32_t*>(out + col) = pack2<BF16>(v0, v1);
                        else
                            *reinterpret_cast<float2*>(dst + col) = make_float2(v0, v1);
                    }
                }
                if (wg == 0 && (lane & 3) == 0) {
                    if (!whole)
                        g.l_cut[cut + r] = l2;
                    else if (u.b < 0)
                        g.l_whole_p[row] = l2;
                    else
                        g.l_whole[row] = l2;
                    if (out) a.f.lse[row] = l2 * kLn2;
                }
            }
    };

    reset();
    enter_unit(unit);
    int first = unit.tile;      // first tile of the unit in this range
    if (n > unit.tiles - unit.tile) touch_next(unit);
    scores();
    softmax(unit);
    for (int t = 0; t < n; ++t) {
        const Spot cur = unit;
        const bool more = t + 1 < n;
        bool fresh = false;
        if (++unit.tile == unit.tiles) {
            if (more) line.next_unit(unit);
            fresh = more;
        }
        if (more) {
            if (fresh) {
                enter_unit(unit);
                if (n - t - 1 > unit.tiles) touch_next(unit);
            }
            scores();
        }
        values(cur);
        if (fresh || !more) {
            finish(cur, first, cur.tile + 1);
            first = 0;
            reset();
        }
        if (more) softmax(unit);
    }
}

// ------------------------------------------------------------------ joining
// The pieces of a unit that begins at place s0: one per range that holds tiles of it.
// The first begins inside its range (cut slot 1 there), later ones at theirs (slot 0).
struct Pieces {
    int first, count;
    bool whole;  // one range holds it all: not in the cut slots
    __device__ Pieces(const Cuts& c, int s0, int tiles)
    {
        first = tiles > 0 ? c.holding(s0 + kUnitPlaces) : 0;
        count = tiles > 0 ? c.holding(s0 + kUnitPlaces + tiles - 1) - first + 1 : 0;
        whole = count == 1;
    }
    __device__ int slot(int i) const { return i == 0 ? 2 * first + 1 : 2 * (first + i); }
};

// A warp per query row (per row and 128 head dims where rows are few), then, when
// scoring, a CTA per kWeighKeys tokens of a kv head. Each warp finds its row's
// pieces by itself: three loads in a row, which many warps per SM hide better
// than sharing would save. LOADS pieces of a row are on their way at once: few
// registers, so many warps, where rows are many and their pieces few.
constexpr int kWeighKeys = 1024;
constexpr int kJoinWarps = kJoinThreads / 32;


template <bool BF16, bool SCORE, int LOADS>
__global__ void __launch_bounds__(kJoinThreads, LOADS > 8 ? 2 : SCORE ? 4 : 3) join_kernel(const LineArgs a, const LineGeo g, const int rows,
                                                            const int row_ctas, const int key_blocks,
                                                            const int parts)
{
    pdl_wait();
    pdl_trigger();
    const Problem& pb = a.f.pb;
    __shared__ float row_l[SCORE ? 512 : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int R = g.R;
    const long long cta = static_cast<long long>(blockIdx.x) + static_cast<long long>(gridDim.x) * blockIdx.y;
    const bool is_row = cta < row_ctas;
    int bh, block = 0, row = 0, part = 0;  // (sequence, kv head)
    if (is_row) {
        const unsigned unit = static_cast<unsigned>(cta) * kJoinWarps + warp;  // below 2^32: line_fits
        if (unit >= static_cast<unsigned>(rows) * parts) return;  // warps are on their own
        row = static_cast<int>(unit / parts);
        part = static_cast<int>(unit - static_cast<unsigned>(row) * parts);
        bh = row / R;
    } else {
        const unsigned rest = static_cast<unsigned>(cta - row_ctas);
        if (!SCORE || rest >= static_cast<unsigned>(pb.B) * pb.Hkv * key_blocks) return;
        bh = static_cast<int>(rest / key_blocks);
        block = static_cast<int>(rest - static_cast<unsigned>(bh) * key_blocks);
    }
    const int b = bh / pb.Hkv, hk = bh - b * pb.Hkv;
    const int len = clamp_len(a, b);
    if (!is_row && block * kWeighKeys >= len) return;
    const int before = g.before[b];
    const Cuts cuts(g, g.before[pb.B]);
    const int tiles = tiles_of(g, len);

    if (is_row) {
        const int r = row - bh * R;
        const int rb = r / g.rows, ur = r - rb * g.rows;
        const Pieces own(cuts, before + (hk * g.rblocks + rb) * places_of(tiles), tiles);
        if (!a.shared && own.whole) return;  // written by the first kernel
        const int rp = b * R + r, rbp = rp / g.rows, urp = rp - rbp * g.rows;
        const Pieces pre(cuts, (hk * g.rblocks_p + rbp) * places_of(g.tiles_p), g.rblocks_p ? g.tiles_p : 0);
        const int np = g.splits ? g.splits : pre.count, pieces = np + own.count;
        auto find = [&](int i, const float*& l, const float*& o) {
            size_t at;
            if (i < np && g.splits) {
                at = (static_cast<size_t>(i) * pb.Hkv + hk) * g.Rp + rp;
                l = g.l_split;
                o = g.o_split;
            } else if (i < np) {
                at = pre.whole ? static_cast<size_t>(hk) * g.Rp + rp : static_cast<size_t>(pre.slot(i)) * g.rows + urp;
                l = pre.whole ? g.l_whole_p : g.l_cut;
                o = pre.whole ? g.o_whole_p : g.o_cut;
            } else {
                at = own.whole ? static_cast<size_t>(bh) * R + r : static_cast<size_t>(own.slot(i - np)) * g.rows + ur;
                l = own.whole ? g.l_whole : g.l_cut;
                o = own.whole ? g.o_whole : g.o_cut;
            }
            l += at;
            o += at * pb.D;
        };
        const int gg = r / pb.Nq, qi = r - gg * pb.Nq;
        uint16_t* out = static_cast<uint16_t*>(a.f.o) + b * pb.vo.sb + (hk * (pb.Hq / pb.Hkv) + gg) * pb.vo.sh + qi * pb.vo.sn;
        // Most rows have up to 32 pieces, a lane for each; more are taken in turn.
        // A piece that is not a number counts in no maximum, but makes the sum one that is none.
        float top = -INFINITY, sum = 0.f, w0 = 0.f;
        bool live = false;  // a piece has keys
        const float *l = nullptr, *o0 = nullptr;
        if (lane < pieces) {
            find(lane, l, o0);
            w0 = *l;
            top = fmaxf(top, w0);
            live = w0 != -INFINITY;
        }
        for (int i = 32 + lane; i < pieces; i += 32) {
            const float* o;
            find(i, l, o);
            top = fmaxf(top, *l);
            live = live || *l != -INFINITY;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        live = __any_sync(0xffffffffu, live);
        if (top == -INFINITY) top = 0.f;
        w0 = lane < pieces ? exp2f(w0 - top) : 0.f;
        for (int c0 = part * 128; c0 < pb.D; c0 += parts * 128) {
            const int col = c0 + lane * 4;
            const bool mine = col < pb.D;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            sum = w0;
            for (int p0 = 0; p0 < pieces && live; p0 += 32) {
                const float* o = o0;
                float w = w0;
                if (p0) {
                    w = 0.f;
                    if (p0 + lane < pieces) {
                        find(p0 + lane, l, o);
                        w = exp2f(*l - top);
                    }
                    sum += w;
                }
                // several loads in flight; past the last piece, its own again with no weight
                const int n = min(32, pieces - p0);
                for (int k0 = 0; k0 < n; k0 += LOADS) {
                    float4 p[LOADS];
#pragma unroll
                    for (int k = 0; k < LOADS; ++k) {
                        const float* ok = reinterpret_cast<const float*>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), min(k0 + k, n - 1)));
                        if (mine) p[k] = *reinterpret_cast<const float4*>(ok + col);
                    }
#pragma unroll
                    for (int k = 0; k < LOADS; ++k) {
                        const float ws = __shfl_sync(0xffffffffu, w, min(k0 + k, n - 1));
                        const float wk = k0 + k < n ? ws : 0.f;
                        if (mine) {
                            v.x = fmaf(wk, p[k].x, v.x);
                            v.y = fmaf(wk, p[k].y, v.y);
                            v.z = fmaf(wk, p[k].z, v.z);
                            v.w = fmaf(wk, p[k].w, v.w);
                        }
                    }
                }
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            if (mine)
                *reinterpret_cast<uint2*>(out + col) =
                    make_uint2(pack2<BF16>(v.x * inv, v.y * inv), pack2<BF16>(v.z * inv, v.w * inv));
        }
        if (part == 0 && lane == 0) a.f.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
        return;
    }
    if constexpr (SCORE) {
        constexpr int kBatch = 512;
        static_assert(kWeighKeys == 4 * kJoinThreads, "four keys per thread");
        const int j = block * kWeighKeys + 4 * tid;
        float acc[4] = {}, old[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) old[k] = j + k < len ? a.weights[static_cast<size_t>(bh) * pb.Nkv + j + k] : 0.f;
        for (int rbase = 0; rbase < R; rbase += kBatch) {
            const int nr = min(kBatch, R - rbase);
            __syncthreads();
            // the rows' log2 sums, eight lanes to a row
            for (int q0 = warp * 4; q0 < nr; q0 += kJoinThreads / 8) {
                const int q = q0 + (lane >> 3), r = rbase + min(q, nr - 1);
                const int rb = r / g.rows, ur = r - rb * g.rows;
                const Pieces own(cuts, before + (hk * g.rblocks + rb) * places_of(tiles), tiles);
                float mx = -INFINITY, sum = 0.f;
                if (own.whole) {
                    mx = g.l_whole[static_cast<size_t>(bh) * R + r];
                    sum = 0.125f;  // of eight lanes
                } else {
#pragma unroll 4
                    for (int k = lane & 7; k < own.count; k += 8)
                        mx = fmaxf(mx, g.l_cut[static_cast<size_t>(own.slot(k)) * g.rows + ur]);
                }
#pragma unroll
                for (int d = 4; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                // (a piece that is not a number is in no maximum, and in the sum)
                if (!own.whole) {
                    if (mx == -INFINITY) mx = 0.f;
                    for (int k = lane & 7; k < own.count; k += 8)
                        sum += exp2f(g.l_cut[static_cast<size_t>(own.slot(k)) * g.rows + ur] - mx);
                }
#pragma unroll
                for (int d = 4; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                // a row that saw no key adds nothing: all its scores are -inf
                if ((lane & 7) == 0 && q < nr) row_l[q] = mx == -INFINITY || sum == 0.f ? 0.f : mx + log2f(sum);
            }
            __syncthreads();
            // eight rows' scores in flight; rows past the last are read again and not added
            const float* src = g.scores + (static_cast<size_t>(bh) * R + rbase) * g.pitch + j;
            for (int q0 = 0; q0 < nr && j < len; q0 += 8) {
                float4 x[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    x[q] = *reinterpret_cast<const float4*>(src + static_cast<size_t>(min(q0 + q, nr - 1)) * g.pitch);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q0 + q < nr) {
                        const float l2 = row_l[q0 + q];
                        acc[0] += exp2f(x[q].x - l2);
                        acc[1] += exp2f(x[q].y - l2);
                        acc[2] += exp2f(x[q].z - l2);
                        acc[3] += exp2f(x[q].w - l2);
                    }
            }
        }
        // (entries behind the last token are not touched: what the scores hold there is not added either)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (j + k < len) a.oweights[static_cast<size_t>(bh) * pb.Nkv + j + k] = old[k] + acc[k];
    }
}

struct LinePlan {
    LineGeo g;
    int ctas;
    int smem;
    size_t o_cut, l_cut, o_whole, l_whole, o_whole_p, l_whole_p, before, scores, o_split, l_split, q_rows, total;  // byte offsets
    Problem prefix;  // the prefix as one batch entry of Rp queries per kv head
};

template <bool BF16, int MT, int CC, int W, bool MANY = false>
cudaError_t launch_variant(const LineArgs& a, const LinePlan& p, const CUtensorMap* m, cudaStream_t s)
{
    auto kern = a.shared ? line_kernel<BF16, MT, CC, MANY, W, false> : line_kernel<BF16, MT, CC, MANY, W, true>;
    // the kernel's allowance of shared memory: once per device
    static std::atomic<uint64_t> allowed[2];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(allowed[a.shared].load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kLineSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) allowed[a.shared].fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_dependent(kern, dim3(p.ctas), line_threads<MT, CC, MANY>(), p.smem, s, m[0], m[1], m[2], m[3], a, p.g);
}

// The two kernels of a call, for one element type (each in a translation unit of its own).
template <bool BF16>
cudaError_t run_line(const LineArgs& a, const LinePlan& p, const CUtensorMap* m, cudaStream_t s)
{
    const LineGeo& g = p.g;
    if (g.chunks > 8) return launch_variant<BF16, 1, 2, 8>(a, p, m, s);
    if (g.rows == 32) return g.warps == 8 ? launch_variant<BF16, 2, 1, 8>(a, p, m, s) : launch_variant<BF16, 2, 1, 0>(a, p, m, s);
    switch (g.warps) {
    case 8: return launch_variant<BF16, 1, 1, 8>(a, p, m, s);
    case 4: return launch_variant<BF16, 1, 1, 4>(a, p, m, s);
    case 7: return launch_variant<BF16, 1, 1, 7, true>(a, p, m, s);
    case 6: return launch_variant<BF16, 1, 1, 6, true>(a, p, m, s);
    case 5: return launch_variant<BF16, 1, 1, 5, true>(a, p, m, s);
    case 3: return launch_variant<BF16, 1, 1, 3, true>(a, p, m, s);
    case 2: return launch_variant<BF16, 1, 1, 2, true>(a, p, m, s);
    default: return launch_variant<BF16, 1, 1, 1, true>(a, p, m, s);
    }
}

template <bool BF16>
cudaError_t run_join(const LineArgs& a, const LinePlan& p, cudaStream_t s)
{
    const Problem& pb = a.f.pb;
    const int rows = pb.B * pb.Hq * pb.Nq;
    const int key_blocks = a.shared ? 0 : (pb.Nkv + kWeighKeys - 1) / kWeighKeys;
    // a warp per 128 head dims of a row as long as one round of warps holds them
    const int slices = (pb.D + 127) >> 7;
    const bool many = static_cast<long long>(rows) * slices > 32LL * p.ctas;
    const int parts = many ? 1 : slices;
    const int row_ctas = static_cast<int>((static_cast<long long>(rows) * parts + kJoinWarps - 1) / kJoinWarps);
    const long long ctas = row_ctas + static_cast<long long>(pb.B) * pb.Hkv * key_blocks;
    const long long x = ctas < 0x40000000LL ? ctas : 0x40000000LL;
    const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>((ctas + x - 1) / x));
    auto join = a.shared ? (many ? join_kernel<BF16, false, 4> : join_kernel<BF16, false, 16>)
                         : (ctas > 2 * p.ctas ? join_kernel<BF16, true, 8> : join_kernel<BF16, true, 16>);
    return launch_dependent(join, grid, kJoinThreads, 0, s, a, p.g, rows, row_ctas, key_blocks, parts);
}

extern template cudaError_t run_line<true>(const LineArgs&, const LinePlan&, const CUtensorMap*, cudaStream_t);
extern template cudaError_t run_line<false>(const LineArgs&, const LinePlan&, const CUtensorMap*, cudaStream_t);
extern template cudaError_t run_join<true>(const LineArgs&, const LinePlan&, cudaStream_t);
extern template cudaError_t run_join<false>(const LineArgs&, const LinePlan&, cudaStream_t);

}  // namespace line
}  // namespace ffpa
