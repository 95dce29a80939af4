// Decode / short-query forward over the paged 4-bit K/V cache.
//
// The operation is ffpa_decode_fwd's on the cached values: S = scale q K^T
// over the sequence's cached tokens (bottom-right causal), O = softmax(S) V,
// LSE = ln sum exp S. The work is reading the cache once: 9/16 of a byte per
// value, so at the HBM rate every SM turns about 42 codes per clock into 16-bit
// operands. That rules the design:
//   - both products run with the cached side as the A operand (16 tokens or 16
//     head dims) and the query rows as the N = 8 side of mma.m16n8k16:
//       S^T = K Q^T,   O^T = V^T P^T.
//     The tiles are stored in A-fragment order, so a lane dequantises its own
//     16 bytes (cvt.e2m1x2 and one fp16 product per pair, both exact) into the
//     fragments of four matrix steps, with no ldmatrix and no 16-bit copy of the
//     cache in shared memory. V's pairs run along tokens: the nibbles of two
//     tokens are interleaved before the conversion, which costs half of what
//     exchanging the converted halves would. The operands of both products are
//     fp16 for either element type: cached values and (power-of-two scaled)
//     queries are exact.
//   - a group of C warps works on a strip of tokens, each warp on up to four
//     64-wide head-dim chunks of it: partial scores are exchanged through shared
//     memory (none when C = 1), the softmax is computed by every warp, and O^T
//     stays in registers. One CTA per SM holds NG groups.
//   - a producer warp, one lane per group, streams the strips by bulk copies into
//     a K ring and a V ring per group.
//   - the softmax keeps a reference instead of the running maximum: it moves (and
//     O is rescaled) only when a score passes it by 2^14, so that the usual step
//     is one vote. P <= 2^14 and its row's largest is >= 2^6 in fp16.
//   - the strips of all (sequence, kv head, row block) units form one line, cut
//     into equal ranges, one per group: lengths live on the device, so the cut is
//     made there. A unit counts kUnitCost strips more than it has, for its start
//     and end. A group that covers a unit alone writes its outputs; parts of
//     others go to the workspace, those that the groups of a CTA end with joined
//     there first, and a second kernel joins the parts in a fixed order. It is
//     launched as a dependent, so its start overlaps the first kernel.
#include "kv4.cuh"

namespace ffpa {
namespace {

constexpr int kComputeWarps = 11;  // at most, and one producer warp: 168 registers per thread
constexpr int kThreads = (kComputeWarps + 1) * 32;
constexpr int kMaxStages = 4;
constexpr int kMaxGroups = kComputeWarps;
constexpr int kStepStrips = 2;     // strips of 16 tokens per step
constexpr int kUnitCost = 4;       // strips' worth of a unit's start and end
constexpr float kRefBelow = 6.f;   // the reference lies this far (log2) below the maximum it was taken from
constexpr float kRefSpan = 14.f;   // and is kept until a score is this far above it
constexpr float kLn2 = 0.693147180559945309f;

enum Kv4Site : uint32_t { KS_K = 0x7b, KS_V, KS_PROD, KS_DRAIN };

struct Kv4Geo {
    int chunks;      // D / 64
    int C;           // warps per group
    int NG;          // groups per CTA
    int rblocks;     // blocks of `rows` query rows per kv head's group of G * Nq
    int rows;        // 8 or 16
    int stages;
    int workers;     // groups of the whole grid
    float* part;     // [workers][2][rows][D] unnormalised partial O
    float* ml;       // [workers][2][rows][2] reference (log2) and sum
};

// K or V of a step
__host__ __device__ inline int stage_bytes(int chunks) { return kStepStrips * chunks * kKv4Tile; }

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Bounded wait for a copy, kept out of the loop's code. A wait that runs out raises the CTA's abort flag, after
// which no later one waits; another sequence's error in the status word does not end it.
__device__ __noinline__ void wait_slow(uint64_t* bar, uint32_t phase, volatile int* abort_flag, uint32_t* status,
                                       uint64_t limit_ns, uint32_t site)
{
    if (*abort_flag == 0) mbar_wait(bar, phase, abort_flag, status, limit_ns, site, false);
}

// 8 x 8 matrix of 16-bit values held as an MMA fragment -> its transpose.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Two words of eight codes (two tokens, the same head dims) -> the even and the odd head dims with the two tokens'
// codes side by side in each byte (the first in the low nibble).
__device__ __forceinline__ void interleave(uint32_t x, uint32_t y, uint32_t& even, uint32_t& odd)
{
    const uint32_t m = 0x0f0f0f0fu;
    even = (x & m) | ((y << 4) & ~m);
    odd = ((x >> 4) & m) | (y & ~m);
}

// The scales in bytes i and j of s, as an fp16 pair.
__device__ __forceinline__ uint32_t scale_pair(uint32_t s, int i, int j)
{
    return __byte_perm(s, 0, i | 0x40 | (j << 8) | 0x4000) << 7;
}

// Cached tokens of sequence b; 0 (and the status word) when the length is outside the block table.
__device__ __forceinline__ int cached_len(const Kv4Decode& a, int b)
{
    const int len = a.seq_lens[b];
    if (len < 0 || len > static_cast<long long>(a.cache.max_blocks) * a.cache.page_size) {
        kv4_invalid(a.f.ctl.status, VS_KV4_DECODE, b);
        return 0;
    }
    return len;
}

__device__ __forceinline__ int strips_of(int len) { return (len >> 4) + ((len & 15) != 0); }
// places of one unit on the line
__device__ __forceinline__ int cost_of(int len) { return len > 0 ? strips_of(len) + kUnitCost : 0; }

// A run of strips [s0, s1) of one unit within a group's range [.., end) of the line; `unit` is the line place where
// the unit begins, its first strip lies kUnitCost behind.
struct Piece {
    int b, hk, rb, len;
    int s0, s1;
    long long unit, end;
};

__device__ __forceinline__ void piece_end(Piece& p)
{
    const int n = strips_of(p.len);
    const long long left = p.end - p.unit - kUnitCost;
    p.s1 = left < n ? static_cast<int>(left) : n;
}

// The run that begins at place `at` of the line, in sequence b whose units begin at place `b_at`; false when the
// range holds no strip.
__device__ __forceinline__ bool first_piece(const Kv4Decode& a, const Kv4Geo& gm, Piece& p, long long at, long long end,
                                            int b, long long b_at)
{
    if (at >= end) return false;
    p.b = b;
    p.len = cached_len(a, b);
    p.end = end;
    const int cost = cost_of(p.len), u = static_cast<int>((at - b_at) / cost);
    p.unit = b_at + static_cast<long long>(u) * cost;
    p.hk = u / gm.rblocks;
    p.rb = u - p.hk * gm.rblocks;
    const int r = static_cast<int>(at - p.unit);
    p.s0 = r > kUnitCost ? r - kUnitCost : 0;
    piece_end(p);
    return p.s1 > p.s0;
}

__device__ __forceinline__ bool next_piece(const Kv4Decode& a, const Kv4Geo& gm, Piece& p)
{
    p.unit += cost_of(p.len);
    if (p.unit + kUnitCost >= p.end) return false;
    if (++p.rb == gm.rblocks) {
        p.rb = 0;
        if (++p.hk == a.f.pb.Hkv) {
            p.hk = 0;
            do {  // places are left, so a later sequence has tokens
                if (++p.b >= a.f.pb.B) return false;
                p.len = cached_len(a, p.b);
            } while (p.len == 0);
        }
    }
    p.s0 = 0;
    piece_end(p);
    return p.s1 > 0;
}

struct __align__(16) DecShared {
    uint64_t full_k[kMaxGroups][kMaxStages], full_v[kMaxGroups][kMaxStages];
    uint64_t empty_k[kMaxGroups][kMaxStages], empty_v[kMaxGroups][kMaxStages];
    long long sums[kThreads / 32];
    long long first_at[kMaxGroups];   // place where the units of each group's first sequence begin
    int first_b[kMaxGroups];
    int abort_flag;
    int last[kMaxGroups][3];          // sequence (-1: none), kv head and row block of the part a group ends with
    float ml[kMaxGroups][16][2];      // its references and sums
    uint32_t qmax[kComputeWarps][16]; // largest query magnitudes over a warp's chunks
};

template <int CH, int NB, bool SPLIT, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) decode_kv4_kernel(const Kv4Decode a, const Kv4Geo gm)
{
    pdl_trigger();
    const Problem& pb = a.f.pb;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int warps = blockDim.x >> 5;
    const int G = pb.Hq / pb.Hkv, R = G * pb.Nq;
    const int units_b = pb.Hkv * gm.rblocks;          // units per sequence
    __shared__ DecShared sh;
    extern __shared__ __align__(128) uint8_t smem[];

    // ---- the line's length and the sequence in which each of my groups begins
    long long chunk, total;
    {
        const int per = (pb.B + blockDim.x - 1) / blockDim.x;
        const int b0 = min(static_cast<int>(threadIdx.x) * per, pb.B), b1 = min(b0 + per, pb.B);
        long long sum = 0;
        for (int b = b0; b < b1; ++b) sum += cost_of(cached_len(a, b));
        long long incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += x;
        }
        if (lane == 31) sh.sums[warp] = incl;
        if (threadIdx.x < gm.NG * kMaxStages) {
            uint64_t* bar = &sh.full_k[0][0] + threadIdx.x;
            constexpr int kSet = kMaxGroups * kMaxStages;  // full_k, full_v, empty_k, empty_v
            mbar_init(bar, 1);
            mbar_init(bar + kSet, 1);
            mbar_init(bar + 2 * kSet, gm.C);
            mbar_init(bar + 3 * kSet, gm.C);
            fence_barrier_init();
        }
        if (threadIdx.x == 0) sh.abort_flag = 0;
        __syncthreads();
        total = 0;
        for (int w = 0; w < warps; ++w) {
            if (w < warp) incl += sh.sums[w];
            total += sh.sums[w];
        }
        total *= units_b;
        chunk = (total + gm.workers - 1) / gm.workers;
        const long long lo = (incl - sum) * units_b, hi = incl * units_b;
        for (int i = 0; i < gm.NG; ++i) {
            const long long at = (static_cast<long long>(blockIdx.x) * gm.NG + i) * chunk;
            if (at < lo || at >= hi || at >= total) continue;
            long long b_at = lo;
            for (int b = b0; b < b1; ++b) {
                const long long n = static_cast<long long>(cost_of(cached_len(a, b))) * units_b;
                if (at < b_at + n) {
                    sh.first_b[i] = b;
                    sh.first_at[i] = b_at;
                    break;
                }
                b_at += n;
            }
        }
        __syncthreads();
    }
    if (static_cast<long long>(blockIdx.x) * gm.NG * chunk >= total) return;

    const int st_bytes = stage_bytes(gm.chunks), strip_bytes = gm.chunks * kKv4Tile;
    auto range = [&](int grp, Piece& p) {
        const long long at = (static_cast<long long>(blockIdx.x) * gm.NG + grp) * chunk;
        return first_piece(a, gm, p, at, min(at + chunk, total), sh.first_b[grp], sh.first_at[grp]);
    };

    Piece cur{};
    bool pending = false;  // my group's last part is still in its registers
    const int group = warp / gm.C, wg = warp - group * gm.C;  // my group, my place in it
    // my chunks are chunk0 .. chunk0 + CH - 1; those before wg * CH are another warp's too, here with queries of zero
    const int chunk0 = min(wg * CH, gm.chunks - CH);
    float acc[CH][4][NB][4];
    float m[NB][2], l[NB][2];

    if (warp == warps - 1) {
        // ------------------------------------------------------------ producer: one lane per group
        bool more = lane < gm.NG;
        if (more) more = range(lane, cur);
        uint8_t* const ring_k = smem + static_cast<size_t>(lane) * 2 * gm.stages * st_bytes;
        uint8_t* const ring_v = ring_k + gm.stages * st_bytes;
        const int spp = a.cache.page_size >> 4;  // strips per page
        const size_t v_off = static_cast<size_t>(pb.Hkv) * spp * strip_bytes, page_bytes = 2 * v_off;
        int s = cur.s0, slot = 0, loads = 0;     // next strip; steps whose K was issued, with ring slot and parity
        uint32_t phase = 1;
        bool v_next = false;                     // K of the step is issued, its V is not
        const uint8_t *src0 = nullptr, *src1 = nullptr;
        int ns = 0;
        bool joint = false;                      // the two strips are neighbours in a page
        uint64_t t0 = global_timer_ns();
        while (__any_sync(0xffffffffu, more)) {
            bool moved = false;
            if (more) {
                uint64_t* empty = v_next ? &sh.empty_v[lane][slot] : &sh.empty_k[lane][slot];
                if (mbar_test(empty, phase)) {
                    moved = true;
                    uint64_t* bar = v_next ? &sh.full_v[lane][slot] : &sh.full_k[lane][slot];
                    uint8_t* dst = (v_next ? ring_v : ring_k) + slot * st_bytes;
                    if (!v_next) {
                        const int* row = a.cache.table + cur.b * a.cache.table_stride;
                        const int blk0 = s / spp, in0 = s - blk0 * spp;
                        ns = min(kStepStrips, cur.s1 - s);
                        joint = ns == 2 && in0 + 1 < spp;
                        const int blk1 = ns == 2 && !joint ? blk0 + 1 : blk0, in1 = joint ? in0 + 1 : 0;
                        int page0 = row[blk0], page1 = row[blk1];
                        if (static_cast<unsigned>(page0) >= static_cast<unsigned>(a.cache.num_pages) ||
                            static_cast<unsigned>(page1) >= static_cast<unsigned>(a.cache.num_pages)) {
                            // the sequence's rows are undefined, but the copies stay inside the cache
                            kv4_invalid(a.f.ctl.status, VS_KV4_DECODE, cur.b);
                            page0 = page1 = 0;
                        }
                        const uint8_t* head = a.cache.data + static_cast<size_t>(cur.hk) * spp * strip_bytes;
                        src0 = head + page0 * page_bytes + static_cast<size_t>(in0) * strip_bytes;
                        src1 = head + page1 * page_bytes + static_cast<size_t>(in1) * strip_bytes;
                    }
                    const size_t off = v_next ? v_off : 0;
                    mbar_arrive_expect_tx(bar, ns * strip_bytes);
                    bulk_load(dst, src0 + off, (joint ? 2 : 1) * strip_bytes, bar);
                    if (ns == 2 && !joint) bulk_load(dst + strip_bytes, src1 + off, strip_bytes, bar);
                    if (!v_next) {
                        ++loads;
                    } else {
                        s += ns;
                        if (++slot == gm.stages) {
                            slot = 0;
                            phase ^= 1u;
                        }
                        if (s >= cur.s1) {
                            more = next_piece(a, gm, cur);
                            s = 0;
                        }
                    }
                    v_next = !v_next;
                }
            }
            if (__any_sync(0xffffffffu, moved)) {
                t0 = global_timer_ns();
                continue;
            }
            __nanosleep(150);  // a copy has a whole step of slack
            bool stop = *reinterpret_cast<volatile int*>(&sh.abort_flag) != 0;
            if (global_timer_ns() - t0 > a.f.ctl.limit_ns) {
                stop = true;
                if (lane == 0) atomicCAS(a.f.ctl.status, 0u, DEV_TIMEOUT | (KS_PROD << 8) | (blockIdx.x << 16));
            }
            if (__any_sync(0xffffffffu, stop)) {
                // copies in flight end before the CTA does
                sh.abort_flag = 1;
                if (lane < gm.NG)
                    for (int k = max(0, loads - gm.stages); k < loads; ++k) {
                        const uint32_t ph = static_cast<uint32_t>((k / gm.stages) & 1);
                        mbar_wait(&sh.full_k[lane][k % gm.stages], ph, &sh.abort_flag, a.f.ctl.status, a.f.ctl.limit_ns,
                                  KS_DRAIN, false);
                        if (k + 1 < loads || !v_next)
                            mbar_wait(&sh.full_v[lane][k % gm.stages], ph, &sh.abort_flag, a.f.ctl.status,
                                      a.f.ctl.limit_ns, KS_DRAIN, false);
                    }
                break;
            }
        }
        if (lane < gm.NG) sh.last[lane][0] = -1;
        __syncwarp();
    } else {
        // ------------------------------------------------------------ compute warps
        const uint8_t* const ring_k = smem + static_cast<size_t>(group) * 2 * gm.stages * st_bytes;
        const uint8_t* const ring_v = ring_k + gm.stages * st_bytes;
        constexpr int kExch = kStepStrips * NB * 32;  // float4 per warp and buffer
        float4* const exch = reinterpret_cast<float4*>(smem + static_cast<size_t>(gm.NG) * 2 * gm.stages * st_bytes) +
                             group * 2 * gm.C * kExch + lane;
        const int exch_size = gm.C * kExch;  // float4 of one of the two buffers
        float4* ex = exch;               // the buffer in use
        // ring places: byte offset of the stage, its barrier and the barrier's parity
        const uint8_t *kp = ring_k, *vp = ring_v;
        uint64_t *kb_full = sh.full_k[group], *vb_full = sh.full_v[group];
        uint32_t k_phase = 0, v_phase = 0;
        constexpr int kEmpty = 2 * kMaxGroups * kMaxStages;  // from a full barrier to its empty one
        uint32_t qf[NB][CH][4][2];
        float c2[NB][2];                 // log2-domain scale of the scores
        float s[kStepStrips][NB][4];
        uint32_t pf[kStepStrips][NB][2];
        int limits[NB][2];               // first token that my columns' rows do not see
        int least = 0;                   // and that some row does not see
        auto arrived = [&](uint64_t* bar, uint32_t phase, uint32_t site) {
            if (!mbar_try_wait(smem_u32(bar), phase))
                wait_slow(bar, phase, &sh.abort_flag, a.f.ctl.status, a.f.ctl.limit_ns, site);
            __syncwarp();
        };

        // S^T of a step over my chunks: left in s, or in the exchange buffer. A step of one strip computes on what
        // the second one's place holds, and masks it.
        auto scores = [&]() {
            arrived(kb_full, k_phase, KS_K);
            const uint8_t* kb = kp + chunk0 * kKv4Tile;
#pragma unroll
            for (int i = 0; i < kStepStrips; ++i) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint8_t* tile = kb + i * strip_bytes + c * kKv4Tile;
                    const uint4 w = *reinterpret_cast<const uint4*>(tile + lane * 16);
                    const uint32_t sc = *reinterpret_cast<const uint16_t*>(tile + 512 + lane * 2);
                    const uint32_t lo = scale_pair(sc, 0, 0), hi = scale_pair(sc, 1, 1);
                    uint32_t x[4], y[4], z[4], u[4];
                    kv4_dequant8(w.x, lo, x);
                    kv4_dequant8(w.y, lo, y);
                    kv4_dequant8(w.z, hi, z);
                    kv4_dequant8(w.w, hi, u);
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        mma_f16_16816(s[i][n], x[0], z[0], x[1], z[1], qf[n][c][0][0], qf[n][c][0][1]);
                        mma_f16_16816(s[i][n], x[2], z[2], x[3], z[3], qf[n][c][1][0], qf[n][c][1][1]);
                        mma_f16_16816(s[i][n], y[0], u[0], y[1], u[1], qf[n][c][2][0], qf[n][c][2][1]);
                        mma_f16_16816(s[i][n], y[2], u[2], y[3], u[3], qf[n][c][3][0], qf[n][c][3][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(kb_full + kEmpty);
            kp += st_bytes;
            ++kb_full;
            if (kp == ring_v) {
                kp = ring_k;
                kb_full -= gm.stages;
                k_phase ^= 1u;
            }
            if (SPLIT) {
#pragma unroll
                for (int i = 0; i < kStepStrips; ++i)
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        ex[wg * kExch + (i * NB + n) * 32] =
                            make_float4(s[i][n][0], s[i][n][1], s[i][n][2], s[i][n][3]);
            }
        };

        // sums of the partial scores, mask, P^T fragments; tok: the step's first token
        auto softmax = [&](int ns, int tok, bool first) {
            if (SPLIT) {
                asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(gm.C * 32) : "memory");
                const float4* x = ex;
#pragma unroll
                for (int i = 0; i < kStepStrips; ++i)
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const float4 v0 = x[(i * NB + n) * 32], v1 = x[kExch + (i * NB + n) * 32];
                        s[i][n][0] = v0.x + v1.x;
                        s[i][n][1] = v0.y + v1.y;
                        s[i][n][2] = v0.z + v1.z;
                        s[i][n][3] = v0.w + v1.w;
                    }
                for (int w = 2; w < gm.C; ++w) {  // one order for every warp: all get the same bits
                    x += w == 2 ? 2 * kExch : kExch;
#pragma unroll
                    for (int i = 0; i < kStepStrips; ++i)
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            const float4 v = x[(i * NB + n) * 32];
                            s[i][n][0] += v.x;
                            s[i][n][1] += v.y;
                            s[i][n][2] += v.z;
                            s[i][n][3] += v.w;
                        }
                }
                ex = ex == exch ? exch + exch_size : exch;
            }
            // scores in log2 units above the reference; keys that a row does not see have none
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < kStepStrips; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][n][e] = fmaf(s[i][n][e], c2[n][e & 1], -m[n][e & 1]);
            if (tok + 16 * kStepStrips > least || ns < kStepStrips) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int i = 0; i < kStepStrips; ++i)
                            if (i >= ns || tok + 16 * i + g + 8 * (e >> 1) >= limits[n][e & 1]) s[i][n][e] = -INFINITY;
            }
            float top = -INFINITY;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < kStepStrips; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, s[i][n][e]);
            if (first || __any_sync(0xffffffffu, top > kRefSpan)) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int i = 0; i < kStepStrips; ++i) mx = fmaxf(mx, fmaxf(s[i][n][q], s[i][n][q + 2]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        // how far the reference moves; a row's keys come first, so one without any in the piece's first
                        // step has none in the piece
                        float up = mx - kRefBelow;
                        if (first ? mx == -INFINITY : up < 0.f) up = 0.f;
                        const float al = first ? 0.f : ex2_approx(-up);
                        m[n][q] += up;
                        l[n][q] *= al;
#pragma unroll
                        for (int i = 0; i < kStepStrips; ++i) {
                            s[i][n][q] -= up;
                            s[i][n][q + 2] -= up;
                        }
#pragma unroll
                        for (int c = 0; c < CH; ++c)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                acc[c][i][n][q] *= al;
                                acc[c][i][n][q + 2] *= al;
                            }
                    }
            }
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < kStepStrips; ++i) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = ex2_approx(s[i][n][e]);
                    l[n][0] += p[0] + p[2];
                    l[n][1] += p[1] + p[3];
                    // fp16 P: half a step of 2^-11, an eighth of what bf16 operands would cost
                    pf[i][n][0] = transpose8x8(pack2<false>(p[0], p[1]));
                    pf[i][n][1] = transpose8x8(pack2<false>(p[2], p[3]));
                }
        };

        // O^T += V^T P^T over my chunks
        auto values = [&](int ns, int tok) {
            arrived(vb_full, v_phase, KS_V);
            const uint8_t* vb = vp + chunk0 * kKv4Tile;
#pragma unroll
            for (int i = 0; i < kStepStrips; ++i) {
                // cells behind the last token hold anything, as does the place of a second strip that is not there:
                // their scales count as zero
                uint32_t keep = 0xffffffffu;
                if (i >= ns) {
                    keep = 0;
                } else if (tok + 16 * i + 16 > cur.len) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (tok + 16 * i + 2 * t + (j & 1) + 8 * (j >> 1) >= cur.len) keep &= ~(0xffu << (8 * j));
                }
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint8_t* tile = vb + i * strip_bytes + c * kKv4Tile;
                    const uint4 w = *reinterpret_cast<const uint4*>(tile + lane * 16);
                    const uint32_t sc = *reinterpret_cast<const uint32_t*>(tile + 512 + ((g >> 1) * 4 + t) * 4) & keep;
                    const uint32_t lo = scale_pair(sc, 0, 1), hi = scale_pair(sc, 2, 3);
                    uint32_t even, odd, a0[4], a1[4], a2[4], a3[4];
                    interleave(w.x, w.y, even, odd);
                    kv4_dequant8(even, lo, a0);
                    kv4_dequant8(odd, lo, a1);
                    interleave(w.z, w.w, even, odd);
                    kv4_dequant8(even, hi, a2);
                    kv4_dequant8(odd, hi, a3);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int n = 0; n < NB; ++n)
                            mma_f16_16816(acc[c][e][n], a0[e], a1[e], a2[e], a3[e], pf[i][n][0], pf[i][n][1]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(vb_full + kEmpty);
            vp += st_bytes;
            ++vb_full;
            if (vp == ring_v + gm.stages * st_bytes) {
                vp = ring_v;
                vb_full -= gm.stages;
                v_phase ^= 1u;
            }
        };

        // a part of the piece's rows to a slot of the workspace
        auto store_part = [&](size_t slot) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int r = n * 8 + 2 * t + q;
                    if (cur.rb * gm.rows + r >= R) continue;
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        if (chunk0 + c < wg * CH) continue;
                        float4* o = reinterpret_cast<float4*>(gm.part + (slot * gm.rows + r) * pb.D + (chunk0 + c) * 64 + 8 * g);
                        o[0] = make_float4(acc[c][0][n][q], acc[c][0][n][q + 2], acc[c][1][n][q], acc[c][1][n][q + 2]);
                        o[1] = make_float4(acc[c][2][n][q], acc[c][2][n][q + 2], acc[c][3][n][q], acc[c][3][n][q + 2]);
                    }
                    if (wg == 0 && g == 0) {
                        gm.ml[(slot * gm.rows + r) * 2] = m[n][q];
                        gm.ml[(slot * gm.rows + r) * 2 + 1] = l[n][q];
                    }
                }
        };
        const size_t worker = static_cast<size_t>(blockIdx.x) * gm.NG + group;

        bool more = range(group, cur);
        while (more) {
            // ---- Q of the piece's rows over my chunks, as B fragments: fp16, scaled by a power of two into its range
            // (bf16 has the wider one). A lane holds query g, head dims 16 t .. 16 t + 15 of every chunk.
            const int r0 = cur.rb * gm.rows;
            least = pb.causal ? cur.len - pb.Nq + 1 : cur.len;  // first token that some row does not see
            uint32_t amax[NB];  // magnitudes of 16-bit floats order as their bits do
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int r = r0 + n * 8 + g;
                const int h = cur.hk * G + r / pb.Nq, i = r % pb.Nq;
                const uint16_t* q = static_cast<const uint16_t*>(a.f.q) + cur.b * pb.vq.sb + h * pb.vq.sh + i * pb.vq.sn;
                amax[n] = 0;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    uint4 x = make_uint4(0, 0, 0, 0), y = x;
                    if (r < R && chunk0 + c >= wg * CH) {
                        const uint4* src = reinterpret_cast<const uint4*>(q + (chunk0 + c) * 64 + t * 16);
                        x = src[0];
                        y = src[1];
                    }
                    const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        qf[n][c][e >> 1][e & 1] = w[e];
                        if (BF16) amax[n] = max(amax[n], max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
                    }
                }
                if (BF16) {
                    amax[n] = max(amax[n], __shfl_xor_sync(0xffffffffu, amax[n], 1));
                    amax[n] = max(amax[n], __shfl_xor_sync(0xffffffffu, amax[n], 2));
                    if (SPLIT && t == 0) sh.qmax[warp][n * 8 + g] = amax[n];
                }
            }
            // (the steps of a piece have this barrier too, so the last piece's maxima are read by now)
            if (BF16 && SPLIT) asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(gm.C * 32) : "memory");
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                float mul = 1.f;
                if (BF16) {
                    if (SPLIT)
                        for (int w = 0; w < gm.C; ++w) amax[n] = max(amax[n], sh.qmax[group * gm.C + w][n * 8 + g]);
                    // largest magnitude to [2^14, 2^15); rows of zeros or that are not finite stay as they are
                    const int e = static_cast<int>(amax[n] >> 7);
                    if (amax[n] > 0 && e < 255) mul = __uint_as_float(static_cast<uint32_t>(min(14 + 127 - e, 126) + 127) << 23);
#pragma unroll
                    for (int c = 0; c < CH; ++c)
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float2 f = unpack2<true>(qf[n][c][k >> 1][k & 1]);
                            qf[n][c][k >> 1][k & 1] = pack2<false>(f.x * mul, f.y * mul);
                        }
                }
                const float scale = pb.scale_log2 / mul;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    c2[n][e] = __shfl_sync(0xffffffffu, scale, (2 * t + e) * 4);
                    limits[n][e] = pb.causal ? min(cur.len, least + (r0 + n * 8 + 2 * t + e) % pb.Nq) : cur.len;
                    m[n][e] = 0.f;
                    l[n][e] = 0.f;
                }
            }
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[c][i][n][e] = 0.f;

            // ---- the scores of a step are issued before the values of the one before
            for (int at = cur.s0;; at += kStepStrips) {
                const bool in = at < cur.s1;
                if (in) scores();
                if (at > cur.s0) values(min(kStepStrips, cur.s1 - at + kStepStrips), (at - kStepStrips) * 16);
                if (!in) break;
                softmax(min(kStepStrips, cur.s1 - at), at * 16, at == cur.s0);
            }
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    l[n][q] += __shfl_xor_sync(0xffffffffu, l[n][q], 4);
                    l[n][q] += __shfl_xor_sync(0xffffffffu, l[n][q], 8);
                    l[n][q] += __shfl_xor_sync(0xffffffffu, l[n][q], 16);
                    if (l[n][q] == 0.f) m[n][q] = -INFINITY;  // no keys, no reference
                }

            // ---- a whole unit's outputs, or a part of one
            if (cur.s0 == 0 && cur.s1 == strips_of(cur.len)) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int r = r0 + n * 8 + 2 * t + q;
                        if (r >= R) continue;
                        const int h = cur.hk * G + r / pb.Nq, i = r % pb.Nq;
                        const float inv = l[n][q] == 0.f ? 0.f : 1.f / l[n][q];
                        uint16_t* o = static_cast<uint16_t*>(a.f.o) + cur.b * pb.vo.sb + h * pb.vo.sh + i * pb.vo.sn;
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            if (chunk0 + c < wg * CH) continue;
                            uint32_t x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[e] = pack2<BF16>(acc[c][e][n][q] * inv, acc[c][e][n][q + 2] * inv);
                            *reinterpret_cast<uint4*>(o + (chunk0 + c) * 64 + 8 * g) = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                        if (wg == 0 && g == 0)
                            a.f.lse[(static_cast<long long>(cur.b) * pb.Hq + h) * pb.Nq + i] =
                                l[n][q] == 0.f ? -INFINITY : (m[n][q] + lg2_approx(l[n][q])) * kLn2;
                    }
                more = next_piece(a, gm, cur);
            } else {
                Piece next = cur;
                more = next_piece(a, gm, next);
                if (more) {
                    store_part(2 * worker);
                    cur = next;
                } else {
                    pending = true;
                }
            }
        }
        if (pending && wg == 0) {
            if (lane == 0) {
                sh.last[group][1] = cur.hk;
                sh.last[group][2] = cur.rb;
            }
            if (g == 0)
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        sh.ml[group][n * 8 + 2 * t + q][0] = m[n][q];
                        sh.ml[group][n * 8 + 2 * t + q][1] = l[n][q];
                    }
        }
    }
    __syncthreads();  // every copy has been read: the rings are free
    if (pending && wg == 0 && lane == 0) sh.last[group][0] = cur.b;
    __syncthreads();
    const bool compute = warp < warps - 1;

    // ---- neighbouring groups that end in the same unit join their parts in shared memory, each group a share of it
    int run0 = group, run1 = group;
    if (compute && pending) {
        auto same = [&](int i) {
            return sh.last[i][0] == cur.b && sh.last[i][1] == cur.hk && sh.last[i][2] == cur.rb;
        };
        while (run0 > 0 && same(run0 - 1)) --run0;
        while (run1 + 1 < gm.NG && same(run1 + 1)) ++run1;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int r = n * 8 + 2 * t + q;
                float mx = -INFINITY, sum = 0.f;
                for (int i = run0; i <= run1; ++i) mx = fmaxf(mx, sh.ml[i][r][0]);
                const float mu = mx == -INFINITY ? 0.f : mx;
                for (int i = run0; i <= run1; ++i) sum += sh.ml[i][r][1] * ex2_approx(sh.ml[i][r][0] - mu);
                const float f = ex2_approx(m[n][q] - mu);
                m[n][q] = mx;
                l[n][q] = sum;
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[c][i][n][q] *= f;
                        acc[c][i][n][q + 2] *= f;
                    }
            }
    }
    float4* const buf = reinterpret_cast<float4*>(smem) + lane;
    constexpr int kRegs = CH * 4 * NB;  // float4 per lane
    if (compute && pending) {
        float4* mine = buf + static_cast<size_t>(warp) * kRegs * 32;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    mine[((c * 4 + i) * NB + n) * 32] =
                        make_float4(acc[c][i][n][0], acc[c][i][n][1], acc[c][i][n][2], acc[c][i][n][3]);
    }
    __syncthreads();
    if (!compute || !pending) return;
    // the part goes to slot 1 of the run's last group
    const size_t slot = 2 * (static_cast<size_t>(blockIdx.x) * gm.NG + run1) + 1;
    const int r0 = cur.rb * gm.rows;
    for (int e = group - run0; e < kRegs; e += run1 - run0 + 1) {
        const int c = e / (4 * NB), i = e / NB % 4, n = e % NB;
        if (chunk0 + c < wg * CH) continue;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = run0; k <= run1; ++k) {
            const float4 v = buf[(static_cast<size_t>(k * gm.C + wg) * kRegs + e) * 32];
            x.x += v.x;
            x.y += v.y;
            x.z += v.z;
            x.w += v.w;
        }
        const int r = n * 8 + 2 * t;
        float* o = gm.part + (slot * gm.rows + r) * pb.D + (chunk0 + c) * 64 + 8 * g + 2 * i;
        if (r0 + r < R) *reinterpret_cast<float2*>(o) = make_float2(x.x, x.z);
        if (r0 + r + 1 < R) *reinterpret_cast<float2*>(o + pb.D) = make_float2(x.y, x.w);
    }
    if (group == run1 && wg == 0 && g == 0)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float* ml = gm.ml + (slot * gm.rows + n * 8 + 2 * t + q) * 2;
                ml[0] = m[n][q];
                ml[1] = l[n][q];
            }
}

// Joins the parts of units that several groups worked on; writes the rows of
// sequences without tokens. One CTA per query row and 128 head dims: its four
// warps take parts in turn, four head dims per lane.
constexpr int kJoinThreads = 128;

template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads) decode_kv4_join_kernel(const Kv4Decode a, const Kv4Geo gm)
{
    const Problem& pb = a.f.pb;
    __shared__ long long sums[2][kJoinThreads / 32];
    __shared__ float4 acc[kJoinThreads];
    extern __shared__ float weight[];  // [CTAs + 1], then the slots
    int* const slots = reinterpret_cast<int*>(weight) + gm.workers / gm.NG + 1;
    const long long row = blockIdx.x;
    const int i = static_cast<int>(row % pb.Nq), h = static_cast<int>(row / pb.Nq % pb.Hq);
    const int b = static_cast<int>(row / (static_cast<long long>(pb.Nq) * pb.Hq));
    const int G = pb.Hq / pb.Hkv, r = (h % G) * pb.Nq + i, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int units_b = pb.Hkv * gm.rblocks;
    long long total = 0, before = 0;  // places of the line, and those before sequence b
    for (int k = threadIdx.x; k < pb.B; k += kJoinThreads) {
        const int c = cost_of(cached_len(a, k));
        total += c;
        before += k < b ? c : 0;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, d);
        before += __shfl_xor_sync(0xffffffffu, before, d);
    }
    if (lane == 0) {
        sums[0][warp] = total;
        sums[1][warp] = before;
    }
    __syncthreads();
    total = before = 0;
    for (int w = 0; w < kJoinThreads / 32; ++w) {
        total += sums[0][w];
        before += sums[1][w];
    }
    total *= units_b;
    const int len = cached_len(a, b), n = strips_of(len);
    const int d = blockIdx.y * 128 + lane * 4;
    uint16_t* o = static_cast<uint16_t*>(a.f.o) + b * pb.vo.sb + h * pb.vo.sh + i * pb.vo.sn + d;
    if (n == 0) {
        pdl_wait();
        if (warp == 0 && d < pb.D) *reinterpret_cast<uint2*>(o) = make_uint2(0, 0);
        if (blockIdx.y == 0 && threadIdx.x == 0) a.f.lse[row] = -INFINITY;
        return;
    }
    // the unit's strips lie at [first, end) of the line; groups v0 .. v1 hold them
    const long long first = before * units_b + static_cast<long long>((h / G) * gm.rblocks + r / gm.rows) * cost_of(len) + kUnitCost;
    const long long end = first + n, chunk = (total + gm.workers - 1) / gm.workers;
    const int v0 = static_cast<int>(first / chunk), v1 = static_cast<int>((end - 1) / chunk);
    pdl_wait();
    if (v0 == v1) return;  // written by its group
    // v1 ends in this unit unless its range reaches strips of the next one; the parts that groups of a CTA end with
    // are in slot 1 of the last of them, a part that is followed by another unit is in slot 0
    const bool ends = min((v1 + 1LL) * chunk, total) <= end + kUnitCost;
    const int vl = ends ? v1 : v1 - 1, c0 = v0 / gm.NG, parts = vl / gm.NG - c0 + 1 + (ends ? 0 : 1);
    float mx = -INFINITY;
    for (int k = lane; k < parts; k += 32) {
        const bool tail = !ends && k == parts - 1;
        const int s = tail ? 2 * v1 : 2 * min(vl, (c0 + k) * gm.NG + gm.NG - 1) + 1;
        if (warp == 0) slots[k] = s;
        mx = fmaxf(mx, gm.ml[(static_cast<size_t>(s) * gm.rows + r % gm.rows) * 2]);
    }
#pragma unroll
    for (int e = 16; e; e >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, e));
    const float mu = mx == -INFINITY ? 0.f : mx;
    __syncthreads();
    float l = 0.f;
    for (int k = lane; k < parts; k += 32) {
        const float* ml = gm.ml + (static_cast<size_t>(slots[k]) * gm.rows + r % gm.rows) * 2;
        const float w = ex2_approx(ml[0] - mu);
        l += w * ml[1];
        if (warp == 0) weight[k] = w;
    }
#pragma unroll
    for (int e = 16; e; e >>= 1) l += __shfl_xor_sync(0xffffffffu, l, e);
    __syncthreads();
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (d < pb.D) {
#pragma unroll 4
        for (int k = warp; k < parts; k += kJoinThreads / 32) {
            const float w = weight[k];
            const float4 v = *reinterpret_cast<const float4*>(
                gm.part + (static_cast<size_t>(slots[k]) * gm.rows + r % gm.rows) * pb.D + d);
            x.x = fmaf(w, v.x, x.x);
            x.y = fmaf(w, v.y, x.y);
            x.z = fmaf(w, v.z, x.z);
            x.w = fmaf(w, v.w, x.w);
        }
    }
    acc[threadIdx.x] = x;
    __syncthreads();
    if (warp == 0 && d < pb.D) {
#pragma unroll
        for (int w = 1; w < kJoinThreads / 32; ++w) {
            const float4 v = acc[w * 32 + lane];
            x.x += v.x;
            x.y += v.y;
            x.z += v.z;
            x.w += v.w;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<uint2*>(o) = make_uint2(pack2<BF16>(x.x * inv, x.y * inv), pack2<BF16>(x.z * inv, x.w * inv));
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) a.f.lse[row] = l == 0.f ? -INFINITY : (mx + lg2_approx(l)) * kLn2;
}

struct Plan {
    Kv4Geo gm;
    int ctas;
    int nb, ch;
    int smem;
    size_t part_floats, bytes;
};

// Eight query rows per step up to G * Nq = 8, else blocks of sixteen. A warp
// holds O^T of its chunks in registers: at most four chunks of eight rows or two
// of sixteen (64 accumulators), dealt out evenly over the group's C warps.
Plan plan(const Problem& pb)
{
    Plan p{};
    Kv4Geo& gm = p.gm;
    const long long R = static_cast<long long>(pb.Hq / pb.Hkv) * pb.Nq;
    gm.chunks = pb.D >> 6;
    p.nb = R <= 8 ? 1 : 2;
    gm.rows = 8 * p.nb;
    gm.rblocks = static_cast<int>((R + gm.rows - 1) / gm.rows);
    const int most = p.nb == 1 ? 4 : 2;
    gm.C = (gm.chunks + most - 1) / most;
    p.ch = (gm.chunks + gm.C - 1) / gm.C;
    // at least two stages for every head dim: five groups with 184 KB of rings and 20 of exchange at D = 512
    for (gm.NG = kComputeWarps / gm.C; gm.NG > 1; --gm.NG) {
        const int exch = gm.C > 1 ? gm.NG * 2 * gm.C * kStepStrips * p.nb * 32 * 16 : 0;
        if (2 * gm.NG * 2 * stage_bytes(gm.chunks) + exch + 1024 + static_cast<int>(sizeof(DecShared)) <= kMaxSmem) break;
    }
    const int exch = gm.C > 1 ? gm.NG * 2 * gm.C * kStepStrips * p.nb * 32 * 16 : 0;
    const int ring = gm.NG * 2 * stage_bytes(gm.chunks);
    gm.stages = (kMaxSmem - 1024 - static_cast<int>(sizeof(DecShared)) - exch) / ring;
    if (gm.stages > kMaxStages) gm.stages = kMaxStages;
    p.smem = exch + gm.stages * ring;
    const int sms = num_sms();
    p.ctas = sms > 0 ? sms : 152;
    gm.workers = p.ctas * gm.NG;
    p.part_floats = static_cast<size_t>(gm.workers) * 2 * gm.rows * pb.D;
    p.bytes = (p.part_floats + static_cast<size_t>(gm.workers) * 2 * gm.rows * 2) * sizeof(float);
    return p;
}

template <int CH, int NB, bool SPLIT>
cudaError_t launch_variant(const Kv4Decode& a, const Plan& p, cudaStream_t s)
{
    auto* kernel = a.f.bf16 ? decode_kv4_kernel<CH, NB, SPLIT, true> : decode_kv4_kernel<CH, NB, SPLIT, false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, p.smem);
    if (e != cudaSuccess) return e;
    kernel<<<p.ctas, (p.gm.NG * p.gm.C + 1) * 32, p.smem, s>>>(a, p.gm);
    return cudaGetLastError();
}

// The chunks per warp that plan() can give, for one warp per group and for several.
cudaError_t launch_main(const Kv4Decode& a, const Plan& p, cudaStream_t s)
{
    if (p.nb == 1) {
        if (p.gm.C > 1) return p.ch == 3 ? launch_variant<3, 1, true>(a, p, s) : launch_variant<4, 1, true>(a, p, s);
        return p.ch == 1   ? launch_variant<1, 1, false>(a, p, s)
               : p.ch == 2 ? launch_variant<2, 1, false>(a, p, s)
               : p.ch == 3 ? launch_variant<3, 1, false>(a, p, s)
                           : launch_variant<4, 1, false>(a, p, s);
    }
    if (p.gm.C > 1) return launch_variant<2, 2, true>(a, p, s);
    return p.ch == 1 ? launch_variant<1, 2, false>(a, p, s) : launch_variant<2, 2, false>(a, p, s);
}

}  // namespace

size_t kv4_decode_workspace_bytes(const Problem& pb) { return plan(pb).bytes; }

cudaError_t launch_decode_kv4(const Kv4Decode& a, void* workspace, cudaStream_t s)
{
    Plan p = plan(a.f.pb);
    p.gm.part = static_cast<float*>(workspace);
    p.gm.ml = p.gm.part + p.part_floats;
    cudaError_t e = launch_main(a, p, s);
    if (e != cudaSuccess) return e;
    const Problem& pb = a.f.pb;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(pb.B) * pb.Hq * pb.Nq), (pb.D + 127) / 128);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 2 * (p.ctas + 1) * sizeof(float);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, a.f.bf16 ? decode_kv4_join_kernel<true> : decode_kv4_join_kernel<false>, a, p.gm);
}

}  // namespace ffpa
