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
//     queries are exact. (tcgen05 would want 128 rows of dequantised operands in
//     shared or tensor memory: the same conversions, and a store of each value.)
//   - a group of C warps works on a step of C * SW strips of 16 tokens. For the
//     scores each warp takes SW strips over the whole head dim, so a softmax is
//     computed once and its scores are never exchanged; for the values it takes
//     one or two 64-wide head-dim chunks over all strips, so O^T stays in
//     registers. Between the two, P goes through shared memory as ready operands.
//     A step has two barriers: after its scores (P is there) and after its values; two more where the softmax's
//     reference moves, as in a unit's first step.
//   - one warp of the group loads the K of the next step after the first barrier,
//     another its V after the second: each copy has the other half of a step to
//     arrive, so one place for K and one for V are enough. A lane copies the part
//     of a step that lies in one page: with one lane walking the pages, pages of
//     16 tokens cost 18% more time than pages of 64, now 4%.
//   - the softmax keeps a reference instead of the running maximum: it moves (and
//     O is rescaled) only when a score passes it by 2^14. P <= 2^14 and its row's
//     largest is >= 2^6 in fp16.
//   - P in fp16 costs as much as the rounding of an fp16 output, up to 1.4 times its error against 64 bits (one sequence
//     of 131000 tokens: 2.9e-4 where 2.1e-4 is the output's own). With up to four rows half of the matrix product's
//     eight columns are idle: for fp16 outputs they take the rows a second time, with the fp16 remainders of P, and the
//     two are added in the end (2.1e-4). That costs 0 to 1% at D >= 256, 2 to 3% below (118.3 -> 121.4 us at D = 64, 604
//     MB; 12.8 -> 12.9 one short sequence). More rows would need a second product of the same values: 108.5 -> 121 us for
//     eight rows, 144 -> 175 for sixteen (D = 512, 604 MB); they and bf16 outputs, whose own rounding is eight times
//     P's, keep one.
//   - the strips of all (sequence, kv head, row block) units form one line, cut
//     into equal ranges, one per group: lengths live on the device, so the cut is
//     made there. A unit counts a few strips more than it has, for its start and
//     end. A group that covers a unit alone writes its outputs; parts of others
//     go to the workspace, those that the groups of a CTA end with joined there
//     first, and a second kernel joins the parts in a fixed order. Ranges are not
//     shared out as groups become free: the shared counter between two barriers
//     cost 8 us of 108, and the tail that it evens out is bound by memory too.
//   - both kernels are launched as dependents of the one before them (31.3 -> 30.5
//     us of a short call).
//
// Measured on a GB300 (a copy runs at 6.77 TB/s), calls in a row, the cache not
// in the L2: 8 sequences of 16384 tokens, 8 kv heads, 4 query heads each,
// D = 512 (604 MB): 105 us, 5.8 TB/s; one sequence of 131000 tokens: 103 us.
// Bound by memory: 6 us pass until a group has its first keys, 96 are the steps
// (the last group is done 3 us after the median one), 3 the second kernel.
// Sixteen rows per head: 144 us for 600 MB at D = 512; 74 instructions and eight
// matrix products a tile, whose conversions (the ALU 44% busy), matrix unit (43%)
// and issue slots (54%) three or four warps per scheduler cannot overlap further.
// Short calls are mostly their start and end: one sequence of 2000 tokens takes
// 12.9 us, 4 until the first keys, 3 of steps, 6 for the second kernel and the
// launches; 64 sequences of 20 to 1000 tokens, 16 heads of D = 128 (69 MB), 26 us.
#include <atomic>

#include "kv4.cuh"

namespace ffpa {
namespace {

constexpr int kMaxWarps = 16;
constexpr float kRefBelow = 6.f;   // the reference lies this far (log2) below the maximum it was taken from
constexpr float kRefSpan = 14.f;   // and is kept until a score is this far above it
constexpr float kLn2 = 0.693147180559945309f;

enum Kv4Site : uint32_t { KS_K = 0x7b, KS_V, KS_DRAIN };

struct Kv4Geo {
    int rblocks;     // blocks of `rows` query rows per kv head's group of G * Nq
    int rows;        // 8 or 16
    int NG;          // groups per CTA
    int workers;     // groups of the whole grid
    int unit_cost;   // strips' worth of a unit's start and end
    int spp;         // strips per page
    int step_blk;    // a step moves by so many pages
    int step_in;     // and strips
    size_t v_off;    // bytes from a page's K to its V
    float* part;     // [workers][2][rows][D] unnormalised partial O
    float* ml;       // [workers][2][rows][2] reference (log2) and sum
};

// Shape of a CTA for N head-dim chunks and NB blocks of eight query rows.
// CH: two chunks of O^T per warp need the fewest exchanges and barriers, but one
// halves its registers (16 warps for sixteen rows) and saves the chunk that two
// warps of an odd N both compute. Two against one, us, at 76 and 605 MB of cache:
//   eight rows    N = 2: 26.7, 26.5 and 110, 131   N = 3: 27.5, 25.3 and 124, 118
//     N = 4: 25.4, 25.7 and 103, 106   N = 5: 26.2, 26.3 and 113, 108
//     N = 6: 25.0, 25.5 and 114, 103   N = 7: 26.2, 26.8 and 114, 120
//     N = 8: 25.7, 25.9 and 105, 108   N = 9: 27.2, 30.6 and 110, 127
//     N = 10: 27.2, 28.9 and 105, 128   N = 11: 27.9, 30.3 and 108, 120
//     N = 12: 27.6, 28.9 and 105, 111   N = 13: 31.0, 32.3 and 132, 127
//   sixteen rows  N = 2: 33.8, 31.9 and 153, 159   N = 3: 36.8, 32.8 and 172, 150
//     N = 4: 34.1, 33.2 and 146, 140   N = 5: 36.4, 37.9 and 148, 144
//     N = 6: 37.1, 36.6 and 155, 136   N = 7: 41.3, 40.4 and 163, 160
//     N = 8: 39.5, 39.4 and 156, 144   N = 9: 46.0, 47.2 and 176, 174
//     N = 10: 45.0, 44.1 and 167, 167   N = 11: 46.9, 46.1 and 154, 157
//     N = 12: 46.9, 46.3 and 149, 146
// So one for N = 3 with eight rows and N <= 8 with sixteen, but not N = 5 there;
// two elsewhere. Where the sizes disagree this is the smaller cache's side, and
// leaves 3 to 4% of large caches at N = 2 (sixteen rows) and 5, 9% at N = 6 (eight
// rows). N = 5 with sixteen rows, further: 23.9, 21.8 at 20 MB, 52.0, 53.0 at 152,
// 84.3, 83.8 at 303; 42.0, 43.9 over 16 contexts of 1 to 8000 tokens (102 MB), which
// end more often inside a step of one chunk's ten strips than of two chunks' six.
// From N = 14 on (13 with sixteen rows) a step with one chunk per warp does not fit.
// NG: as many groups as registers hold, 128 per thread where O^T takes 32 of
// them and 168 where it takes 64 (16 warps there spill: 155 -> 184 us at N = 5,
// 600 MB; the kept shapes spill 4 to 60 bytes: sixteen rows but for N = 6 and N >=
// 13, eight rows at N <= 2). SW: steps as long as shared memory then allows, from eight strips per
// warp in groups of one warp (142 -> 121 us at N = 1 against four, 600 MB) or
// two in others.
struct Shape {
    int CH;           // chunks per warp
    int C;            // warps per group
    int NG;           // groups per CTA
    int SW;           // strips that a warp scores per step
    int group_bytes;  // shared memory of a group
    int smem;
};
constexpr int kStaticBytes = 9 * 1024;  // at least the kernel's static shared memory and the system's

__host__ __device__ constexpr Shape shape_of(int N, int NB)
{
    Shape p{};
    const int room = kMaxSmem - kStaticBytes;
    p.CH = N == 1 || (NB == 1 ? N == 3 : N <= 8 && N != 5) ? 1 : 2;
    p.C = (N + p.CH - 1) / p.CH;
    p.NG = (p.CH * NB <= 2 ? 16 : 12) / p.C;
    for (p.SW = p.C > 1 ? 2 : 8;; p.SW >>= 1) {
        const int strips = p.C * p.SW;
        p.group_bytes = 2 * strips * N * kKv4Tile + N * NB * 1024 + strips * NB * 256;
        if (p.NG * p.group_bytes <= room) break;
        if (p.SW == 1) {
            p.NG = room / p.group_bytes;
            break;
        }
    }
    p.smem = p.NG * p.group_bytes;
    return p;
}

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
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t phase, volatile int* abort_flag, uint32_t* status,
                                       uint64_t limit_ns, uint32_t site)
{
    return *abort_flag == 0 && mbar_wait(bar, phase, abort_flag, status, limit_ns, site, false);
}

// Two values less `minus` (fp16) times their fp16 roundings h, rounded to fp16.
__device__ __forceinline__ uint32_t remainders(uint32_t h, unsigned short minus, float x, float y)
{
    float a, b;
    asm("{\n"
        " .reg .b16 lo, hi;\n"
        " mov.b32 {lo, hi}, %2;\n"
        " fma.rn.f32.f16 %0, lo, %3, %4;\n"
        " fma.rn.f32.f16 %1, hi, %3, %5;\n"
        "}\n"
        : "=f"(a), "=f"(b)
        : "r"(h), "h"(minus), "f"(x), "f"(y));
    return pack2<false>(a, b);
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
__device__ __forceinline__ int cost_of(const Kv4Geo& gm, int len) { return len > 0 ? strips_of(len) + gm.unit_cost : 0; }

__device__ __forceinline__ long long div_up(long long x, int d)
{
    return x < 0x7fffffff ? (static_cast<unsigned>(x) + d - 1) / static_cast<unsigned>(d) : (x + d - 1) / d;
}

// A run of strips [s0, s1) of one unit within a group's range [.., end) of the line; `unit` is the line place where
// the unit begins, its first strip lies gm.unit_cost behind.
struct Piece {
    int b, hk, rb, len;
    int s0, s1;
    long long unit, end;
};

__device__ __forceinline__ void piece_end(const Kv4Geo& gm, Piece& p)
{
    const int n = strips_of(p.len);
    const long long left = p.end - p.unit - gm.unit_cost;
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
    const int cost = cost_of(gm, p.len), u = static_cast<int>(div_up(at - b_at + 1, cost)) - 1;
    p.unit = b_at + static_cast<long long>(u) * cost;
    p.hk = u / gm.rblocks;
    p.rb = u - p.hk * gm.rblocks;
    const int r = static_cast<int>(at - p.unit);
    p.s0 = r > gm.unit_cost ? r - gm.unit_cost : 0;
    piece_end(gm, p);
    return p.s1 > p.s0;
}

__device__ __forceinline__ bool next_piece(const Kv4Decode& a, const Kv4Geo& gm, Piece& p)
{
    p.unit += cost_of(gm, p.len);
    if (p.unit + gm.unit_cost >= p.end) return false;
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
    piece_end(gm, p);
    return p.s1 > 0;
}

// What the warp that loads a group's K (or V) keeps: its piece, and the first strip of the next step with its place in
// the block table (the pages of the step are in the lanes' registers, fetched a step early).
struct Loader {
    Piece piece;
    const uint8_t* head;  // the head's tiles in page 0
    const int* row;
    int s, in;
    int loads;            // steps loaded
    bool more;
};

struct __align__(16) DecShared {
    uint64_t full[kMaxWarps][2];      // per group: K and V of a step are there
    Piece first[kMaxWarps];           // per group: what its range begins with
    bool any[kMaxWarps];              // and whether it holds strips
    Loader load[kMaxWarps][2];
    int abort_flag;
    int up[kMaxWarps][2];             // per group and step parity: the last step in which a score passed the reference
    int last[kMaxWarps][3];           // sequence (-1: none), kv head and row block of the part a group ends with
    float ml[kMaxWarps][16][2];       // its references and sums
    float col[kMaxWarps][16];         // per warp and row: largest query magnitude or score
    float sum[kMaxWarps][16];         // per warp and row: sum of its P
};

// A operands of a K tile: four matrix steps of 16 tokens x 16 head dims.
__device__ __forceinline__ void k_tile(const uint8_t* tile, int lane, uint32_t (&a)[4][4])
{
    const uint4 w = *reinterpret_cast<const uint4*>(tile + lane * 16);
    const uint32_t sc = *reinterpret_cast<const uint16_t*>(tile + 512 + lane * 2);
    const uint32_t lo = scale_pair(sc, 0, 0), hi = scale_pair(sc, 1, 1);
    uint32_t x[4], y[4];
    kv4_dequant8(w.x, lo, x);
    kv4_dequant8(w.z, hi, y);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        a[k][0] = x[2 * k];
        a[k][1] = y[2 * k];
        a[k][2] = x[2 * k + 1];
        a[k][3] = y[2 * k + 1];
    }
    kv4_dequant8(w.y, lo, x);
    kv4_dequant8(w.w, hi, y);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        a[2 + k][0] = x[2 * k];
        a[2 + k][1] = y[2 * k];
        a[2 + k][2] = x[2 * k + 1];
        a[2 + k][3] = y[2 * k + 1];
    }
}

// A operands of a V tile: four blocks of 16 head dims x 16 tokens. keep: bytes of the four tokens' scales that count.
__device__ __forceinline__ void v_tile(const uint8_t* tile, int lane, uint32_t keep, uint32_t (&a)[4][4])
{
    const uint4 w = *reinterpret_cast<const uint4*>(tile + lane * 16);
    const uint32_t sc = *reinterpret_cast<const uint32_t*>(tile + 512 + ((lane >> 3) * 4 + (lane & 3)) * 4) & keep;
    const uint32_t lo = scale_pair(sc, 0, 1), hi = scale_pair(sc, 2, 3);
    uint32_t even, odd, x[4];
    interleave(w.x, w.y, even, odd);
    kv4_dequant8(even, lo, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e][0] = x[e];
    kv4_dequant8(odd, lo, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e][1] = x[e];
    interleave(w.z, w.w, even, odd);
    kv4_dequant8(even, hi, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e][2] = x[e];
    kv4_dequant8(odd, hi, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e][3] = x[e];
}

// N: head-dim chunks (D / 64); NB: blocks of eight query rows.
template <int N, int NB>
__global__ void __launch_bounds__(shape_of(N, NB).NG * shape_of(N, NB).C * 32, 1)
    decode_kv4_kernel(const Kv4Decode a, const Kv4Geo gm)
{
    constexpr Shape kShape = shape_of(N, NB);
    constexpr int CH = kShape.CH, C = kShape.C, NG = kShape.NG, SW = kShape.SW, D = 64 * N, kRows = 8 * NB;
    constexpr int steps = C * SW;                     // strips per step
    constexpr int strip_bytes = N * kKv4Tile;
    static_assert(sizeof(DecShared) + 1024 <= kStaticBytes, "static shared memory");
    const Problem& pb = a.f.pb;
    const bool bf16 = a.f.bf16 != 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int G = pb.Hq / pb.Hkv, R = G * pb.Nq;
    const int units_b = pb.Hkv * gm.rblocks;          // units per sequence
    // fp16 outputs, up to four rows: columns 4 .. 7 hold the rows again, with what P loses in fp16
    const bool again = NB == 1 && R <= 4 && !bf16;
    const unsigned short minus = again && t >= 2 ? 0xbc00 : 0;  // fp16 -1 or 0
    __shared__ DecShared sh;
    extern __shared__ __align__(128) uint8_t smem[];

    if (threadIdx.x < kMaxWarps * 2) {
        mbar_init(&sh.full[0][0] + threadIdx.x, 1);
        (&sh.up[0][0])[threadIdx.x] = 0;
        fence_barrier_init();
    }
    if (threadIdx.x < kMaxWarps) sh.last[threadIdx.x][0] = -1;
    if (threadIdx.x == 0) sh.abort_flag = 0;
    __syncthreads();
    pdl_wait();     // what the call reads and writes may belong to the kernel before it until here
    pdl_trigger();

    const int group = warp / C, wg = warp - group * C;  // my group, my place in it
    // my chunks are chunk0 .. chunk0 + CH - 1; those before wg * CH are another warp's too and are not stored
    const int chunk0 = min(wg * CH, N - CH);
    // shared memory of the group: K and V of a step [strips][chunks], Q operands [chunks][NB][2][32] of 16 bytes,
    // P operands [strips][NB][32] of 8 bytes
    uint8_t* const k_mem = smem + static_cast<size_t>(group) * kShape.group_bytes;
    uint8_t* const v_mem = k_mem + steps * strip_bytes;
    uint4* const q_mem = reinterpret_cast<uint4*>(v_mem + steps * strip_bytes) + lane;
    uint2* const p_mem = reinterpret_cast<uint2*>(q_mem - lane + N * NB * 64) + lane;
    uint64_t* const full = sh.full[group];

    auto group_sync = [&]() {
        if (C == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(C * 32) : "memory");
    };
    // ---- my group's range of the line: its first warp adds the line up, a lane a run of sequences
    if (wg == 0) {
        const int per = (pb.B + 31) >> 5, b0 = min(lane * per, pb.B), b1 = min(b0 + per, pb.B);
        long long sum = 0;
#pragma unroll 4
        for (int b = b0; b < b1; ++b) sum += cost_of(gm, cached_len(a, b));
        long long incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += x;
        }
        const long long total = __shfl_sync(0xffffffffu, incl, 31) * units_b, chunk = div_up(total, gm.workers);
        const long long lo = (incl - sum) * units_b, hi = incl * units_b;
        const long long at = (static_cast<long long>(blockIdx.x) * NG + group) * chunk;
        const unsigned in = __ballot_sync(0xffffffffu, at >= lo && at < hi);
        Piece p{};
        bool any = false;
        if (in != 0) {
            const int src = __ffs(in) - 1;
            long long b_at = __shfl_sync(0xffffffffu, lo, src);
            int b = src * per;
            for (;;) {  // one of that lane's sequences
                const long long n = static_cast<long long>(cost_of(gm, cached_len(a, b))) * units_b;
                if (at < b_at + n) break;
                b_at += n;
                ++b;
            }
            any = first_piece(a, gm, p, at, min(at + chunk, total), b, b_at);
        }
        if (lane == 0) {
            sh.first[group] = p;
            sh.any[group] = any;
        }
        __syncwarp();
    }
    group_sync();
    Piece cur = sh.first[group];
    bool more = sh.any[group];

    // Q of the piece's rows over every C-th chunk: a lane takes query g (of block k), head dims 16 t .. 16 t + 15 of a
    // chunk, zeros where there is no such row, to the places of its operands
    struct Queries {
        uint4 x[NB][CH], y[NB][CH];
    };
    auto fetch_q = [&](Queries& to) {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int r = cur.rb * kRows + k * 8 + (again ? g & 3 : g), hq = r / pb.Nq, h = cur.hk * G + hq, i = r - hq * pb.Nq;
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.f.q) + cur.b * pb.vq.sb +
                                                            h * pb.vq.sh + i * pb.vq.sn + wg * 64 + t * 16);
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const bool in = r < R && wg + j * C < N;
                to.x[k][j] = in ? q[j * C * 8] : make_uint4(0, 0, 0, 0);
                to.y[k][j] = in ? q[j * C * 8 + 1] : make_uint4(0, 0, 0, 0);
            }
        }
    };
    auto put_q = [&](const Queries& from) {
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
            for (int j = 0; j < CH; ++j)
                if (wg + j * C < N) {
                    uint4* const q = q_mem + ((wg + j * C) * NB + k) * 64;
                    q[0] = from.x[k][j];
                    q[32] = from.y[k][j];
                }
    };

    // ---- loads: K by the group's first warp, V by its second. Lane j copies the run of the step's strips that lies in
    // the j-th page, and has fetched that page's number a step early.
    constexpr int v_warp = C > 1 ? 1 : 0, kPlaces = C > 1 ? 1 : 2;  // a group of one warp loads both
    static_assert(steps <= 31, "a lane per page of a step");
    int page[kPlaces];
    // the step's strip that my page begins with, in a step that begins `in` strips into a page (below 2^32)
    auto my_run = [&](int in) { return lane ? lane * static_cast<unsigned>(gm.spp) - in : 0u; };
    auto fetch_pages = [&](const int* row, int in, unsigned n, int kv) {
        if (my_run(in) < n) page[kv < kPlaces ? kv : 0] = row[lane];
    };
    auto begin_piece = [&](Loader& ld, int kv) {
        const int s0 = ld.piece.s0, blk = s0 / gm.spp, in = s0 - blk * gm.spp;
        const int* row = a.cache.table + ld.piece.b * a.cache.table_stride + blk;
        fetch_pages(row, in, min(ld.piece.s1 - s0, steps), kv);
        if (lane == 0) {
            ld.s = s0;
            ld.in = in;
            ld.row = row;
            ld.head = a.cache.data + static_cast<size_t>(ld.piece.hk) * gm.spp * strip_bytes + (kv ? gm.v_off : 0);
        }
    };
    auto load = [&](int kv) {
        Loader& ld = sh.load[group][kv];
        if (!ld.more) return;
        const int s = ld.s, s1 = ld.piece.s1, in = ld.in, n = min(s1 - s, steps);
        const unsigned at = my_run(in);
        if (lane == 0) mbar_arrive_expect_tx(&full[kv], n * strip_bytes);
        __syncwarp();
        if (at < static_cast<unsigned>(n)) {
            int pg = page[kv < kPlaces ? kv : 0];
            if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.cache.num_pages)) {
                // the sequence's rows are undefined, but the copies stay inside the cache
                kv4_invalid(a.f.ctl.status, VS_KV4_DECODE, ld.piece.b);
                pg = 0;
            }
            const int skip = lane ? 0 : in;
            bulk_load((kv ? v_mem : k_mem) + at * strip_bytes,
                      ld.head + pg * (2 * gm.v_off) + static_cast<size_t>(skip) * strip_bytes,
                      min(n - static_cast<int>(at), gm.spp - skip) * strip_bytes, &full[kv]);
        }
        if (s + steps < s1) {
            const int wrap = in + gm.step_in >= gm.spp, next = in + gm.step_in - (wrap ? gm.spp : 0);
            const int* row = ld.row + gm.step_blk + wrap;
            fetch_pages(row, next, min(s1 - s - steps, steps), kv);
            __syncwarp();
            if (lane == 0) {
                ld.s = s + steps;
                ld.in = next;
                ld.row = row;
                ++ld.loads;
            }
        } else {
            __syncwarp();
            if (lane == 0) {
                ++ld.loads;
                ld.more = next_piece(a, gm, ld.piece);
            }
            __syncwarp();
            if (ld.more) begin_piece(ld, kv);
        }
    };
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
        if (wg == (kv ? v_warp : 0)) {
            Loader& ld = sh.load[group][kv];
            if (lane == 0) {
                ld.piece = cur;
                ld.more = more;
                ld.loads = 0;
            }
            __syncwarp();
            if (more) begin_piece(ld, kv);
            __syncwarp();
        }
    if (more) {
        Queries q;
        fetch_q(q);  // on its way while the loads wait for their pages
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
            if (wg == (kv ? v_warp : 0)) load(kv);
        put_q(q);
    }
    __syncwarp();
    // Waits for a copy. After one that ran out of time no more are issued, the group's barriers go on.
    auto arrived = [&](int kv, uint32_t phase) {
        if (!mbar_try_wait(smem_u32(&full[kv]), phase) &&
            !wait_slow(&full[kv], phase, &sh.abort_flag, a.f.ctl.status, a.f.ctl.limit_ns, kv ? KS_V : KS_K))
            sh.load[group][0].more = sh.load[group][1].more = false;
        __syncwarp();
    };

    bool pending = false;  // my group's last part is still in its registers
    float acc[CH][4][NB][4];
    float m[NB][2], l[NB][2];
    int step = 0;                       // steps begun by my group
    float s[SW][NB][4], c2[NB][2];
    int limits[NB][2], least = 0;       // first token that my columns' rows do not see, and that some row does not see

    // S^T of my strips
    auto scores = [&](int n) {
        float sum[SW == 1 ? 2 : 1][SW][NB][4];  // two chains where there is one strip
#pragma unroll
        for (int x = 0; x < (SW == 1 ? 2 : 1); ++x)
#pragma unroll
            for (int i = 0; i < SW; ++i)
#pragma unroll
                for (int k = 0; k < NB; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[x][i][k][e] = 0.f;
        arrived(0, (step - 1) & 1u);
        if (n > 0) {
            const uint8_t* tile = k_mem + wg * SW * strip_bytes;
            const uint4* q = q_mem;
            auto one = [&](float (&to)[SW][NB][4]) {
                uint4 q0[NB], q1[NB];
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    q0[k] = q[k * 64];
                    q1[k] = q[k * 64 + 32];
                }
#pragma unroll
                for (int i = 0; i < SW; ++i) {
                    uint32_t x[4][4];
                    k_tile(tile + i * strip_bytes, lane, x);
#pragma unroll
                    for (int k = 0; k < NB; ++k)
                        mma_f16_16816(to[i][k], x[0][0], x[0][1], x[0][2], x[0][3], q0[k].x, q0[k].y);
#pragma unroll
                    for (int k = 0; k < NB; ++k)
                        mma_f16_16816(to[i][k], x[1][0], x[1][1], x[1][2], x[1][3], q0[k].z, q0[k].w);
#pragma unroll
                    for (int k = 0; k < NB; ++k)
                        mma_f16_16816(to[i][k], x[2][0], x[2][1], x[2][2], x[2][3], q1[k].x, q1[k].y);
#pragma unroll
                    for (int k = 0; k < NB; ++k)
                        mma_f16_16816(to[i][k], x[3][0], x[3][1], x[3][2], x[3][3], q1[k].z, q1[k].w);
                }
                tile += kKv4Tile;
                q += NB * 64;
            };
#pragma unroll
            for (int c = 0; c < N; ++c) one(sum[SW == 1 ? c & 1 : 0]);
        }
#pragma unroll
        for (int i = 0; i < SW; ++i)
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[i][k][e] = SW == 1 ? sum[0][i][k][e] + sum[SW == 1 ? 1 : 0][i][k][e] : sum[0][i][k][e];
    };
    // P of my strips as operands to the step's buffer; their sums
    float dl[NB][2];
    auto store_p = [&]() {
        uint2* p = p_mem + wg * SW * NB * 32;
#pragma unroll
        for (int k = 0; k < NB; ++k) dl[k][0] = dl[k][1] = 0.f;
#pragma unroll
        for (int i = 0; i < SW; ++i)
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = ex2_approx(s[i][k][e]);
                dl[k][0] += x[0] + x[2];
                dl[k][1] += x[1] + x[3];
                // fp16 P: half a step of 2^-11, an eighth of the rounding of a bf16 output
                uint32_t h0 = pack2<false>(x[0], x[1]), h1 = pack2<false>(x[2], x[3]);
                if (again) {
                    h0 = remainders(h0, minus, x[0], x[1]);
                    h1 = remainders(h1, minus, x[2], x[3]);
                }
                p[(i * NB + k) * 32] = make_uint2(transpose8x8(h0), transpose8x8(h1));
            }
    };
    // O^T += V^T P^T over my chunks, for the n strips of a step, whose first token is tok
    auto values = [&](int n, int tok) {
        arrived(1, (step - 1) & 1u);
        const uint8_t* tile = v_mem + chunk0 * kKv4Tile;
        const uint2* p = p_mem;
        // cells behind the last token hold anything: their scales count as zero
        const int tail = cur.len - tok - 16 * (n - 1);
        uint32_t last_keep = 0xffffffffu;
        if (tail < 16) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (2 * t + (j & 1) + 8 * (j >> 1) >= tail) last_keep &= ~(0xffu << (8 * j));
        }
#pragma unroll 2
        for (int i = 0; i < n; ++i) {
            uint2 pf[NB];
#pragma unroll
            for (int k = 0; k < NB; ++k) pf[k] = p[k * 32];
            const uint32_t keep = i == n - 1 ? last_keep : 0xffffffffu;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                uint32_t x[4][4];
                v_tile(tile + c * kKv4Tile, lane, keep, x);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int k = 0; k < NB; ++k)
                        mma_f16_16816(acc[c][e][k], x[e][0], x[e][1], x[e][2], x[e][3], pf[k].x, pf[k].y);
            }
            tile += strip_bytes;
            p += NB * 32;
        }
    };
    // a part of the piece's rows to a slot of the workspace
    auto store_part = [&](size_t slot) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int r = n * 8 + 2 * t + q;
                if (cur.rb * kRows + r >= R) continue;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    if (chunk0 + c < wg * CH) continue;
                    float4* o = reinterpret_cast<float4*>(gm.part + (slot * kRows + r) * D + (chunk0 + c) * 64 + 8 * g);
                    o[0] = make_float4(acc[c][0][n][q], acc[c][0][n][q + 2], acc[c][1][n][q], acc[c][1][n][q + 2]);
                    o[1] = make_float4(acc[c][2][n][q], acc[c][2][n][q + 2], acc[c][3][n][q], acc[c][3][n][q + 2]);
                }
                if (wg == 0 && g == 0) {
                    gm.ml[(slot * kRows + r) * 2] = m[n][q];
                    gm.ml[(slot * kRows + r) * 2 + 1] = l[n][q];
                }
            }
    };

    while (more) {
        // ---- Q as B operands: fp16, scaled by a power of two into its range (bf16 has the wider one)
        const int r0 = cur.rb * kRows;
        least = pb.causal ? cur.len - pb.Nq + 1 : cur.len;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            uint4 x[CH], y[CH];
            uint32_t amax = 0;  // magnitudes of 16-bit floats order as their bits do
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const bool in = wg + j * C < N;
                x[j] = in ? q_mem[((wg + j * C) * NB + k) * 64] : make_uint4(0, 0, 0, 0);
                y[j] = in ? q_mem[((wg + j * C) * NB + k) * 64 + 32] : make_uint4(0, 0, 0, 0);
                const uint32_t w[8] = {x[j].x, x[j].y, x[j].z, x[j].w, y[j].x, y[j].y, y[j].z, y[j].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = max(amax, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
            }
            float mul = 1.f;
            if (bf16) {
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                if (C > 1) {
                    if (t == 0) sh.col[warp][k * 8 + g] = __uint_as_float(amax);
                    group_sync();
                    for (int w = 0; w < C; ++w) amax = max(amax, __float_as_uint(sh.col[group * C + w][k * 8 + g]));
                }
                // largest magnitude to [2^14, 2^15); rows of zeros or that are not finite stay as they are
                const int e = static_cast<int>(amax >> 7);
                if (amax > 0 && e < 255)
                    mul = __uint_as_float(static_cast<uint32_t>(min(14 + 127 - e, 126) + 127) << 23);
#pragma unroll
                for (int j = 0; j < CH; ++j) {
                    uint32_t w[8] = {x[j].x, x[j].y, x[j].z, x[j].w, y[j].x, y[j].y, y[j].z, y[j].w};
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        const float2 f = unpack2<true>(w[v]);
                        w[v] = pack2<false>(f.x * mul, f.y * mul);
                    }
                    x[j] = make_uint4(w[0], w[1], w[2], w[3]);
                    y[j] = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int c = wg + j * C;
                if (c < N) {
                    q_mem[(c * NB + k) * 64] = x[j];
                    q_mem[(c * NB + k) * 64 + 32] = y[j];
                }
            }
            const float scale = pb.scale_log2 / mul;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                c2[k][e] = __shfl_sync(0xffffffffu, scale, (2 * t + e) * 4);
                limits[k][e] = pb.causal ? min(cur.len, least + (r0 + k * 8 + (again ? (2 * t + e) & 3 : 2 * t + e)) % pb.Nq) : cur.len;
                m[k][e] = 0.f;
                l[k][e] = 0.f;
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
        group_sync();

        for (int at = cur.s0; at < cur.s1; at += steps) {
            const int mine = at + wg * SW, n = max(0, min(SW, cur.s1 - mine));  // my strips of the step
            const bool first = at == cur.s0;
            ++step;
            scores(n);
            // scores in log2 units above the reference; keys that a row does not see have none
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int i = 0; i < SW; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][k][e] = fmaf(s[i][k][e], c2[k][e & 1], -m[k][e & 1]);
            if (mine + SW > least >> 4 || n < SW) {  // in strips: tokens may reach 2^31
#pragma unroll
                for (int k = 0; k < NB; ++k)
#pragma unroll
                    for (int i = 0; i < SW; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (i >= n || (mine + i) * 16 + g + 8 * (e >> 1) >= limits[k][e & 1]) s[i][k][e] = -INFINITY;
            }
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int i = 0; i < SW; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, s[i][k][e]);
            if (!first) {
                const bool up = __any_sync(0xffffffffu, top > kRefSpan);
                if (up && lane == 0) sh.up[group][step & 1] = step;
                store_p();
            }
            group_sync();  // P is there, K is read
            if (wg == 0) load(0);
            if (first || *reinterpret_cast<volatile int*>(&sh.up[group][step & 1]) == step) {
                // the reference moves, for all warps of the group alike
#pragma unroll
                for (int k = 0; k < NB; ++k)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int i = 0; i < SW; ++i) mx = fmaxf(mx, fmaxf(s[i][k][q], s[i][k][q + 2]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        if (g == 0) sh.col[warp][k * 8 + 2 * t + q] = mx;
                    }
                group_sync();
#pragma unroll
                for (int k = 0; k < NB; ++k)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float mx = -INFINITY;
                        for (int w = 0; w < C; ++w) mx = fmaxf(mx, sh.col[group * C + w][k * 8 + 2 * t + q]);
                        // how far it moves; a row's keys come first, so one without any in the piece's first step has
                        // none in the piece
                        float up = mx - kRefBelow;
                        if (first ? mx == -INFINITY : up < 0.f) up = 0.f;
                        const float al = first ? 0.f : ex2_approx(-up);
                        m[k][q] += up;
                        l[k][q] *= al;
#pragma unroll
                        for (int i = 0; i < SW; ++i) {
                            s[i][k][q] -= up;
                            s[i][k][q + 2] -= up;
                        }
#pragma unroll
                        for (int c = 0; c < CH; ++c)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                acc[c][i][k][q] *= al;
                                acc[c][i][k][q + 2] *= al;
                            }
                    }
                store_p();
                group_sync();
            }
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int q = 0; q < 2; ++q) l[k][q] += dl[k][q];
            values(min(steps, cur.s1 - at), at * 16);
            group_sync();  // V and P are read
            if (wg == v_warp) load(1);
        }

        // ---- the group's sums
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                l[n][q] += __shfl_xor_sync(0xffffffffu, l[n][q], 4);
                l[n][q] += __shfl_xor_sync(0xffffffffu, l[n][q], 8);
                l[n][q] += __shfl_xor_sync(0xffffffffu, l[n][q], 16);
                if (g == 0) sh.sum[warp][n * 8 + 2 * t + q] = l[n][q];
            }
        group_sync();
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                l[n][q] = 0.f;
                for (int w = 0; w < C; ++w) l[n][q] += sh.sum[group * C + w][n * 8 + 2 * t + q];
                if (l[n][q] == 0.f) m[n][q] = -INFINITY;  // no keys, no reference
            }

        if (again) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[c][i][0][e] += __shfl_xor_sync(0xffffffffu, acc[c][i][0][e], 2);
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
                        for (int e = 0; e < 4; ++e) {
                            const float lo = acc[c][e][n][q] * inv, hi = acc[c][e][n][q + 2] * inv;
                            x[e] = bf16 ? pack2<true>(lo, hi) : pack2<false>(lo, hi);
                        }
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
                store_part(2 * (static_cast<size_t>(blockIdx.x) * NG + group));
                cur = next;
            } else {
                pending = true;
            }
        }
        if (more) {
            Queries q;
            fetch_q(q);
            put_q(q);
        }
    }
    // after a wait that ran out, copies may still be in flight: they end before the CTA does
    if (lane == 0 && *reinterpret_cast<volatile int*>(&sh.abort_flag))
        for (int kv = 0; kv < 2; ++kv)
            if (wg == (kv ? v_warp : 0) && sh.load[group][kv].loads > 0)
                mbar_wait(&full[kv], (sh.load[group][kv].loads - 1) & 1u, &sh.abort_flag, a.f.ctl.status, a.f.ctl.limit_ns,
                          KS_DRAIN, false);
    // ---- a part that the group ends with: to its own shared memory, [warp][row][head dims of the warp's chunks]
    constexpr int kPartPitch = 64 * CH + 4, kPartFloats = kRows * kPartPitch;
    static_assert(C * kPartFloats * 4 <= kShape.group_bytes, "a group's part");
    if (pending) {
        float* mine = reinterpret_cast<float*>(k_mem) + wg * kPartFloats;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int r = n * 8 + 2 * t + q;
                float4* o = reinterpret_cast<float4*>(mine + r * kPartPitch + 8 * g);
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    o[16 * c] = make_float4(acc[c][0][n][q], acc[c][0][n][q + 2], acc[c][1][n][q], acc[c][1][n][q + 2]);
                    o[16 * c + 1] = make_float4(acc[c][2][n][q], acc[c][2][n][q + 2], acc[c][3][n][q], acc[c][3][n][q + 2]);
                }
                if (wg == 0 && g == 0) {
                    sh.ml[group][r][0] = m[n][q];
                    sh.ml[group][r][1] = l[n][q];
                }
            }
        if (wg == 0 && lane == 0) {
            sh.last[group][0] = cur.b;
            sh.last[group][1] = cur.hk;
            sh.last[group][2] = cur.rb;
        }
    }
    __syncthreads();
    if (!pending) return;
    // neighbouring groups that end in the same unit join their parts, their threads taking the values in turn; the sum
    // goes to slot 1 of the last of them
    int run0 = group, run1 = group;
    auto same = [&](int i) { return sh.last[i][0] == cur.b && sh.last[i][1] == cur.hk && sh.last[i][2] == cur.rb; };
    while (run0 > 0 && same(run0 - 1)) --run0;
    while (run1 + 1 < NG && same(run1 + 1)) ++run1;
    const size_t slot = 2 * (static_cast<size_t>(blockIdx.x) * NG + run1) + 1;
    const int items = min(kRows, R - cur.rb * kRows) * (D / 4);
#pragma unroll 1
    for (int e = ((group - run0) * C + wg) * 32 + lane; e < items; e += (run1 - run0 + 1) * C * 32) {
        const int r = e / (D / 4), d = e % (D / 4) * 4, w = d / (64 * CH);
        const float* at =
            reinterpret_cast<const float*>(smem) + w * kPartFloats + r * kPartPitch + d - 64 * min(w * CH, N - CH);
        float mx = -INFINITY, sum = 0.f;
#pragma unroll 1
        for (int k = run0; k <= run1; ++k) mx = fmaxf(mx, sh.ml[k][r][0]);
        const float mu = mx == -INFINITY ? 0.f : mx;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k = run0; k <= run1; ++k) {
            const float f = ex2_approx(sh.ml[k][r][0] - mu);
            const float4 v = *reinterpret_cast<const float4*>(at + k * (kShape.group_bytes / 4));
            sum += sh.ml[k][r][1] * f;
            x.x = fmaf(v.x, f, x.x);
            x.y = fmaf(v.y, f, x.y);
            x.z = fmaf(v.z, f, x.z);
            x.w = fmaf(v.w, f, x.w);
        }
        *reinterpret_cast<float4*>(gm.part + (slot * kRows + r) * D + d) = x;
        if (d == 0) *reinterpret_cast<float2*>(gm.ml + (slot * kRows + r) * 2) = make_float2(mx, sum);
    }
}

// Joins the parts of units that several groups worked on; writes the rows of
// sequences without tokens. One CTA per query row and 128 head dims: its four
// warps take parts in turn, four head dims per lane.
constexpr int kJoinThreads = 128;

template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads) decode_kv4_join_kernel(const Kv4Decode a, const Kv4Geo gm)
{
    pdl_trigger();
    const Problem& pb = a.f.pb;
    __shared__ long long sums[2][kJoinThreads / 32];
    __shared__ float4 accs[kJoinThreads];
    __shared__ float2 mls[kJoinThreads / 32];
    const long long row = blockIdx.x;
    const int i = static_cast<int>(row % pb.Nq), h = static_cast<int>(row / pb.Nq % pb.Hq);
    const int b = static_cast<int>(row / (static_cast<long long>(pb.Nq) * pb.Hq));
    const int G = pb.Hq / pb.Hkv, r = (h % G) * pb.Nq + i, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int units_b = pb.Hkv * gm.rblocks;
    long long total = 0, before = 0;  // places of the line, and those before sequence b
    for (int k = threadIdx.x; k < pb.B; k += kJoinThreads) {
        const int c = cost_of(gm, cached_len(a, k));
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
    const int unit = (h / G) * gm.rblocks + r / gm.rows;
    const long long first = before * units_b + static_cast<long long>(unit) * cost_of(gm, len) + gm.unit_cost;
    const long long end = first + n, chunk = div_up(total, gm.workers);
    const int v0 = static_cast<int>(first / chunk), v1 = static_cast<int>((end - 1) / chunk);
    pdl_wait();
    if (v0 == v1) return;  // written by its group
    // v1 ends in this unit unless its range reaches strips of the next one; the parts that groups of a CTA end with
    // are in slot 1 of the last of them, a part that is followed by another unit is in slot 0
    const bool ends = min((v1 + 1LL) * chunk, total) <= end + gm.unit_cost;
    const int vl = ends ? v1 : v1 - 1, c0 = v0 / gm.NG, parts = vl / gm.NG - c0 + 1 + (ends ? 0 : 1), rr = r % gm.rows;
    const bool in = d < pb.D;
    // a warp's parts relative to their own largest reference; four in flight
    float m = -INFINITY, l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = warp; k0 < parts; k0 += 4 * (kJoinThreads / 32)) {
        float2 ml[4];
        float4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = k0 + e * (kJoinThreads / 32);
            ml[e] = make_float2(-INFINITY, 0.f);
            v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k >= parts) continue;
            const size_t slot = !ends && k == parts - 1 ? 2 * v1 : 2 * min(vl, (c0 + k) * gm.NG + gm.NG - 1) + 1;
            ml[e] = *reinterpret_cast<const float2*>(gm.ml + (slot * gm.rows + rr) * 2);
            if (in) v[e] = *reinterpret_cast<const float4*>(gm.part + (slot * gm.rows + rr) * pb.D + d);
        }
        const float mx = fmaxf(fmaxf(m, fmaxf(ml[0].x, ml[1].x)), fmaxf(ml[2].x, ml[3].x));
        const float mu = mx == -INFINITY ? 0.f : mx, f0 = ex2_approx(m - mu);
        l *= f0;
        x = make_float4(x.x * f0, x.y * f0, x.z * f0, x.w * f0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float f = ex2_approx(ml[e].x - mu);
            l = fmaf(ml[e].y, f, l);
            x.x = fmaf(v[e].x, f, x.x);
            x.y = fmaf(v[e].y, f, x.y);
            x.z = fmaf(v[e].z, f, x.z);
            x.w = fmaf(v[e].w, f, x.w);
        }
        m = mx;
    }
    accs[threadIdx.x] = x;
    if (lane == 0) mls[warp] = make_float2(m, l);
    __syncthreads();
    if (warp != 0) return;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) mx = fmaxf(mx, mls[w].x);
    const float mu = mx == -INFINITY ? 0.f : mx;
    x = make_float4(0.f, 0.f, 0.f, 0.f);
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) {
        const float f = ex2_approx(mls[w].x - mu);
        const float4 v = accs[w * 32 + lane];
        l = fmaf(mls[w].y, f, l);
        x.x = fmaf(v.x, f, x.x);
        x.y = fmaf(v.y, f, x.y);
        x.z = fmaf(v.z, f, x.z);
        x.w = fmaf(v.w, f, x.w);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (in)
        *reinterpret_cast<uint2*>(o) = make_uint2(pack2<BF16>(x.x * inv, x.y * inv), pack2<BF16>(x.z * inv, x.w * inv));
    if (blockIdx.y == 0 && lane == 0) a.f.lse[row] = l == 0.f ? -INFINITY : (mx + lg2_approx(l)) * kLn2;
}

struct Plan {
    Kv4Geo gm;
    int ctas, nb;
    size_t part_floats, bytes;
};

// Eight query rows per step up to G * Nq = 8, else blocks of sixteen.
Plan plan(const Problem& pb)
{
    Plan p{};
    Kv4Geo& gm = p.gm;
    const long long R = static_cast<long long>(pb.Hq / pb.Hkv) * pb.Nq;
    p.nb = R <= 8 ? 1 : 2;
    gm.rows = 8 * p.nb;
    gm.rblocks = static_cast<int>((R + gm.rows - 1) / gm.rows);
    gm.NG = shape_of(pb.D >> 6, p.nb).NG;
    // Its queries, its sums and its part or outputs. With eight rows 2 strips cost up to 5% (64 sequences of 20 to 1000
    // tokens) and 8 the same to 2%, none 50%; with sixteen 4 cost up to 10% (5000 tokens on one head), 12 up to 4%.
    gm.unit_cost = 4 * p.nb;
    const int sms = num_sms();
    p.ctas = sms > 0 ? sms : 152;
    gm.workers = p.ctas * gm.NG;
    p.part_floats = static_cast<size_t>(gm.workers) * 2 * gm.rows * pb.D;
    p.bytes = (p.part_floats + static_cast<size_t>(gm.workers) * 2 * gm.rows * 2) * sizeof(float);
    return p;
}

template <int N, int NB>
cudaError_t launch_shape(const Kv4Decode& a, const Plan& p, cudaStream_t s)
{
    constexpr Shape shape = shape_of(N, NB);
    auto* kernel = decode_kv4_kernel<N, NB>;
    // the attribute outlasts a call: once per device (those past 64 set it every time)
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, shape.smem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    return launch_dependent(kernel, dim3(p.ctas), shape.NG * shape.C * 32, shape.smem, s, a, p.gm);
}

template <int N>
cudaError_t launch_chunks(const Kv4Decode& a, const Plan& p, cudaStream_t s)
{
    if (a.f.pb.D >> 6 == N) return p.nb == 1 ? launch_shape<N, 1>(a, p, s) : launch_shape<N, 2>(a, p, s);
    if constexpr (N > 1) return launch_chunks<N - 1>(a, p, s);
    return cudaErrorInvalidValue;
}

}  // namespace

size_t kv4_decode_workspace_bytes(const Problem& pb) { return plan(pb).bytes; }

cudaError_t launch_decode_kv4(const Kv4Decode& a, void* workspace, cudaStream_t s)
{
    Plan p = plan(a.f.pb);
    const Shape shape = shape_of(a.f.pb.D >> 6, p.nb);
    p.gm.spp = a.cache.page_size >> 4;
    p.gm.step_blk = shape.C * shape.SW / p.gm.spp;
    p.gm.step_in = shape.C * shape.SW % p.gm.spp;
    p.gm.v_off = static_cast<size_t>(a.f.pb.Hkv) * p.gm.spp * (a.f.pb.D >> 6) * kKv4Tile;
    p.gm.part = static_cast<float*>(workspace);
    p.gm.ml = p.gm.part + p.part_floats;
    const cudaError_t ran = launch_chunks<16>(a, p, s);
    if (ran != cudaSuccess) return ran;
    const Problem& pb = a.f.pb;
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(pb.B) * pb.Hq * pb.Nq), (pb.D + 127) / 128);
    auto* join = a.f.bf16 ? decode_kv4_join_kernel<true> : decode_kv4_join_kernel<false>;
    return launch_dependent(join, grid, kJoinThreads, 0, s, a, p.gm);
}

}  // namespace ffpa
