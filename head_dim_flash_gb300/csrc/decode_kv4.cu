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
//     cache in shared memory. The operands of both products are fp16 for either
//     element type: cached values and (power-of-two scaled) queries are exact.
//   - a group of C warps owns a strip of tokens, each warp up to four 64-wide
//     head-dim chunks of it: partial scores are exchanged through shared memory
//     (none when C = 1), the softmax is computed by every warp, and O^T stays in
//     registers. NG groups per CTA work on different strips; one CTA per SM.
//   - strips arrive by bulk copies into a K ring and a V ring per group. The
//     group's one barrier per step (after the exchange) also frees the K stage of
//     the step and the V stage of the one before, so that every copy has a whole
//     step to arrive.
//   - the softmax keeps a reference instead of the running maximum: it moves (and
//     O is rescaled) only when a score passes it by 2^14, so that the usual step
//     is one vote. P <= 2^14 and its row's largest is >= 2^6 in fp16.
//   - the strips of all (sequence, kv head, row block) units form one line, cut
//     into equal ranges, one per CTA: lengths live on the device, so the cut is
//     made there. A unit that a range covers alone is finished by its CTA, the
//     parts of others go to the workspace (two at most per CTA) and a second
//     kernel joins them in a fixed order. It is launched as a dependent, so its
//     start overlaps the first kernel.
#include "kv4.cuh"

namespace ffpa {
namespace {

constexpr int kMaxWarps = 10;      // per CTA: up to 200 registers each
constexpr int kThreads = kMaxWarps * 32;
constexpr int kMaxStages = 4;
constexpr int kMaxGroups = kMaxWarps;
constexpr int kStepStrips = 2;     // strips of 16 tokens per step
constexpr float kRefBelow = 6.f;   // the reference lies this far (log2) below the maximum it was taken from
constexpr float kRefSpan = 14.f;   // and is kept until a score is this far above it
constexpr float kLn2 = 0.693147180559945309f;

enum Kv4Site : uint32_t { KS_K = 0x7b, KS_V, KS_DRAIN };

struct Kv4Geo {
    int chunks;      // D / 64
    int C;           // warps per group
    int NG;          // groups per CTA
    int rblocks;     // blocks of `rows` query rows per kv head's group of G * Nq
    int rows;        // 8 or 16
    int stages;
    int ctas;
    float* part;     // [ctas][2][rows][D] unnormalised partial O
    float* ml;       // [ctas][2][rows][2] reference (log2) and sum
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
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 matrix of 16-bit values held as an MMA fragment -> its transpose.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
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

__device__ __forceinline__ long long strips_of(int len) { return (static_cast<long long>(len) + 15) >> 4; }

// Strips of all sequences before b (b = B: of all), by every thread of the block; `red`: a sum per warp.
struct LineSums {
    long long before, total;
};
__device__ __forceinline__ LineSums line_sums(const Kv4Decode& a, int b_end, long long (*red)[kMaxWarps])
{
    long long before = 0, total = 0;
    for (int b = threadIdx.x; b < a.f.pb.B; b += blockDim.x) {
        const long long n = strips_of(cached_len(a, b));
        total += n;
        before += b < b_end ? n : 0;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, d);
        before += __shfl_xor_sync(0xffffffffu, before, d);
    }
    if ((threadIdx.x & 31) == 0) {
        red[0][threadIdx.x >> 5] = total;
        red[1][threadIdx.x >> 5] = before;
    }
    __syncthreads();
    LineSums s{0, 0};
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
        s.total += red[0][w];
        s.before += red[1][w];
    }
    __syncthreads();
    return s;
}

// First strip of CTA c's range of a line of `total` strips.
__device__ __forceinline__ long long range_begin(long long total, int c, int ctas) { return total * c / ctas; }

// A run of strips [s0, s1) of one unit within a CTA's range; w is its place on the line.
struct Piece {
    int b, hk, rb, len;
    int s0, s1;
    long long w;
};

struct __align__(16) DecShared {
    uint64_t full_k[kMaxGroups][kMaxStages], full_v[kMaxGroups][kMaxStages];
    long long red[2][kMaxWarps];
    long long first;   // strips of the sequences before the range's first one
    int first_b;
    int abort_flag;
    float c2[16];                      // log2-domain score scale of each row
    float ml[kMaxGroups][16][2];       // reference and sum of each group and row
};

template <int CH, int NB, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) decode_kv4_kernel(const Kv4Decode a, const Kv4Geo gm)
{
    pdl_trigger();
    const Problem& pb = a.f.pb;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int group = warp / gm.C, wg = warp % gm.C;  // my group, my place in it
    const int G = pb.Hq / pb.Hkv, R = G * pb.Nq;
    const int units_b = pb.Hkv * gm.rblocks;          // units per sequence
    __shared__ DecShared sh;
    extern __shared__ __align__(128) uint8_t smem[];

    // ---- my range of the line
    const LineSums all = line_sums(a, 0, sh.red);
    const long long total = all.total * units_b;
    const long long w0 = range_begin(total, blockIdx.x, gm.ctas), w1 = range_begin(total, blockIdx.x + 1, gm.ctas);
    if (w0 >= w1) return;
    {
        long long base = 0;
        for (int b0 = 0; b0 < pb.B; b0 += blockDim.x) {
            const int b = b0 + threadIdx.x;
            const long long n = b < pb.B ? strips_of(cached_len(a, b)) : 0;
            long long incl = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += x;
            }
            if (lane == 31) sh.red[0][warp] = incl;
            __syncthreads();
            long long chunk = 0;
            for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
                if (w < warp) incl += sh.red[0][w];
                chunk += sh.red[0][w];
            }
            if ((base + incl - n) * units_b <= w0 && w0 < (base + incl) * units_b) {
                sh.first = base + incl - n;
                sh.first_b = b;
            }
            base += chunk;
            __syncthreads();
            if (base * units_b > w0) break;
        }
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < gm.NG; ++i)
            for (int s = 0; s < gm.stages; ++s) {
                mbar_init(&sh.full_k[i][s], 1);
                mbar_init(&sh.full_v[i][s], 1);
            }
        sh.abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();

    auto piece_end = [&](Piece& p) {
        const long long n = strips_of(p.len), left = w1 - p.w;
        p.s1 = static_cast<int>(n - p.s0 < left ? n : p.s0 + left);
    };
    auto next_piece = [&](Piece& p) {
        p.w += p.s1 - p.s0;
        if (p.w >= w1) return false;
        p.s0 = 0;
        if (++p.rb == gm.rblocks) {
            p.rb = 0;
            if (++p.hk == pb.Hkv) {
                p.hk = 0;
                do {  // strips are left, so a later sequence has some
                    if (++p.b >= pb.B) return false;
                    p.len = cached_len(a, p.b);
                } while (p.len == 0);
            }
        }
        piece_end(p);
        return true;
    };
    // strips per step: one where a piece has no more strips than there are groups
    auto per_step = [&](const Piece& p) { return p.s1 - p.s0 <= gm.NG ? 1 : kStepStrips; };

    Piece cur;
    {
        const long long off = w0 - sh.first * units_b;
        cur.b = sh.first_b;
        cur.len = cached_len(a, cur.b);
        const long long n = strips_of(cur.len);
        const int u = static_cast<int>(off / n);
        cur.s0 = static_cast<int>(off - u * n);
        cur.hk = u / gm.rblocks;
        cur.rb = u % gm.rblocks;
        cur.w = w0;
        piece_end(cur);
    }

    // ---- shared memory: ring stages of every group, score exchange, then Q staging / the join
    const int st_bytes = stage_bytes(gm.chunks);
    const int strip_bytes = gm.chunks * kKv4Tile;
    uint8_t* const ring_k = smem + static_cast<size_t>(group) * 2 * gm.stages * st_bytes;
    uint8_t* const ring_v = ring_k + gm.stages * st_bytes;
    float4* const after = reinterpret_cast<float4*>(smem + static_cast<size_t>(gm.NG) * 2 * gm.stages * st_bytes);
    constexpr int kExch = kStepStrips * NB * 32;  // float4 per warp and buffer
    float4* const exch = after + group * 2 * gm.C * kExch;
    float4* const join = after + gm.NG * 2 * gm.C * kExch;
    uint16_t* const qs = reinterpret_cast<uint16_t*>(join);  // [rows][D + 8]
    uint64_t *const full_k = sh.full_k[group], *const full_v = sh.full_v[group];

    // ---- loads: the group's first warp walks the group's steps ahead of the products
    const int spp = a.cache.page_size >> 4;  // strips per page
    const size_t v_off = static_cast<size_t>(pb.Hkv) * spp * strip_bytes;
    Piece lp = cur;
    int l_step = group;
    int l_page0 = 0, l_page1 = 0;  // pages of the next step's strips, fetched one step ahead
    bool l_more = true;
    auto fetch = [&]() {
        for (;;) {
            const int per = per_step(lp);
            const int s = lp.s0 + l_step * per;
            if (s < lp.s1) {
                const int* row = a.cache.table + lp.b * a.cache.table_stride;
                l_page0 = row[s / spp];
                l_page1 = per > 1 && s + 1 < lp.s1 ? row[(s + 1) / spp] : l_page0;
                return;
            }
            if (!next_piece(lp)) {
                l_more = false;
                return;
            }
            l_step = group;
        }
    };
    // K tiles of a step's strips (V lies v_off behind); n = 0: no step
    struct Source {
        const uint8_t *s0, *s1;
        int n;
        bool joint;  // the two strips are neighbours in one page
    };
    auto next_source = [&]() {
        Source x{nullptr, nullptr, 0, false};
        if (!l_more) return x;
        const int per = per_step(lp), s = lp.s0 + l_step * per;
        x.n = min(per, lp.s1 - s);
        x.joint = x.n == 2 && s % spp + 1 < spp;
        if (static_cast<unsigned>(l_page0) >= static_cast<unsigned>(a.cache.num_pages) ||
            static_cast<unsigned>(l_page1) >= static_cast<unsigned>(a.cache.num_pages)) {
            // the sequence's rows are undefined, but the copies stay inside the cache
            if (lane == 0) kv4_invalid(a.f.ctl.status, VS_KV4_DECODE, lp.b);
            l_page0 = l_page1 = 0;
        }
        x.s0 = a.cache.data + kv4_strip_offset(a.cache, pb.Hkv, gm.chunks, l_page0, 0, lp.hk, s % spp);
        x.s1 = a.cache.data + kv4_strip_offset(a.cache, pb.Hkv, gm.chunks, l_page1, 0, lp.hk, (s + 1) % spp);
        l_step += gm.NG;
        fetch();
        return x;
    };
    auto load = [&](const Source& x, size_t off, uint8_t* dst, uint64_t* bar) {
        if (lane != 0 || x.n == 0) return;
        mbar_arrive_expect_tx(bar, x.n * strip_bytes);
        bulk_load(dst, x.s0 + off, (x.joint ? 2 : 1) * strip_bytes, bar);
        if (x.n == 2 && !x.joint) bulk_load(dst + strip_bytes, x.s1 + off, strip_bytes, bar);
    };
    int k_loads = 0, v_loads = 0;  // steps whose K / V copies were issued, or that do not exist
    Source last{nullptr, nullptr, 0, false};
    // K of the next step, into the stage that is free; its V follows a step later
    auto load_k = [&]() {
        last = next_source();
        const int slot = k_loads % gm.stages;
        load(last, 0, ring_k + slot * st_bytes, &full_k[slot]);
        k_loads += last.n > 0;
    };
    auto load_v = [&]() {
        const int slot = v_loads % gm.stages;
        load(last, v_off, ring_v + slot * st_bytes, &full_v[slot]);
        v_loads += last.n > 0;
    };
    if (wg == 0) {
        fetch();
        for (int i = 0; i < gm.stages; ++i) {
            load_k();
            if (i + 1 < gm.stages) load_v();
        }
    }

    // ---- state of the products
    const int my = (gm.chunks - wg + gm.C - 1) / gm.C;  // my chunks: wg, wg + C, ...
    int done = 0;    // steps of my group finished
    int eb = 0;      // exchange buffer
    bool ok = true;
    uint32_t qf[NB][CH][4][2];
    float acc[CH][4][NB][4];
    float m[NB][2], l[NB][2], c2[NB][2];
    float s[kStepStrips][NB][4];
    uint32_t pf[kStepStrips][NB][2];

    auto group_sync = [&]() {
        if (gm.C == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(gm.C * 32) : "memory");
    };

    // Waits for a copy. One that runs out of time ends the warp's work, not its barriers; another sequence's error
    // in the status word does not end it.
    auto arrived = [&](uint64_t* bar, int k, uint32_t site) {
        if (ok)
            ok = __all_sync(0xffffffffu, mbar_wait(bar, static_cast<uint32_t>((k / gm.stages) & 1), &sh.abort_flag,
                                                   a.f.ctl.status, a.f.ctl.limit_ns, site, false));
    };

    // S^T of a step over my chunks, left in s (C = 1) or in the exchange buffer
    auto scores = [&](int ns, int k) {
        const int slot = k % gm.stages;
        arrived(&full_k[slot], k, KS_K);
        const uint8_t* kb = ring_k + slot * st_bytes;
#pragma unroll
        for (int i = 0; i < kStepStrips; ++i) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
            if (i >= ns || !ok) continue;
#pragma unroll
            for (int cc = 0; cc < CH; ++cc) {
                if (cc >= my) break;
                const uint8_t* tile = kb + i * strip_bytes + (wg + cc * gm.C) * kKv4Tile;
                const uint4 w = *reinterpret_cast<const uint4*>(tile + lane * 16);
                const uint32_t sc = *reinterpret_cast<const uint16_t*>(tile + 512 + lane * 2);
                const uint32_t lo = kv4_scale2(sc), hi = kv4_scale2(sc >> 8);
                uint32_t x[4], y[4], z[4], u[4];
                kv4_dequant8(w.x, lo, x);
                kv4_dequant8(w.y, lo, y);
                kv4_dequant8(w.z, hi, z);
                kv4_dequant8(w.w, hi, u);
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    mma_f16_16816(s[i][n], x[0], z[0], x[1], z[1], qf[n][cc][0][0], qf[n][cc][0][1]);
                    mma_f16_16816(s[i][n], x[2], z[2], x[3], z[3], qf[n][cc][1][0], qf[n][cc][1][1]);
                    mma_f16_16816(s[i][n], y[0], u[0], y[1], u[1], qf[n][cc][2][0], qf[n][cc][2][1]);
                    mma_f16_16816(s[i][n], y[2], u[2], y[3], u[3], qf[n][cc][3][0], qf[n][cc][3][1]);
                }
            }
        }
        if (gm.C > 1) {
#pragma unroll
            for (int i = 0; i < kStepStrips; ++i)
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    exch[(eb * gm.C + wg) * kExch + (i * NB + n) * 32 + lane] =
                        make_float4(s[i][n][0], s[i][n][1], s[i][n][2], s[i][n][3]);
        }
    };

    // sums of the partial scores, mask, P^T fragments; tok: the step's first token
    auto softmax = [&](int ns, int tok, int len) {
        if (gm.C > 1) {
#pragma unroll
            for (int i = 0; i < kStepStrips; ++i)
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    float4 v = exch[eb * gm.C * kExch + (i * NB + n) * 32 + lane];
                    for (int w = 1; w < gm.C; ++w) {  // one order for every warp: all get the same bits
                        const float4 x = exch[(eb * gm.C + w) * kExch + (i * NB + n) * 32 + lane];
                        v.x += x.x;
                        v.y += x.y;
                        v.z += x.z;
                        v.w += x.w;
                    }
                    s[i][n][0] = v.x;
                    s[i][n][1] = v.y;
                    s[i][n][2] = v.z;
                    s[i][n][3] = v.w;
                }
            eb ^= 1;
        }
        const int least = pb.causal ? len - pb.Nq + 1 : len;  // first token that some row does not see
        const bool mask = tok + 16 * ns > least || ns < kStepStrips;
        bool up = false;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                int lim = len;
                if (mask && pb.causal) lim = min(len, least + (cur.rb * gm.rows + n * 8 + 2 * t + (e & 1)) % pb.Nq);
#pragma unroll
                for (int i = 0; i < kStepStrips; ++i) {
                    float x = s[i][n][e] * c2[n][e & 1];
                    if (mask) x = i < ns && tok + 16 * i + g + 8 * (e >> 1) < lim ? x : -INFINITY;
                    s[i][n][e] = x;
                    up |= x > m[n][e & 1] + kRefSpan;
                }
            }
        if (__any_sync(0xffffffffu, up)) {
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
                    const float mn = fmaxf(m[n][q], mx - kRefBelow);
                    const float al = m[n][q] == -INFINITY ? 0.f : ex2_approx(m[n][q] - mn);
                    m[n][q] = mn;
                    l[n][q] *= al;
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
        for (int n = 0; n < NB; ++n) {
            float mu[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) mu[q] = m[n][q] == -INFINITY ? 0.f : m[n][q];
#pragma unroll
            for (int i = 0; i < kStepStrips; ++i) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = ex2_approx(s[i][n][e] - mu[e & 1]);
                l[n][0] += p[0] + p[2];
                l[n][1] += p[1] + p[3];
                // fp16 P: half a step of 2^-11, an eighth of what bf16 operands would cost
                pf[i][n][0] = transpose8x8(pack2<false>(p[0], p[1]));
                pf[i][n][1] = transpose8x8(pack2<false>(p[2], p[3]));
            }
        }
    };

    // O^T += V^T P^T over my chunks
    auto values = [&](int ns, int tok, int len, int k) {
        const int slot = k % gm.stages;
        arrived(&full_v[slot], k, KS_V);
        if (!ok) return;
        const uint8_t* vb = ring_v + slot * st_bytes;
#pragma unroll
        for (int i = 0; i < kStepStrips; ++i) {
            if (i >= ns) break;
            uint32_t keep = 0xffffffffu;  // cells behind the last token hold anything: their scales count as zero
            if (tok + 16 * i + 16 > len) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (tok + 16 * i + 2 * t + (j & 1) + 8 * (j >> 1) >= len) keep &= ~(0xffu << (8 * j));
            }
#pragma unroll
            for (int cc = 0; cc < CH; ++cc) {
                if (cc >= my) break;
                const uint8_t* tile = vb + i * strip_bytes + (wg + cc * gm.C) * kKv4Tile;
                const uint4 w = *reinterpret_cast<const uint4*>(tile + lane * 16);
                const uint32_t sc = *reinterpret_cast<const uint32_t*>(tile + 512 + ((g >> 1) * 4 + t) * 4) & keep;
                uint32_t x[4], y[4], z[4], u[4];
                kv4_dequant8(w.x, kv4_scale2(sc), x);
                kv4_dequant8(w.y, kv4_scale2(sc >> 8), y);
                kv4_dequant8(w.z, kv4_scale2(sc >> 16), z);
                kv4_dequant8(w.w, kv4_scale2(sc >> 24), u);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t a0 = __byte_perm(x[e], y[e], 0x5410), a1 = __byte_perm(x[e], y[e], 0x7632);
                    const uint32_t a2 = __byte_perm(z[e], u[e], 0x5410), a3 = __byte_perm(z[e], u[e], 0x7632);
#pragma unroll
                    for (int n = 0; n < NB; ++n) mma_f16_16816(acc[cc][e][n], a0, a1, a2, a3, pf[i][n][0], pf[i][n][1]);
                }
            }
        }
    };

    for (bool more = true; more;) {
        // ---- Q of the piece's rows: fp16, scaled by a power of two into its range (bf16 has the wider one)
        const int r0 = cur.rb * gm.rows;
        for (int r = warp; r < gm.rows; r += blockDim.x >> 5) {
            uint4 v[4];
            float amax = 0.f;
            const bool row = r0 + r < R;
            const int h = cur.hk * G + (r0 + r) / pb.Nq, i = (r0 + r) % pb.Nq;
            const uint16_t* q = static_cast<const uint16_t*>(a.f.q) + cur.b * pb.vq.sb + h * pb.vq.sh + i * pb.vq.sn;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = make_uint4(0, 0, 0, 0);
                const int d = e * 256 + lane * 8;
                if (row && d < pb.D) v[e] = *reinterpret_cast<const uint4*>(q + d);
            }
            float mul = 1.f;
            if (BF16) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = unpack2<true>(w[j]);
                        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
#pragma unroll
                for (int d = 16; d; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
                // largest magnitude to [2^14, 2^15); rows of zeros or with infinities stay as they are
                const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
                if (amax > 0.f && e < 128) mul = __uint_as_float(static_cast<uint32_t>(min(14 - e, 126) + 127) << 23);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = e * 256 + lane * 8;
                if (d >= pb.D) break;
                if (BF16) {
                    uint32_t w[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = unpack2<true>(w[j]);
                        w[j] = pack2<false>(f.x * mul, f.y * mul);
                    }
                    v[e] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                *reinterpret_cast<uint4*>(qs + r * (pb.D + 8) + d) = v[e];
            }
            if (lane == 0) sh.c2[r] = pb.scale_log2 / mul;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int cc = 0; cc < CH; ++cc) {
                if (cc >= my) break;
                const uint4* src = reinterpret_cast<const uint4*>(qs + (n * 8 + g) * (pb.D + 8) +
                                                                  (wg + cc * gm.C) * 64 + t * 16);
                const uint4 x = src[0], y = src[1];
                qf[n][cc][0][0] = x.x;
                qf[n][cc][0][1] = x.y;
                qf[n][cc][1][0] = x.z;
                qf[n][cc][1][1] = x.w;
                qf[n][cc][2][0] = y.x;
                qf[n][cc][2][1] = y.y;
                qf[n][cc][3][0] = y.z;
                qf[n][cc][3][1] = y.w;
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                c2[n][q] = sh.c2[n * 8 + 2 * t + q];
                m[n][q] = -INFINITY;
                l[n][q] = 0.f;
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

        // ---- my group's steps of the piece; the scores of a step are issued before the values of the last one
        const int per = per_step(cur), steps = (cur.s1 - cur.s0 + per - 1) / per;
        const int mine = group < steps ? (steps - group + gm.NG - 1) / gm.NG : 0;
        auto first_strip = [&](int j) { return cur.s0 + (group + j * gm.NG) * per; };
        if (mine > 0) scores(min(per, cur.s1 - first_strip(0)), done);
        for (int j = 0; j < mine; ++j) {
            group_sync();  // the exchange is written; K of this step and V of the one before are read by all
            if (wg == 0 && ok) {
                load_v();
                load_k();
            }
            const int s0 = first_strip(j), ns = min(per, cur.s1 - s0);
            softmax(ns, s0 * 16, cur.len);
            if (j + 1 < mine) scores(min(per, cur.s1 - first_strip(j + 1)), done + 1);
            values(ns, s0 * 16, cur.len, done);
            ++done;
        }

        // ---- join the groups: their references and sums, then O in turn (a fixed order)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                l[n][q] += __shfl_xor_sync(0xffffffffu, l[n][q], 4);
                l[n][q] += __shfl_xor_sync(0xffffffffu, l[n][q], 8);
                l[n][q] += __shfl_xor_sync(0xffffffffu, l[n][q], 16);
                if (wg == 0 && lane < 4) {
                    sh.ml[group][n * 8 + 2 * t + q][0] = m[n][q];
                    sh.ml[group][n * 8 + 2 * t + q][1] = l[n][q];
                }
            }
        __syncthreads();
        const int active = min(steps, gm.NG);
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int r = n * 8 + 2 * t + q;
                float mx = -INFINITY, sum = 0.f;
                for (int i = 0; i < active; ++i) mx = fmaxf(mx, sh.ml[i][r][0]);
                const float mu = mx == -INFINITY ? 0.f : mx;
                for (int i = 0; i < active; ++i) sum += sh.ml[i][r][1] * ex2_approx(sh.ml[i][r][0] - mu);
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
        for (int turn = 0; turn < active; ++turn) {
            if (turn == group) {
                float4* buf = join + wg * (CH * 4 * NB * 32) + lane;
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            float(&x)[4] = acc[c][i][n];
                            float4* at = buf + ((c * 4 + i) * NB + n) * 32;
                            if (turn > 0) {
                                const float4 v = *at;
                                x[0] += v.x;
                                x[1] += v.y;
                                x[2] += v.z;
                                x[3] += v.w;
                            }
                            if (turn + 1 < active) *at = make_float4(x[0], x[1], x[2], x[3]);
                        }
            }
            __syncthreads();
        }
        if (group == active - 1) {
            const bool whole = cur.s0 == 0 && cur.s1 == strips_of(cur.len);
            const int slot = 2 * blockIdx.x + (cur.s0 > 0 ? 0 : 1);  // a unit that an earlier CTA began, or not
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int r = n * 8 + 2 * t + q;
                    if (r0 + r >= R) continue;
                    const int h = cur.hk * G + (r0 + r) / pb.Nq, i = (r0 + r) % pb.Nq;
                    const float inv = l[n][q] == 0.f ? 0.f : 1.f / l[n][q];
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        if (c >= my) break;
                        const int d = (wg + c * gm.C) * 64 + 8 * g;
                        float x[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[2 * e] = acc[c][e][n][q];
                            x[2 * e + 1] = acc[c][e][n][q + 2];
                        }
                        if (whole) {
                            uint16_t* o = static_cast<uint16_t*>(a.f.o) + cur.b * pb.vo.sb + h * pb.vo.sh + i * pb.vo.sn;
                            *reinterpret_cast<uint4*>(o + d) =
                                make_uint4(pack2<BF16>(x[0] * inv, x[1] * inv), pack2<BF16>(x[2] * inv, x[3] * inv),
                                           pack2<BF16>(x[4] * inv, x[5] * inv), pack2<BF16>(x[6] * inv, x[7] * inv));
                        } else {
                            float4* o = reinterpret_cast<float4*>(gm.part + (static_cast<size_t>(slot) * gm.rows + r) * pb.D + d);
                            o[0] = make_float4(x[0], x[1], x[2], x[3]);
                            o[1] = make_float4(x[4], x[5], x[6], x[7]);
                        }
                    }
                    if (wg == 0 && g == 0) {
                        if (whole) {
                            a.f.lse[(static_cast<long long>(cur.b) * pb.Hq + h) * pb.Nq + i] =
                                l[n][q] == 0.f ? -INFINITY : (m[n][q] + lg2_approx(l[n][q])) * kLn2;
                        } else {
                            float* ml = gm.ml + (static_cast<size_t>(slot) * gm.rows + r) * 2;
                            ml[0] = m[n][q];
                            ml[1] = l[n][q];
                        }
                    }
                }
        }
        more = next_piece(cur);
    }
    // after a wait that ran out, copies may still be in flight: they end before the CTA does
    if (wg == 0 && lane == 0 && !ok) {
        auto drain = [&](uint64_t* full, int loads) {
            for (int k = max(0, loads - gm.stages); k < loads; ++k)
                mbar_wait(&full[k % gm.stages], static_cast<uint32_t>((k / gm.stages) & 1), &sh.abort_flag,
                          a.f.ctl.status, a.f.ctl.limit_ns, KS_DRAIN, false);
        };
        drain(full_k, k_loads);
        drain(full_v, v_loads);
    }
}

// Joins the parts of units that several CTAs worked on; writes the rows of
// sequences without tokens. One CTA per query row and 128 head dims: its four
// warps take parts in turn, four head dims per lane.
constexpr int kJoinThreads = 128;

template <bool BF16>
__global__ void __launch_bounds__(kJoinThreads) decode_kv4_join_kernel(const Kv4Decode a, const Kv4Geo gm)
{
    const Problem& pb = a.f.pb;
    __shared__ long long red[2][kMaxWarps];
    __shared__ float4 sum[kJoinThreads];
    extern __shared__ float weight[];  // [ctas]
    const long long row = blockIdx.x;
    const int i = static_cast<int>(row % pb.Nq), h = static_cast<int>(row / pb.Nq % pb.Hq);
    const int b = static_cast<int>(row / (static_cast<long long>(pb.Nq) * pb.Hq));
    const int G = pb.Hq / pb.Hkv, r = (h % G) * pb.Nq + i, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int units_b = pb.Hkv * gm.rblocks;
    const LineSums line = line_sums(a, b, red);
    const long long total = line.total * units_b, n = strips_of(cached_len(a, b));
    const long long u0 = line.before * units_b + ((h / G) * gm.rblocks + r / gm.rows) * n;
    const int d = blockIdx.y * 128 + lane * 4;
    uint16_t* o = static_cast<uint16_t*>(a.f.o) + b * pb.vo.sb + h * pb.vo.sh + i * pb.vo.sn + d;
    pdl_wait();
    if (n == 0) {
        if (warp == 0 && d < pb.D) *reinterpret_cast<uint2*>(o) = make_uint2(0, 0);
        if (blockIdx.y == 0 && threadIdx.x == 0) a.f.lse[row] = -INFINITY;
        return;
    }
    auto cta_of = [&](long long w) {  // the CTA whose range holds strip w
        int c = static_cast<int>(static_cast<double>(w) * gm.ctas / static_cast<double>(total));
        c = max(0, min(c, gm.ctas - 1));
        while (range_begin(total, c, gm.ctas) > w) --c;
        while (range_begin(total, c + 1, gm.ctas) <= w) ++c;
        return c;
    };
    const int c0 = cta_of(u0), c1 = cta_of(u0 + n - 1);
    if (c0 == c1) return;
    // slot of the unit's part in CTA c: 0 when the unit began before the CTA's range
    auto slot = [&](int c) { return 2 * c + (range_begin(total, c, gm.ctas) > u0 ? 0 : 1); };
    auto has = [&](int c) { return range_begin(total, c, gm.ctas) < range_begin(total, c + 1, gm.ctas); };
    float mx = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32)
        if (has(c)) mx = fmaxf(mx, gm.ml[(static_cast<size_t>(slot(c)) * gm.rows + r % gm.rows) * 2]);
#pragma unroll
    for (int e = 16; e; e >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, e));
    const float mu = mx == -INFINITY ? 0.f : mx;
    float l = 0.f;
    for (int c = c0 + lane; c <= c1; c += 32) {
        float w = 0.f;
        if (has(c)) {
            const float* ml = gm.ml + (static_cast<size_t>(slot(c)) * gm.rows + r % gm.rows) * 2;
            w = ex2_approx(ml[0] - mu);
            l += w * ml[1];
        }
        if (warp == 0) weight[c - c0] = w;
    }
#pragma unroll
    for (int e = 16; e; e >>= 1) l += __shfl_xor_sync(0xffffffffu, l, e);
    __syncthreads();
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (d < pb.D) {
#pragma unroll 4
        for (int c = c0 + warp; c <= c1; c += 4) {
            if (!has(c)) continue;
            const float w = weight[c - c0];
            const float4 v =
                *reinterpret_cast<const float4*>(gm.part + (static_cast<size_t>(slot(c)) * gm.rows + r % gm.rows) * pb.D + d);
            x.x = fmaf(w, v.x, x.x);
            x.y = fmaf(w, v.y, x.y);
            x.z = fmaf(w, v.z, x.z);
            x.w = fmaf(w, v.w, x.w);
        }
    }
    sum[threadIdx.x] = x;
    __syncthreads();
    if (warp == 0 && d < pb.D) {
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            const float4 v = sum[w * 32 + lane];
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
    gm.NG = kMaxGroups / gm.C;
    const int exch = gm.NG * 2 * gm.C * kStepStrips * p.nb * 32 * 16;
    const int join = gm.C * p.ch * 4 * p.nb * 32 * 16, q = gm.rows * (pb.D + 8) * 2;
    const int fixed = exch + (join > q ? join : q), ring = gm.NG * 2 * stage_bytes(gm.chunks);
    // at least two stages for every head dim: 184 KB of ring, 20 of exchange, 16 of join at D = 512
    gm.stages = (kMaxSmem - 1024 - static_cast<int>(sizeof(DecShared)) - fixed) / ring;
    if (gm.stages > kMaxStages) gm.stages = kMaxStages;
    p.smem = fixed + gm.stages * ring;
    const int sms = num_sms();
    gm.ctas = sms > 0 ? sms : 152;
    p.part_floats = static_cast<size_t>(gm.ctas) * 2 * gm.rows * pb.D;
    p.bytes = (p.part_floats + static_cast<size_t>(gm.ctas) * 2 * gm.rows * 2) * sizeof(float);
    return p;
}

template <int CH, int NB>
cudaError_t launch_variant(const Kv4Decode& a, const Plan& p, cudaStream_t s)
{
    auto* kernel = a.f.bf16 ? decode_kv4_kernel<CH, NB, true> : decode_kv4_kernel<CH, NB, false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, p.smem);
    if (e != cudaSuccess) return e;
    kernel<<<p.gm.ctas, p.gm.NG * p.gm.C * 32, p.smem, s>>>(a, p.gm);
    return cudaGetLastError();
}

}  // namespace

size_t kv4_decode_workspace_bytes(const Problem& pb) { return plan(pb).bytes; }

cudaError_t launch_decode_kv4(const Kv4Decode& a, void* workspace, cudaStream_t s)
{
    Plan p = plan(a.f.pb);
    p.gm.part = static_cast<float*>(workspace);
    p.gm.ml = p.gm.part + p.part_floats;
    cudaError_t e;
    if (p.nb == 1)
        e = p.ch == 1   ? launch_variant<1, 1>(a, p, s)
            : p.ch == 2 ? launch_variant<2, 1>(a, p, s)
            : p.ch == 3 ? launch_variant<3, 1>(a, p, s)
                        : launch_variant<4, 1>(a, p, s);
    else
        e = p.ch == 1 ? launch_variant<1, 2>(a, p, s) : launch_variant<2, 2>(a, p, s);
    if (e != cudaSuccess) return e;
    const Problem& pb = a.f.pb;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(pb.B) * pb.Hq * pb.Nq), (pb.D + 127) / 128);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = p.gm.ctas * sizeof(float);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, a.f.bf16 ? decode_kv4_join_kernel<true> : decode_kv4_join_kernel<false>, a, p.gm);
}

}  // namespace ffpa
