// Rotary positions on queries and keys, and their inverse (the gradient).
//
// Pair p of a head's first `rot` dims is a point of the plane that is turned
// by position * theta_p: (x, y) -> m (x cos - y sin, x sin + y cos). A turn is
// all that matters, so theta_p is kept as turns per position in 64-bit
// fixed point (units of 2^-64): position * turns, wrapped, is the angle's
// fraction of a turn within 2^-33 for every 32-bit position, where an fp32
// product at position 10^6 is off by a thirtieth of a radian. Its upper 32 bits
// become an fp32 (within 2^-26 turns); sin, cos and the products are fp32, too;
// one rounding at the end.
//
// One pass, bound by memory: each value is read and written once. A CTA takes
// a few tokens and the heads of both tensors; their cos and sin are computed
// once into shared memory, while the first values are on their way, and serve
// every head. A thread owns 16 head dims of a row, two 16-byte accesses: 8
// pairs, or a piece of the head dims behind `rot`, which are copied.
//
// Measured on a GB300 against a copy of the same tensors (us): 8192 tokens of 40
// heads of D = 512 108 against 100, 16000 of 20 of D = 320 with interleaved pairs on 128
// dims 64 against 63, 32768 of 40 of D = 128 100 against 100; 32 tokens 2.8, a
// launch. Four CTAs per SM instead of three (64 registers, streaming loads and
// stores): no difference.
#include "cache_ops.h"
#include "kv4.cuh"

namespace ffpa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopePairs = 2048;  // cos and sin that a CTA's table holds
constexpr int kRopeTokens = 64;   // tokens of a CTA, at most
constexpr int kRopeBatch = 4;     // rows that a thread has in flight

struct RopeToken {
    long long q, oq, k, ok;  // element offsets of the token's head 0
    long long pos;
    int there;
};

template <bool BF16, bool INTERLEAVED>
__device__ __forceinline__ void turn16(uint4& a, uint4& b, const float4* cs, int nu)
{
    // cs[j * nu]: cos, sin of pairs 2 j and 2 j + 1
    uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 t = cs[j * nu];
        if constexpr (INTERLEAVED) {
            const float2 p = unpack2<BF16>(x[2 * j]), r = unpack2<BF16>(x[2 * j + 1]);
            x[2 * j] = pack2<BF16>(p.x * t.x - p.y * t.y, p.x * t.y + p.y * t.x);
            x[2 * j + 1] = pack2<BF16>(r.x * t.z - r.y * t.w, r.x * t.w + r.y * t.z);
        } else {
            const float2 p = unpack2<BF16>(x[j]), r = unpack2<BF16>(x[4 + j]);
            x[j] = pack2<BF16>(p.x * t.x - r.x * t.y, p.y * t.z - r.y * t.w);
            x[4 + j] = pack2<BF16>(p.x * t.y + r.x * t.x, p.y * t.w + r.y * t.z);
        }
    }
    a = make_uint4(x[0], x[1], x[2], x[3]);
    b = make_uint4(x[4], x[5], x[6], x[7]);
}

template <bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a)
{
    pdl_wait();
    pdl_trigger();
    __shared__ __align__(16) float2 table[kRopePairs];  // [token][pair % 8 / 2][unit][pair % 2], read by two
    __shared__ RopeToken tok[kRopeTokens];
    const int tid = threadIdx.x;
    const long long T = a.cu ? a.total : static_cast<long long>(a.B) * a.N;
    const long long t0 = static_cast<long long>(blockIdx.x) * a.per_cta;
    const int nt = static_cast<int>(T - t0 < a.per_cta ? T - t0 : a.per_cta);
    const int h0 = blockIdx.y * a.heads_per;
    const int heads = min(a.heads_per, a.Hq + a.Hk - h0);
    const int units = a.D >> 4, nu = a.rot >> 4;

    if (a.cu) {
        // the sequence of each token: the last one that begins at or before it.
        // Sixteen lanes look for a token's, entries in turn.
        for (int i = tid >> 4; i < nt; i += kRopeThreads >> 4) {
            const long long t = t0 + i;
            int b = -1;  // entries [0, b] begin at or before t
            for (int e = tid & 15; e <= a.B; e += 16)
                if (a.cu[e] <= t) b = max(b, e);
#pragma unroll
            for (int d = 8; d; d >>= 1) b = max(b, __shfl_xor_sync(0xffffu << (tid & 16), b, d));
            if (a.zero_rest && (b < 0 || b >= a.B))  // here, where it costs the other rows nothing
                for (int e = tid & 15; e < heads * (a.D >> 3); e += 16) {
                    const int h = h0 + e / (a.D >> 3);
                    uint16_t* row = h < a.Hq ? static_cast<uint16_t*>(a.oq) + t * a.voq.sn + h * a.voq.sh
                                             : static_cast<uint16_t*>(a.ok) + t * a.vok.sn + (h - a.Hq) * a.vok.sh;
                    reinterpret_cast<uint4*>(row)[e % (a.D >> 3)] = make_uint4(0u, 0u, 0u, 0u);
                }
            if ((tid & 15) == 0) {
                RopeToken k{};
                k.there = b >= 0 && b < a.B;
                if (k.there) {
                    k.pos = a.pos ? a.pos[t] : (a.start ? a.start[b] : 0) + (t - a.cu[b]);
                    k.q = t * a.vq.sn;
                    k.oq = t * a.voq.sn;
                    k.k = t * a.vk.sn;
                    k.ok = t * a.vok.sn;
                }
                tok[i] = k;
            }
        }
    } else if (tid < nt) {
        const long long t = t0 + tid;
        const long long b = t / a.N, n = t - b * a.N;
        RopeToken k;
        k.there = 1;
        k.pos = a.pos ? a.pos[t] : (a.start ? a.start[b] : 0) + n;
        k.q = b * a.vq.sb + n * a.vq.sn;
        k.oq = b * a.voq.sb + n * a.voq.sn;
        k.k = b * a.vk.sb + n * a.vk.sn;
        k.ok = b * a.vok.sb + n * a.vok.sn;
        tok[tid] = k;
    }
    __syncthreads();

    const int slots = kRopeThreads / units;
    const int slot = tid / units, u = tid - slot * units;
    const int items = slot < slots ? nt * heads : 0;  // threads past the last whole slot have none
    const bool turned = u < nu;
    // my two vectors of a row
    const int e0 = turned && !INTERLEAVED ? 8 * u : 16 * u;
    const int e1 = turned && !INTERLEAVED ? (a.rot >> 1) + 8 * u : 16 * u + 8;
    bool built = false;
    for (int first = slot;; first += slots * kRopeBatch) {
        uint4 x[kRopeBatch], y[kRopeBatch];
        uint16_t* dst[kRopeBatch];
        int of[kRopeBatch];
#pragma unroll
        for (int j = 0; j < kRopeBatch; ++j) {
            const int item = first + j * slots;
            dst[j] = nullptr;
            of[j] = 0;
            if (item < items) {
                const int i = item / heads, h = h0 + item - i * heads;
                const RopeToken& k = tok[i];
                const bool is_q = h < a.Hq;
                const uint16_t* src = is_q ? static_cast<const uint16_t*>(a.q) + k.q + h * a.vq.sh
                                           : static_cast<const uint16_t*>(a.k) + k.k + (h - a.Hq) * a.vk.sh;
                if (k.there && (turned || (is_q ? a.copy_q : a.copy_k))) {
                    dst[j] = is_q ? static_cast<uint16_t*>(a.oq) + k.oq + h * a.voq.sh
                                  : static_cast<uint16_t*>(a.ok) + k.ok + (h - a.Hq) * a.vok.sh;
                    of[j] = i;
                    x[j] = *reinterpret_cast<const uint4*>(src + e0);
                    y[j] = *reinterpret_cast<const uint4*>(src + e1);
                }
            }
        }
        if (!built) {
            const int pairs = a.rot >> 1;
            for (int e = tid; e < nt * pairs; e += kRopeThreads) {
                const int i = e / pairs, p = e - i * pairs;
                const unsigned long long turn = static_cast<unsigned long long>(tok[i].pos) * a.turns[p];
                // the fraction's upper half as half-turns in [-1, 1)
                const float half = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;
                float sn, cs;
                sincospif(half, &sn, &cs);
                table[((i * 4 + (p & 7) / 2) * nu + (p >> 3)) * 2 + (p & 1)] =
                    make_float2(cs * a.mscale, sn * a.mscale * a.sign);
            }
            __syncthreads();
            built = true;
        }
#pragma unroll
        for (int j = 0; j < kRopeBatch; ++j)
            if (dst[j]) {
                if (turned)
                    turn16<BF16, INTERLEAVED>(x[j], y[j],
                                              reinterpret_cast<const float4*>(table) + of[j] * 4 * nu + u, nu);
                *reinterpret_cast<uint4*>(dst[j] + e0) = x[j];
                *reinterpret_cast<uint4*>(dst[j] + e1) = y[j];
            }
        if (first + slots * kRopeBatch >= items) break;
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& args, cudaStream_t s)
{
    RopeArgs a = args;
    const long long T = a.cu ? a.total : static_cast<long long>(a.B) * a.N;
    const int heads = a.Hq + a.Hk, units = a.D >> 4, slots = kRopeThreads / units;
    const long long sms = num_sms() > 0 ? num_sms() : 152;
    // Tokens per CTA: enough rows for two batches of every thread, as long as
    // four CTAs per SM are left and the table holds their cos and sin.
    long long per = 2 * kRopeBatch * slots / heads;
    if (per > T / (4 * sms)) per = T / (4 * sms);
    if (per > 2 * kRopePairs / a.rot) per = 2 * kRopePairs / a.rot;
    if (per > kRopeTokens) per = kRopeTokens;
    if (per < 1) per = 1;
    const long long ctas = (T + per - 1) / per;
    // few tokens: their heads are dealt out over CTAs, a slot's row at least each
    long long split = (4 * sms + ctas - 1) / ctas;
    const long long most = (heads * per + slots - 1) / slots;
    if (split > most) split = most;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.per_cta = static_cast<int>(per);
    a.heads_per = static_cast<int>((heads + split - 1) / split);
    if ((heads + a.heads_per - 1) / a.heads_per > 65535) a.heads_per = (heads + 65534) / 65535;
    a.copy_q = a.rot < a.D && a.q != a.oq;
    a.copy_k = a.rot < a.D && a.k != a.ok;
    const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>((heads + a.heads_per - 1) / a.heads_per));
    auto kern = a.bf16 ? (a.interleaved ? rope_kernel<true, true> : rope_kernel<true, false>)
                       : (a.interleaved ? rope_kernel<false, true> : rope_kernel<false, false>);
    return launch_dependent(kern, grid, kRopeThreads, 0, s, a);
}

}  // namespace ffpa
