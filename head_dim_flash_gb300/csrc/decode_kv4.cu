// Decode / short-query forward over the paged 4-bit K/V cache.
//
// The operation is ffpa_decode_fwd's on the cached values: S = scale q K^T
// over the sequence's cached tokens (bottom-right causal), O = softmax(S) V,
// LSE = ln sum exp S. One CTA per query row; its warps take strips of 16
// tokens in turn, keep a running maximum and sum each, and are joined at the
// end.
#include "kv4.cuh"

namespace ffpa {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxChunks = 16;

template <bool BF16>
__global__ void __launch_bounds__(kWarps * 32) decode_kv4_kernel(const Kv4Decode a)
{
    const Problem& pb = a.f.pb;
    const long long u = unit_id();
    if (u >= static_cast<long long>(pb.B) * pb.Hq * pb.Nq) return;
    const int i = static_cast<int>(u % pb.Nq), h = static_cast<int>(u / pb.Nq % pb.Hq);
    const int b = static_cast<int>(u / (static_cast<long long>(pb.Nq) * pb.Hq)), hk = h / (pb.Hq / pb.Hkv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, chunks = pb.D >> 6;
    long long len = a.seq_lens[b];
    if (len < 0 || len > static_cast<long long>(a.cache.max_blocks) * a.cache.page_size) {
        if (threadIdx.x == 0) kv4_invalid(a.f.ctl.status, VS_KV4_DECODE, b);
        len = 0;
    }
    const int end = static_cast<int>(pb.causal ? len - pb.Nq + 1 + i : len);  // first key the row does not see
    __shared__ float qs[1024], os[1024], ms[kWarps], ls[kWarps];
    const uint16_t* q = static_cast<const uint16_t*>(a.f.q) + b * pb.vq.sb + h * pb.vq.sh + i * pb.vq.sn;
    for (int d = 2 * threadIdx.x; d < pb.D; d += 2 * blockDim.x) {
        const float2 f = unpack2<BF16>(*reinterpret_cast<const uint32_t*>(q + d));
        qs[d] = f.x;
        qs[d + 1] = f.y;
    }
    __syncthreads();
    float m = -INFINITY, l = 0.f, o[kMaxChunks][8];
    for (int c = 0; c < kMaxChunks; ++c)
        for (int e = 0; e < 8; ++e) o[c][e] = 0.f;
    for (int t0 = warp * 16; t0 < end; t0 += kWarps * 16) {
        const int block = t0 / a.cache.page_size;
        const int page = a.cache.table[b * a.cache.table_stride + block];
        if (page < 0 || page >= a.cache.num_pages) {
            if (lane == 0) kv4_invalid(a.f.ctl.status, VS_KV4_DECODE, b);
            continue;
        }
        const uint8_t* base =
            a.cache.data + kv4_strip_offset(a.cache, pb.Hkv, chunks, page, 0, hk, (t0 - block * a.cache.page_size) >> 4);
        const size_t v_off = static_cast<size_t>(pb.Hkv) * (a.cache.page_size >> 4) * chunks * kKv4Tile;
        float s[2] = {0.f, 0.f};  // tokens g, g + 8
        for (int c = 0; c < chunks; ++c) {
            const uint8_t* tile = base + c * kKv4Tile;
            const uint4 w = *reinterpret_cast<const uint4*>(tile + lane * 16);
            const uint32_t code[4] = {w.x, w.y, w.z, w.w};
            const uint32_t sc = *reinterpret_cast<const uint16_t*>(tile + 512 + lane * 2);
            for (int e = 0; e < 4; ++e) {
                uint32_t x[4];
                kv4_dequant8(code[e], kv4_scale2(sc >> (8 * (e >> 1))), x);
                const float* qq = qs + c * 64 + t * 16 + (e & 1) * 8;
                for (int p = 0; p < 4; ++p) {
                    const float2 f = unpack2<false>(x[p]);
                    s[e >> 1] += f.x * qq[2 * p] + f.y * qq[2 * p + 1];
                }
            }
        }
        for (int hi = 0; hi < 2; ++hi) {
            s[hi] += __shfl_xor_sync(0xffffffffu, s[hi], 1);
            s[hi] += __shfl_xor_sync(0xffffffffu, s[hi], 2);
            s[hi] = t0 + g + 8 * hi < end ? s[hi] * pb.scale_log2 : -INFINITY;
        }
        float mx = fmaxf(s[0], s[1]);
        for (int d = 4; d < 32; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m, mx), al = mn == -INFINITY ? 1.f : exp2f(m - mn);
        m = mn;
        const float mu = mn == -INFINITY ? 0.f : mn;
        float p[2] = {exp2f(s[0] - mu), exp2f(s[1] - mu)}, sum = p[0] + p[1];
        for (int d = 4; d < 32; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l = l * al + sum;
        float pv[4];  // tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9
        for (int j = 0; j < 4; ++j) pv[j] = __shfl_sync(0xffffffffu, p[j >> 1], (2 * t + (j & 1)) * 4);
#pragma unroll
        for (int c = 0; c < kMaxChunks; ++c) {
            if (c >= chunks) break;
            const uint8_t* tile = base + v_off + c * kKv4Tile;
            const uint4 w = *reinterpret_cast<const uint4*>(tile + lane * 16);
            const uint32_t code[4] = {w.x, w.y, w.z, w.w};
            const uint32_t sc = *reinterpret_cast<const uint32_t*>(tile + 512 + ((g >> 1) * 4 + t) * 4);
            for (int e = 0; e < 8; ++e) o[c][e] *= al;
            for (int j = 0; j < 4; ++j) {
                if (t0 + 2 * t + (j & 1) + 8 * (j >> 1) >= end) continue;  // cells behind the row's keys hold anything
                uint32_t x[4];
                kv4_dequant8(code[j], kv4_scale2(sc >> (8 * j)), x);
                for (int k = 0; k < 4; ++k) {
                    const float2 f = unpack2<false>(x[k]);
                    o[c][2 * k] += pv[j] * f.x;
                    o[c][2 * k + 1] += pv[j] * f.y;
                }
            }
        }
    }
    if (lane == 0) {
        ms[warp] = m;
        ls[warp] = l;
    }
    for (int d = threadIdx.x; d < pb.D; d += blockDim.x) os[d] = 0.f;
    __syncthreads();
    float mx = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, ms[w]);
    const float mu = mx == -INFINITY ? 0.f : mx;
    for (int w = 0; w < kWarps; ++w) sum += ls[w] * exp2f(ms[w] - mu);
    const float f = sum > 0.f ? exp2f(m - mu) / sum : 0.f;
    for (int w = 0; w < kWarps; ++w) {  // in turn: the sum's order is fixed
        if (w == warp)
#pragma unroll
            for (int c = 0; c < kMaxChunks; ++c) {
                if (c >= chunks) break;
                for (int e = 0; e < 8; ++e) {
                    float x = o[c][e];
                    x += __shfl_xor_sync(0xffffffffu, x, 1);
                    x += __shfl_xor_sync(0xffffffffu, x, 2);
                    if (t == 0) os[c * 64 + 8 * g + e] += x * f;
                }
            }
        __syncthreads();
    }
    uint16_t* out = static_cast<uint16_t*>(a.f.o) + b * pb.vo.sb + h * pb.vo.sh + i * pb.vo.sn;
    for (int d = 2 * threadIdx.x; d < pb.D; d += 2 * blockDim.x)
        *reinterpret_cast<uint32_t*>(out + d) = pack2<BF16>(os[d], os[d + 1]);
    if (threadIdx.x == 0) a.f.lse[u] = sum > 0.f ? (mx + log2f(sum)) * 0.693147180559945309f : -INFINITY;
}

}  // namespace

size_t kv4_decode_workspace_bytes(const Problem&) { return 0; }

cudaError_t launch_decode_kv4(const Kv4Decode& a, void*, cudaStream_t s)
{
    dim3 grid;
    if (!unit_grid(1, static_cast<long long>(a.f.pb.B) * a.f.pb.Hq * a.f.pb.Nq, &grid)) return cudaErrorInvalidConfiguration;
    if (a.f.bf16)
        decode_kv4_kernel<true><<<grid, kWarps * 32, 0, s>>>(a);
    else
        decode_kv4_kernel<false><<<grid, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace ffpa
