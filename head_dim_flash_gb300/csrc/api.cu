// C ABI entry points (declared in include/ffpa.h): argument validation,
// workspace carving, device status word, and dispatch to the kernels.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>

#include "../../include/ffpa.h"
#include "cache_ops.h"
#include "kernels.h"
#include "kv4.h"
#include "ptx.cuh"

namespace {

thread_local std::string g_err;
std::atomic<uint64_t> g_limit_ns{2000000000ull};

ffpa_status fail(ffpa_status s, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_err = buf;
    return s;
}

ffpa_status ok()
{
    g_err.clear();
    return FFPA_OK;
}

}  // namespace

// One status word per device; kernels record the first failing wait here.
__device__ uint32_t g_ffpa_status_word;

namespace {

constexpr int kMaxDevices = 64;
uint32_t* g_status_ptr[kMaxDevices];
int g_cc_ok[kMaxDevices];  // 0 unknown, 1 yes, -1 no
std::mutex g_dev_mu;

// Device address of the status word on the current device (looked up once).
bool device_state(uint32_t** status, bool* cc_ok)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (!g_status_ptr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_ffpa_status_word) != cudaSuccess) return false;
        g_status_ptr[dev] = static_cast<uint32_t*>(p);
        int major = 0, minor = 0;
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        g_cc_ok[dev] = (major == 10 && minor == 3) ? 1 : -1;
    }
    *status = g_status_ptr[dev];
    *cc_ok = g_cc_ok[dev] == 1;
    return true;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

ffpa_status check_common(ffpa_dtype dt, int Hq, int Hkv, int D, float scale)
{
    if (dt != FFPA_BF16 && dt != FFPA_FP16) return fail(FFPA_ERR_NOT_SUPPORTED, "dtype %d: only bf16 (0) and fp16 (1)", (int)dt);
    if (D < 64 || D > 1024 || D % 32 != 0)
        return fail(FFPA_ERR_NOT_SUPPORTED, "head dim D=%d: supported D is a multiple of 32 in [64, 1024]", D);
    if (Hq < 0 || Hkv < 0) return fail(FFPA_ERR_INVALID_VALUE, "negative head count Hq=%d Hkv=%d", Hq, Hkv);
    if (Hq > 0 && (Hkv == 0 || Hq % Hkv != 0))
        return fail(FFPA_ERR_INVALID_VALUE, "Hq=%d must be a positive multiple of Hkv=%d", Hq, Hkv);
    if (!std::isfinite(scale)) return fail(FFPA_ERR_INVALID_VALUE, "scale must be finite");
    return FFPA_OK;
}

ffpa_status check_ptr(const void* p, bool needed, const char* name)
{
    if (!needed) return FFPA_OK;
    if (!p) return fail(FFPA_ERR_INVALID_VALUE, "%s is NULL", name);
    if (!aligned16(p)) return fail(FFPA_ERR_INVALID_VALUE, "%s is not 16-byte aligned", name);
    return FFPA_OK;
}

ffpa_status device_ctl(ffpa::DeviceCtl* ctl)
{
    bool cc_ok = false;
    uint32_t* st = nullptr;
    if (!device_state(&st, &cc_ok)) return fail(FFPA_ERR_CUDA, "no usable CUDA device");
    if (!cc_ok) return fail(FFPA_ERR_NOT_SUPPORTED, "device is not compute capability 10.3 (sm_103)");
    if (!ffpa::encode_fn()) return fail(FFPA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable from the driver");
    ctl->status = st;
    ctl->limit_ns = g_limit_ns.load();
    return FFPA_OK;
}

ffpa_status launch_result(cudaError_t e, const char* what)
{
    if (e != cudaSuccess) return fail(FFPA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return ok();
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Work units one launch can index (unit_grid: 65535 x 65535 clusters).
constexpr long long kMaxUnits = 65535LL * 65535LL;

size_t ws_bytes(long rows) { return rows <= 0 ? 0 : 2 * align256(static_cast<size_t>(rows) * sizeof(float)); }

// Strides of a contiguous [B, H, N, D] tensor, and of a packed [T, H, D] one.
ffpa::View contiguous_view(int H, int N, int D)
{
    return ffpa::View{static_cast<long long>(H) * N * D, static_cast<long long>(N) * D, D};
}

ffpa::View packed_view(int H, int D) { return ffpa::View{0, D, static_cast<long long>(H) * D}; }

// A strided view as the ABI describes it: strides are multiples of 8 elements
// (16 bytes), non-negative, positive along every dimension with more than one
// entry, and below 2^39 elements (the tensor-map limit of 2^40 bytes).
ffpa_status check_view(const ffpa_view& v, bool needed, const char* name, int B, int H, int N)
{
    if (!needed) return FFPA_OK;
    if (!v.data) return fail(FFPA_ERR_INVALID_VALUE, "%s: data is NULL", name);
    if (reinterpret_cast<uintptr_t>(v.data) & 15u) return fail(FFPA_ERR_INVALID_VALUE, "%s: data is not 16-byte aligned", name);
    const int64_t st[3] = {v.stride_b, v.stride_h, v.stride_n};
    const int ext[3] = {B, H, N};
    const char* dim[3] = {"stride_b", "stride_h", "stride_n"};
    for (int i = 0; i < 3; ++i) {
        if (st[i] < 0 || st[i] % 8 != 0 || st[i] >= (int64_t(1) << 39))
            return fail(FFPA_ERR_INVALID_VALUE, "%s: %s=%lld must be a non-negative multiple of 8 below 2^39", name, dim[i],
                        (long long)st[i]);
        if (ext[i] > 1 && st[i] == 0) return fail(FFPA_ERR_INVALID_VALUE, "%s: %s is 0 for an extent of %d", name, dim[i], ext[i]);
    }
    return FFPA_OK;
}

ffpa::View to_view(const ffpa_view& v) { return ffpa::View{v.stride_b, v.stride_h, v.stride_n}; }

ffpa::Problem dense_problem(int B, int Hq, int Hkv, int Nq, int Nkv, int D, int causal, float scale)
{
    ffpa::Problem pb{};
    pb.varlen = 0;
    pb.B = B;
    pb.Hq = Hq;
    pb.Hkv = Hkv;
    pb.Nq = Nq;
    pb.Nkv = Nkv;
    pb.D = D;
    pb.causal = causal ? 1 : 0;
    pb.scale = scale;
    pb.scale_log2 = scale * 1.4426950408889634f;
    pb.vq = pb.vo = pb.vdo = pb.vdq = contiguous_view(Hq, Nq, D);
    pb.vk = pb.vv = pb.vdk = pb.vdv = contiguous_view(Hkv, Nkv, D);
    return pb;
}

ffpa_status check_dense_sizes(int B, int Hq, int Nq, int Nkv)
{
    if (B < 0 || Nq < 0 || Nkv < 0) return fail(FFPA_ERR_INVALID_VALUE, "negative size B=%d Nq=%d Nkv=%d", B, Nq, Nkv);
    // (batch, head) pairs index the launch grids as int
    if (static_cast<long>(B) * Hq > INT_MAX || static_cast<long>(B) * Hq * ((Nq > Nkv ? Nq : Nkv) / 128 + 1) > kMaxUnits)
        return fail(FFPA_ERR_NOT_SUPPORTED, "B*Hq=%ld with N=%d exceeds the launch grid's %lld work units", (long)B * Hq,
                    Nq > Nkv ? Nq : Nkv, kMaxUnits);
    return FFPA_OK;
}

ffpa_status check_varlen_sizes(int batch, int total_q, int total_k, int max_q, int max_k, int Hq, const int* cu_q,
                               const int* cu_k)
{
    if (batch < 0 || total_q < 0 || total_k < 0 || max_q < 0 || max_k < 0)
        return fail(FFPA_ERR_INVALID_VALUE, "negative varlen size");
    if (static_cast<long>(batch) * Hq > INT_MAX ||
        static_cast<long>(batch) * Hq * ((max_q > max_k ? max_q : max_k) / 128 + 1) > kMaxUnits)
        return fail(FFPA_ERR_NOT_SUPPORTED, "batch*Hq=%ld with max_seqlen %d exceeds the launch grid's %lld work units",
                    (long)batch * Hq, max_q > max_k ? max_q : max_k, kMaxUnits);
    if (batch > 0 && (!cu_q || !cu_k))
        return fail(FFPA_ERR_INVALID_VALUE, "cu_seqlens_q and cu_seqlens_k are both required (varlen-one-sided)");
    if ((reinterpret_cast<uintptr_t>(cu_q) & 3u) || (reinterpret_cast<uintptr_t>(cu_k) & 3u))
        return fail(FFPA_ERR_INVALID_VALUE, "cu_seqlens must be 4-byte aligned");
    return FFPA_OK;
}

#define FFPA_TRY(x)                              \
    do {                                         \
        const ffpa_status s_ = (x);              \
        if (s_ != FFPA_OK) return s_;            \
    } while (0)

ffpa_status run_fwd(ffpa_dtype dt, const void* q, const void* k, const void* v, void* o, float* lse,
                    const ffpa::Problem& pb, long q_rows, long k_rows, ffpa_stream_t stream)
{
    FFPA_TRY(check_ptr(q, q_rows > 0, "q"));
    FFPA_TRY(check_ptr(o, q_rows > 0, "o"));
    FFPA_TRY(check_ptr(lse, q_rows > 0, "lse"));
    FFPA_TRY(check_ptr(k, q_rows > 0 && k_rows > 0, "k"));
    FFPA_TRY(check_ptr(v, q_rows > 0 && k_rows > 0, "v"));
    if (q_rows == 0) return ok();
    // the forward operation of the cluster-exchange kernel: each unit of a
    // cluster scores its own key tiles, the units agree on the running row
    // maximum and exchange P, and every unit accumulates its head-dim slab of O
    ffpa::XArgs a{};
    a.pb = pb;
    FFPA_TRY(device_ctl(&a.ctl));
    a.bf16 = dt == FFPA_BF16;
    a.q = q;
    a.k = k;
    a.v = v;
    a.o = o;
    a.lse = lse;
    return launch_result(ffpa::launch_xchg(ffpa::XOP_FWD, a, reinterpret_cast<cudaStream_t>(stream)),
                         "forward launch");
}

// Layout of the stored-tile part of a backward workspace (byte offsets; 0 =
// absent) for a workspace of `bytes` whose row statistics take `need`.
struct StoredPlan {
    size_t ds_off, p_off;
    int chunk_groups;  // > 0: chunks of this many kv groups
    size_t used;       // bytes the plan uses
};

StoredPlan stored_plan(const ffpa::Problem& pb, size_t need, size_t bytes, bool chunks_allowed)
{
    StoredPlan s{0, 0, 0, need};
    if (!ffpa::dsq_supported(pb)) return s;
    const size_t t_all = ffpa::dsq_ds_bytes(pb), t_g = ffpa::dsq_group_bytes(pb);
    if (bytes >= need + align256(t_all) + t_all) {  // every head at once
        s.ds_off = need;
        s.p_off = need + align256(t_all);
        s.used = s.p_off + t_all;
        return s;
    }
    if (chunks_allowed && t_g > 0 && bytes >= need + align256(t_g) + t_g) {
        // as many kv groups per chunk as fit, then the chunks evened out
        // (ceil(Hkv / chunks) groups each), so that no launch is a small tail
        long ng = static_cast<long>((bytes - need) / (2 * t_g + 256));
        if (ng < 1) ng = 1;
        while (ng > 1 && need + align256(ng * t_g) + ng * t_g > bytes) --ng;
        const long chunks = (pb.Hkv + ng - 1) / ng;
        ng = (pb.Hkv + chunks - 1) / chunks;
        s.chunk_groups = static_cast<int>(ng);
        s.ds_off = need;
        s.p_off = need + align256(ng * t_g);
        s.used = s.p_off + ng * t_g;
        return s;
    }
    if (bytes >= need + t_all) {  // dS^T of every head
        s.ds_off = need;
        s.used = need + t_all;
    }
    return s;
}

// Largest useful backward workspace within `budget` bytes: every head's tiles
// if they fit, else the largest chunk of kv groups that fits (evened out),
// else the row statistics alone.
size_t budget_bytes(const ffpa::Problem& pb, size_t need, size_t budget)
{
    if (budget <= need) return need;
    return stored_plan(pb, need, budget, true).used;
}

ffpa_status run_bwd(ffpa_dtype dt, const void* q, const void* k, const void* v, const void* o, const float* lse,
                    const void* dO, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                    const ffpa::Problem& pb, long q_rows, long k_rows, long stat_rows, unsigned stages,
                    ffpa_stream_t stream)
{
    const bool any = q_rows > 0 || k_rows > 0;
    FFPA_TRY(check_ptr(q, q_rows > 0, "q"));
    FFPA_TRY(check_ptr(o, q_rows > 0, "o"));
    FFPA_TRY(check_ptr(lse, q_rows > 0, "lse"));
    FFPA_TRY(check_ptr(dO, q_rows > 0, "dO"));
    FFPA_TRY(check_ptr(dq, q_rows > 0, "dq"));
    FFPA_TRY(check_ptr(k, k_rows > 0, "k"));
    FFPA_TRY(check_ptr(v, k_rows > 0, "v"));
    FFPA_TRY(check_ptr(dk, k_rows > 0, "dk"));
    FFPA_TRY(check_ptr(dv, k_rows > 0, "dv"));
    const size_t need = ws_bytes(stat_rows);
    if (workspace_bytes < need)
        return fail(FFPA_ERR_INVALID_VALUE, "workspace too small: %zu < %zu bytes", workspace_bytes, need);
    if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return fail(FFPA_ERR_INVALID_VALUE, "workspace must be non-NULL and 256-byte aligned");
    if (!any) return ok();
    ffpa::BwdArgs a{};
    a.pb = pb;
    a.stages = stages & 63u;
    // The workspace after the row statistics decides the stored-tile path
    // (where it applies): room for dS^T and P^T of every head has the dK
    // launch store both, and dV and dQ are GEMMs over them; room for both
    // tile sets of at least one kv group (and a call that runs dV, dK and dQ)
    // runs that path in chunks of as many groups as fit; room for dS^T of
    // every head alone stores dS only (dV recomputes); less recomputes.
    a.ds = nullptr;
    a.p = nullptr;
    a.chunk_groups = 0;
    const StoredPlan plan = stored_plan(pb, need, workspace_bytes, (stages & 14u) == 14u && !(stages & 48u));
    if (plan.ds_off) a.ds = static_cast<char*>(workspace) + plan.ds_off;
    if (plan.p_off) a.p = static_cast<char*>(workspace) + plan.p_off;
    a.chunk_groups = plan.chunk_groups;
    if ((a.stages & 16u) && a.ds == nullptr)
        return fail(FFPA_ERR_INVALID_VALUE, "stage bit 4 (dQ from stored dS) needs the larger workspace of "
                                            "ffpa_bwd_workspace_bytes_ds on a dense problem with D % 64 == 0, D <= 1024");
    if ((a.stages & 32u) && a.p == nullptr)
        return fail(FFPA_ERR_INVALID_VALUE, "stage bit 5 (stored P) needs the workspace of "
                                            "ffpa_bwd_workspace_bytes_ds on a dense problem with D % 64 == 0, D <= 1024");
    FFPA_TRY(device_ctl(&a.ctl));
    a.bf16 = dt == FFPA_BF16;
    a.q = q;
    a.k = k;
    a.v = v;
    a.o = o;
    a.dO = dO;
    a.lse = lse;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.delta = static_cast<float*>(workspace);
    a.lse_log2 = reinterpret_cast<float*>(static_cast<char*>(workspace) + need / 2);
    return launch_result(ffpa::launch_bwd(a, reinterpret_cast<cudaStream_t>(stream)), "backward launch");
}

ffpa::Problem varlen_problem(int batch, int total_q, int total_k, int max_q, int max_k, int Hq, int Hkv, int D,
                             int causal, float scale, const int* cu_q, const int* cu_k)
{
    ffpa::Problem pb = dense_problem(batch, Hq, Hkv, max_q, max_k, D, causal, scale);
    pb.varlen = 1;
    pb.total_q = total_q;
    pb.total_k = total_k;
    pb.cu_q = cu_q;
    pb.cu_k = cu_k;
    pb.vq = pb.vo = pb.vdo = pb.vdq = packed_view(Hq, D);
    pb.vk = pb.vv = pb.vdk = pb.vdv = packed_view(Hkv, D);
    return pb;
}

__global__ void selftest_wait_kernel(uint32_t* status, uint64_t limit_ns)
{
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        ffpa::mbar_init(&bar, 1);
        abort_flag = 0;
        ffpa::fence_barrier_init();
        // nothing ever arrives on `bar`: the wait must give up by itself
        ffpa::mbar_wait(&bar, 0, &abort_flag, status, limit_ns, 255);
    }
}

}  // namespace

int ffpa::set_error(int status, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_err = buf;
    return status;
}

extern "C" {

ffpa_status ffpa_fwd(ffpa_dtype dt, const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                     int Hkv, int Nq, int Nkv, int D, int causal, float scale, ffpa_stream_t stream)
{
    FFPA_TRY(check_common(dt, Hq, Hkv, D, scale));
    FFPA_TRY(check_dense_sizes(B, Hq, Nq, Nkv));
    const long q_rows = static_cast<long>(B) * Hq * Nq;
    const long k_rows = static_cast<long>(B) * Hkv * Nkv;
    return run_fwd(dt, q, k, v, o, lse, dense_problem(B, Hq, Hkv, Nq, Nkv, D, causal, scale), q_rows, k_rows, stream);
}

ffpa_status ffpa_fwd_strided(ffpa_dtype dt, ffpa_view q, ffpa_view k, ffpa_view v, ffpa_view o, float* lse, int B,
                             int Hq, int Hkv, int Nq, int Nkv, int D, int causal, float scale, ffpa_stream_t stream)
{
    FFPA_TRY(check_common(dt, Hq, Hkv, D, scale));
    FFPA_TRY(check_dense_sizes(B, Hq, Nq, Nkv));
    const long q_rows = static_cast<long>(B) * Hq * Nq;
    const long k_rows = static_cast<long>(B) * Hkv * Nkv;
    FFPA_TRY(check_view(q, q_rows > 0, "q", B, Hq, Nq));
    FFPA_TRY(check_view(o, q_rows > 0, "o", B, Hq, Nq));
    FFPA_TRY(check_view(k, q_rows > 0 && k_rows > 0, "k", B, Hkv, Nkv));
    FFPA_TRY(check_view(v, q_rows > 0 && k_rows > 0, "v", B, Hkv, Nkv));
    ffpa::Problem pb = dense_problem(B, Hq, Hkv, Nq, Nkv, D, causal, scale);
    pb.vq = to_view(q);
    pb.vo = to_view(o);
    pb.vk = to_view(k);
    pb.vv = to_view(v);
    return run_fwd(dt, q.data, k.data, v.data, o.data, lse, pb, q_rows, k_rows, stream);
}

size_t ffpa_decode_workspace_bytes(ffpa_dtype, int B, int Hq, int Hkv, int Nq, int Nkv, int D)
{
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq <= 0 || Nkv < 0 || D <= 0 || Hq % Hkv != 0) return 0;
    return ffpa::decode_plan(dense_problem(B, Hq, Hkv, Nq, Nkv, D, 0, 1.f)).workspace_bytes;
}

ffpa_status ffpa_decode_fwd(ffpa_dtype dt, ffpa_view q, ffpa_view k, ffpa_view v, ffpa_view o, float* lse,
                            void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int Nkv, int D,
                            int causal, float scale, ffpa_stream_t stream)
{
    FFPA_TRY(check_common(dt, Hq, Hkv, D, scale));
    FFPA_TRY(check_dense_sizes(B, Hq, Nq, Nkv));
    if (D % 64 != 0) return fail(FFPA_ERR_NOT_SUPPORTED, "decode path: D=%d must be a multiple of 64", D);
    if (Hq > 0 && static_cast<long long>(B) * Hkv * ((static_cast<long long>(Hq / Hkv) * Nq + ffpa::kDecodeRows - 1) /
                                                     ffpa::kDecodeRows) > kMaxUnits)
        return fail(FFPA_ERR_NOT_SUPPORTED, "decode path: B*Hkv*ceil((Hq/Hkv)*Nq/%d) exceeds the grid's %lld units",
                    ffpa::kDecodeRows, kMaxUnits);
    const long q_rows = static_cast<long>(B) * Hq * Nq;
    const long k_rows = static_cast<long>(B) * Hkv * Nkv;
    FFPA_TRY(check_view(q, q_rows > 0, "q", B, Hq, Nq));
    FFPA_TRY(check_view(o, q_rows > 0, "o", B, Hq, Nq));
    FFPA_TRY(check_view(k, q_rows > 0 && k_rows > 0, "k", B, Hkv, Nkv));
    FFPA_TRY(check_view(v, q_rows > 0 && k_rows > 0, "v", B, Hkv, Nkv));
    FFPA_TRY(check_ptr(lse, q_rows > 0, "lse"));
    if (q_rows == 0) return ok();
    ffpa::Problem pb = dense_problem(B, Hq, Hkv, Nq, Nkv, D, causal, scale);
    pb.vq = to_view(q);
    pb.vo = to_view(o);
    pb.vk = to_view(k);
    pb.vv = to_view(v);
    const size_t need = ffpa::decode_plan(pb).workspace_bytes;
    if (workspace_bytes < need)
        return fail(FFPA_ERR_INVALID_VALUE, "decode workspace too small: %zu < %zu bytes", workspace_bytes, need);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return fail(FFPA_ERR_INVALID_VALUE, "decode workspace must be non-NULL and 256-byte aligned");
    ffpa::FwdArgs a{};
    a.pb = pb;
    FFPA_TRY(device_ctl(&a.ctl));
    a.bf16 = dt == FFPA_BF16;
    a.q = q.data;
    a.k = k.data;
    a.v = v.data;
    a.o = o.data;
    a.lse = lse;
    return launch_result(ffpa::launch_decode(a, workspace, reinterpret_cast<cudaStream_t>(stream)), "decode launch");
}

size_t ffpa_fp8_workspace_layout(int B, int Hq, int Hkv, int Nq, int Nkv, int D, size_t* offsets)
{
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq < 0 || Nkv < 0 || D < 64 || D > 1024 || Hq % Hkv != 0 || D % 32 != 0)
        return 0;
    const ffpa::Fp8Layout L = ffpa::fp8_layout(B, Hq, Hkv, Nq, Nkv, D);
    if (offsets) {
        offsets[0] = L.q8;
        offsets[1] = L.k8;
        offsets[2] = L.v8t;
        offsets[3] = L.sq;
        offsets[4] = L.sk;
        offsets[5] = L.sv;
        offsets[6] = static_cast<size_t>(L.ldv);
        offsets[7] = L.total;
    }
    return L.total;
}

size_t ffpa_fp8_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nkv, int D)
{
    return ffpa_fp8_workspace_layout(B, Hq, Hkv, Nq, Nkv, D, nullptr);
}

}  // extern "C"

namespace {

// Validation shared by the FP8 entry points; fills `pb` on success.
ffpa_status check_fp8(ffpa_dtype dt, const ffpa_view& q, const ffpa_view& k, const ffpa_view& v, const void* ws,
                      size_t ws_bytes, int B, int Hq, int Hkv, int Nq, int Nkv, int D, float scale, ffpa::Problem* pb)
{
    FFPA_TRY(check_common(dt, Hq, Hkv, D, scale));
    FFPA_TRY(check_dense_sizes(B, Hq, Nq, Nkv));
    const long q_rows = static_cast<long>(B) * Hq * Nq;
    if (q_rows > 0 && Nkv < 1) return fail(FFPA_ERR_NOT_SUPPORTED, "fp8 forward: Nkv must be >= 1");
    FFPA_TRY(check_view(q, q_rows > 0, "q", B, Hq, Nq));
    FFPA_TRY(check_view(k, q_rows > 0, "k", B, Hkv, Nkv));
    FFPA_TRY(check_view(v, q_rows > 0, "v", B, Hkv, Nkv));
    if (q_rows > 0) {
        const size_t need = ffpa::fp8_layout(B, Hq, Hkv, Nq, Nkv, D).total;
        if (ws_bytes < need)
            return fail(FFPA_ERR_INVALID_VALUE, "fp8 workspace too small: %zu < %zu bytes", ws_bytes, need);
        if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u))
            return fail(FFPA_ERR_INVALID_VALUE, "fp8 workspace must be non-NULL and 256-byte aligned");
    }
    *pb = dense_problem(B, Hq, Hkv, Nq, Nkv, D, 0, scale);
    pb->vq = to_view(q);
    pb->vk = to_view(k);
    pb->vv = to_view(v);
    return ok();
}

}  // namespace

extern "C" {

ffpa_status ffpa_fp8_quantize(ffpa_dtype dt, ffpa_view q, ffpa_view k, ffpa_view v, void* workspace,
                              size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int Nkv, int D,
                              ffpa_stream_t stream)
{
    ffpa::Problem pb;
    FFPA_TRY(check_fp8(dt, q, k, v, workspace, workspace_bytes, B, Hq, Hkv, Nq, Nkv, D, 1.f, &pb));
    if (static_cast<long>(B) * Hq * Nq == 0) return ok();
    ffpa::FwdArgs a{};
    a.pb = pb;
    FFPA_TRY(device_ctl(&a.ctl));
    a.bf16 = dt == FFPA_BF16;
    a.q = q.data;
    a.k = k.data;
    a.v = v.data;
    return launch_result(ffpa::launch_fp8_quantize(a, workspace, reinterpret_cast<cudaStream_t>(stream)),
                         "fp8 quantize launch");
}

ffpa_status ffpa_fwd_fp8(ffpa_dtype dt, ffpa_view q, ffpa_view k, ffpa_view v, ffpa_view o, float* lse,
                         void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int Nkv, int D,
                         int causal, float scale, ffpa_stream_t stream)
{
    ffpa::Problem pb;
    FFPA_TRY(check_fp8(dt, q, k, v, workspace, workspace_bytes, B, Hq, Hkv, Nq, Nkv, D, scale, &pb));
    const long q_rows = static_cast<long>(B) * Hq * Nq;
    FFPA_TRY(check_view(o, q_rows > 0, "o", B, Hq, Nq));
    FFPA_TRY(check_ptr(lse, q_rows > 0, "lse"));
    if (q_rows == 0) return ok();
    pb.causal = causal != 0;
    pb.vo = to_view(o);
    ffpa::FwdArgs a{};
    a.pb = pb;
    FFPA_TRY(device_ctl(&a.ctl));
    a.bf16 = dt == FFPA_BF16;
    a.q = q.data;
    a.k = k.data;
    a.v = v.data;
    a.o = o.data;
    a.lse = lse;
    return launch_result(ffpa::launch_fwd_fp8(a, workspace, reinterpret_cast<cudaStream_t>(stream), true),
                         "fp8 launch");
}

ffpa_status ffpa_fwd_fp8_quantized(ffpa_dtype dt, ffpa_view o, float* lse, const void* workspace,
                                   size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int Nkv, int D, int causal,
                                   float scale, ffpa_stream_t stream)
{
    // the views of q/k/v are not read: validate with dense views over the workspace
    void* ws = const_cast<void*>(workspace);
    const ffpa_view vq{ws, static_cast<long long>(Hq) * Nq * D, static_cast<long long>(Nq) * D, D};
    const ffpa_view vk{ws, static_cast<long long>(Hkv) * Nkv * D, static_cast<long long>(Nkv) * D, D};
    ffpa::Problem pb;
    FFPA_TRY(check_fp8(dt, vq, vk, vk, workspace, workspace_bytes, B, Hq, Hkv, Nq, Nkv, D, scale, &pb));
    const long q_rows = static_cast<long>(B) * Hq * Nq;
    FFPA_TRY(check_view(o, q_rows > 0, "o", B, Hq, Nq));
    FFPA_TRY(check_ptr(lse, q_rows > 0, "lse"));
    if (q_rows == 0) return ok();
    pb.causal = causal != 0;
    pb.vo = to_view(o);
    ffpa::FwdArgs a{};
    a.pb = pb;
    FFPA_TRY(device_ctl(&a.ctl));
    a.bf16 = dt == FFPA_BF16;
    a.o = o.data;
    a.lse = lse;
    return launch_result(ffpa::launch_fwd_fp8(a, const_cast<void*>(workspace),
                                              reinterpret_cast<cudaStream_t>(stream), false),
                         "fp8 launch");
}

size_t ffpa_varlen_fp8_workspace_bytes(int batch, int total_q, int total_k, int max_seqlen_q, int max_seqlen_k, int Hq,
                                       int Hkv, int D)
{
    if (batch <= 0 || total_q < 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || Hq <= 0 || Hkv <= 0 ||
        D < 64 || D > 1024 || Hq % Hkv != 0 || D % 32 != 0)
        return 0;
    return ffpa::fp8_varlen_layout(batch, Hq, Hkv, total_q, total_k, max_seqlen_q, max_seqlen_k, D).total;
}

ffpa_status ffpa_varlen_fwd_fp8(ffpa_dtype dt, const void* q, const void* k, const void* v, void* o, float* lse,
                                const int* cu_seqlens_q, const int* cu_seqlens_k, int batch, int total_q,
                                int total_k, int max_seqlen_q, int max_seqlen_k, int Hq, int Hkv, int D, int causal,
                                float scale, void* workspace, size_t workspace_bytes, ffpa_stream_t stream)
{
    FFPA_TRY(check_common(dt, Hq, Hkv, D, scale));
    FFPA_TRY(check_varlen_sizes(batch, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, cu_seqlens_q, cu_seqlens_k));
    const long q_rows = batch > 0 ? static_cast<long>(total_q) * Hq : 0;
    if (q_rows > 0 && total_k < 1) return fail(FFPA_ERR_NOT_SUPPORTED, "fp8 forward: total_k must be >= 1");
    FFPA_TRY(check_ptr(q, q_rows > 0, "q"));
    FFPA_TRY(check_ptr(k, q_rows > 0, "k"));
    FFPA_TRY(check_ptr(v, q_rows > 0, "v"));
    FFPA_TRY(check_ptr(o, q_rows > 0, "o"));
    FFPA_TRY(check_ptr(lse, q_rows > 0, "lse"));
    if (q_rows == 0) return ok();
    const size_t need =
        ffpa::fp8_varlen_layout(batch, Hq, Hkv, total_q, total_k, max_seqlen_q, max_seqlen_k, D).total;
    if (workspace_bytes < need)
        return fail(FFPA_ERR_INVALID_VALUE, "fp8 workspace too small: %zu < %zu bytes", workspace_bytes, need);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return fail(FFPA_ERR_INVALID_VALUE, "fp8 workspace must be non-NULL and 256-byte aligned");
    ffpa::FwdArgs a{};
    a.pb = varlen_problem(batch, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, D, causal, scale, cu_seqlens_q,
                          cu_seqlens_k);
    FFPA_TRY(device_ctl(&a.ctl));
    a.bf16 = dt == FFPA_BF16;
    a.q = q;
    a.k = k;
    a.v = v;
    a.o = o;
    a.lse = lse;
    return launch_result(ffpa::launch_fwd_fp8(a, workspace, reinterpret_cast<cudaStream_t>(stream), true),
                         "fp8 varlen launch");
}

size_t ffpa_kv4_cache_bytes(int num_pages, int page_size, int Hkv, int D)
{
    if (num_pages < 0 || page_size <= 0 || page_size % 16 != 0 || Hkv < 0 || D < 64 || D > 1024 || D % 64 != 0) return 0;
    return static_cast<size_t>(num_pages) * 2 * Hkv * (page_size / 16) * (D / 64) * ffpa::kKv4Tile;
}

}  // extern "C"

namespace {

// Validation shared by the entry points over the 4-bit cache (`used`: the call reaches it).
ffpa_status check_kv4_cache(const ffpa_kv4_cache& c, bool used, int Hkv, int D, ffpa::Kv4Cache* out)
{
    if (D % 64 != 0) return fail(FFPA_ERR_NOT_SUPPORTED, "4-bit cache: D=%d must be a multiple of 64", D);
    if (c.page_size <= 0 || c.page_size % 16 != 0)
        return fail(FFPA_ERR_INVALID_VALUE, "page_size=%d must be a positive multiple of 16", c.page_size);
    if (c.num_pages < 0 || c.max_blocks < 0) return fail(FFPA_ERR_INVALID_VALUE, "negative num_pages or max_blocks");
    if (c.block_stride < c.max_blocks)
        return fail(FFPA_ERR_INVALID_VALUE, "block_stride=%lld is below max_blocks=%d", (long long)c.block_stride,
                    c.max_blocks);
    FFPA_TRY(check_ptr(c.data, used && c.num_pages > 0 && Hkv > 0, "cache data"));
    if (used && c.max_blocks > 0 && !c.block_table) return fail(FFPA_ERR_INVALID_VALUE, "block_table is NULL");
    if (reinterpret_cast<uintptr_t>(c.block_table) & 3u)
        return fail(FFPA_ERR_INVALID_VALUE, "block_table must be 4-byte aligned");
    out->data = static_cast<uint8_t*>(c.data);
    out->num_pages = c.num_pages;
    out->page_size = c.page_size;
    out->table = c.block_table;
    out->max_blocks = c.num_pages > 0 ? c.max_blocks : 0;  // a cache without pages holds no tokens
    out->table_stride = c.block_stride;
    return FFPA_OK;
}

// Writes (read = false) or reads a batch; dense with views, packed with cu_seqlens.
ffpa_status run_kv4_io(bool read, ffpa_dtype dt, const ffpa_view& k, const ffpa_view& v, const ffpa_kv4_cache& cache,
                       const int* start, const int* count, const int* cu, int B, int total, int Hkv, int N, int D,
                       ffpa_stream_t stream)
{
    FFPA_TRY(check_common(dt, Hkv, Hkv, D, 1.f));
    if (B < 0 || N < 0 || total < 0) return fail(FFPA_ERR_INVALID_VALUE, "negative size B=%d N=%d total=%d", B, N, total);
    if (static_cast<long long>(B) * Hkv > kMaxUnits)
        return fail(FFPA_ERR_NOT_SUPPORTED, "B*Hkv=%lld exceeds the launch grid's %lld units", (long long)B * Hkv,
                    kMaxUnits);
    ffpa::Kv4Io a{};
    const bool any = B > 0 && Hkv > 0 && N > 0 && (!cu || total > 0);
    FFPA_TRY(check_kv4_cache(cache, any, Hkv, D, &a.cache));
    if ((reinterpret_cast<uintptr_t>(start) & 3u) || (reinterpret_cast<uintptr_t>(count) & 3u) ||
        (reinterpret_cast<uintptr_t>(cu) & 3u))
        return fail(FFPA_ERR_INVALID_VALUE, "start, count and cu_seqlens must be 4-byte aligned");
    const int ext_b = cu ? 1 : B, ext_n = cu ? total : N;
    FFPA_TRY(check_view(k, any, "k", ext_b, Hkv, ext_n));
    FFPA_TRY(check_view(v, any, "v", ext_b, Hkv, ext_n));
    if (!any) return ok();
    ffpa::DeviceCtl ctl;
    FFPA_TRY(device_ctl(&ctl));
    a.bf16 = dt == FFPA_BF16;
    a.B = B;
    a.Hkv = Hkv;
    a.N = N;
    a.D = D;
    a.k = k.data;
    a.v = v.data;
    a.vk = to_view(k);
    a.vv = to_view(v);
    a.start = start;
    a.count = count;
    a.cu = cu;
    a.total = total;
    a.status = ctl.status;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return read ? launch_result(ffpa::launch_kv4_read(a, s), "4-bit cache read launch")
                : launch_result(ffpa::launch_kv4_write(a, s), "4-bit cache write launch");
}

ffpa_view packed_rows(void* p, int Hkv, int D) { return ffpa_view{p, 0, D, static_cast<int64_t>(Hkv) * D}; }

}  // namespace

extern "C" {

ffpa_status ffpa_kv4_write(ffpa_dtype dt, ffpa_view k, ffpa_view v, ffpa_kv4_cache cache, const int* start,
                           const int* count, int B, int Hkv, int N, int D, ffpa_stream_t stream)
{
    return run_kv4_io(false, dt, k, v, cache, start, count, nullptr, B, 0, Hkv, N, D, stream);
}

ffpa_status ffpa_kv4_read(ffpa_dtype dt, ffpa_kv4_cache cache, ffpa_view k, ffpa_view v, const int* start,
                          const int* count, int B, int Hkv, int N, int D, ffpa_stream_t stream)
{
    return run_kv4_io(true, dt, k, v, cache, start, count, nullptr, B, 0, Hkv, N, D, stream);
}

ffpa_status ffpa_varlen_kv4_write(ffpa_dtype dt, const void* k, const void* v, ffpa_kv4_cache cache,
                                  const int* cu_seqlens, const int* start, int batch, int total, int max_seqlen,
                                  int Hkv, int D, ffpa_stream_t stream)
{
    if (batch > 0 && !cu_seqlens) return fail(FFPA_ERR_INVALID_VALUE, "cu_seqlens is NULL");
    return run_kv4_io(false, dt, packed_rows(const_cast<void*>(k), Hkv, D), packed_rows(const_cast<void*>(v), Hkv, D),
                      cache, start, nullptr, cu_seqlens, batch, total, Hkv, max_seqlen, D, stream);
}

ffpa_status ffpa_varlen_kv4_read(ffpa_dtype dt, ffpa_kv4_cache cache, void* k, void* v, const int* cu_seqlens,
                                 const int* start, int batch, int total, int max_seqlen, int Hkv, int D,
                                 ffpa_stream_t stream)
{
    if (batch > 0 && !cu_seqlens) return fail(FFPA_ERR_INVALID_VALUE, "cu_seqlens is NULL");
    return run_kv4_io(true, dt, packed_rows(k, Hkv, D), packed_rows(v, Hkv, D), cache, start, nullptr, cu_seqlens,
                      batch, total, Hkv, max_seqlen, D, stream);
}

size_t ffpa_decode_kv4_workspace_bytes(ffpa_dtype, int B, int Hq, int Hkv, int Nq, int D)
{
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq <= 0 || Hq % Hkv != 0 || D < 64 || D > 1024 || D % 64 != 0) return 0;
    return ffpa::kv4_decode_workspace_bytes(dense_problem(B, Hq, Hkv, Nq, 0, D, 0, 1.f));
}

ffpa_status ffpa_decode_fwd_kv4(ffpa_dtype dt, ffpa_view q, ffpa_kv4_cache cache, const int* seq_lens, ffpa_view o,
                                float* lse, void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int Nq,
                                int D, int causal, float scale, ffpa_stream_t stream)
{
    FFPA_TRY(check_common(dt, Hq, Hkv, D, scale));
    FFPA_TRY(check_dense_sizes(B, Hq, Nq, 0));
    const long q_rows = static_cast<long>(B) * Hq * Nq;
    if (q_rows > INT_MAX) return fail(FFPA_ERR_NOT_SUPPORTED, "B*Hq*Nq=%ld exceeds 2^31 - 1 query rows", q_rows);
    ffpa::Kv4Decode a{};
    FFPA_TRY(check_kv4_cache(cache, q_rows > 0, Hkv, D, &a.cache));
    FFPA_TRY(check_view(q, q_rows > 0, "q", B, Hq, Nq));
    FFPA_TRY(check_view(o, q_rows > 0, "o", B, Hq, Nq));
    FFPA_TRY(check_ptr(lse, q_rows > 0, "lse"));
    if (q_rows > 0 && !seq_lens) return fail(FFPA_ERR_INVALID_VALUE, "seq_lens is NULL");
    if (reinterpret_cast<uintptr_t>(seq_lens) & 3u) return fail(FFPA_ERR_INVALID_VALUE, "seq_lens must be 4-byte aligned");
    if (q_rows == 0) return ok();
    ffpa::Problem pb = dense_problem(B, Hq, Hkv, Nq, 0, D, causal, scale);
    pb.vq = to_view(q);
    pb.vo = to_view(o);
    const size_t need = ffpa::kv4_decode_workspace_bytes(pb);
    if (workspace_bytes < need)
        return fail(FFPA_ERR_INVALID_VALUE, "decode workspace too small: %zu < %zu bytes", workspace_bytes, need);
    if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return fail(FFPA_ERR_INVALID_VALUE, "decode workspace must be non-NULL and 256-byte aligned");
    a.f.pb = pb;
    FFPA_TRY(device_ctl(&a.f.ctl));
    a.f.bf16 = dt == FFPA_BF16;
    a.f.q = q.data;
    a.f.o = o.data;
    a.f.lse = lse;
    a.seq_lens = seq_lens;
    return launch_result(ffpa::launch_decode_kv4(a, workspace, reinterpret_cast<cudaStream_t>(stream)),
                         "4-bit decode launch");
}

}  // extern "C"

// ------------------------------------------------ rotary positions, cache operators
namespace {

ffpa_status run_rope(ffpa_dtype dt, const ffpa_view& q, const ffpa_view& k, const ffpa_view& q_out,
                     const ffpa_view& k_out, const ffpa_rope_plan& plan, const int* start, const int* positions,
                     const int* cu, int B, int total, int Hq, int Hkv, int N, int D, int inverse, int zero_rest,
                     ffpa_stream_t stream)
{
    FFPA_TRY(check_common(dt, 0, 0, D, 1.f));
    if (B < 0 || N < 0 || total < 0 || Hq < 0 || Hkv < 0)
        return fail(FFPA_ERR_INVALID_VALUE, "negative size B=%d N=%d total=%d Hq=%d Hkv=%d", B, N, total, Hq, Hkv);
    if (plan.rot_dim < 16 || plan.rot_dim > D || plan.rot_dim % 16 != 0)
        return fail(FFPA_ERR_NOT_SUPPORTED, "rot_dim=%d must be a multiple of 16 in [16, D=%d]", plan.rot_dim, D);
    if (!std::isfinite(plan.mscale)) return fail(FFPA_ERR_INVALID_VALUE, "mscale must be finite");
    if (static_cast<long long>(Hq) + Hkv > INT_MAX / 64)
        return fail(FFPA_ERR_NOT_SUPPORTED, "Hq + Hkv = %lld heads exceed %d", static_cast<long long>(Hq) + Hkv, INT_MAX / 64);
    const long long tokens = cu ? total : static_cast<long long>(B) * N;
    if (tokens > INT_MAX) return fail(FFPA_ERR_NOT_SUPPORTED, "%lld tokens exceed 2^31 - 1", tokens);
    const bool any = tokens > 0 && (B > 0 || zero_rest) && Hq + Hkv > 0;
    if (any && !plan.turns) return fail(FFPA_ERR_INVALID_VALUE, "the plan's turns are NULL");
    if (reinterpret_cast<uintptr_t>(plan.turns) & 7u) return fail(FFPA_ERR_INVALID_VALUE, "turns must be 8-byte aligned");
    if ((reinterpret_cast<uintptr_t>(start) & 3u) || (reinterpret_cast<uintptr_t>(positions) & 3u) ||
        (reinterpret_cast<uintptr_t>(cu) & 3u))
        return fail(FFPA_ERR_INVALID_VALUE, "start, positions and cu_seqlens must be 4-byte aligned");
    if (start && positions) return fail(FFPA_ERR_INVALID_VALUE, "give start or positions, not both");
    const int eb = cu ? 1 : B, en = cu ? total : N;
    FFPA_TRY(check_view(q, any && Hq > 0, "q", eb, Hq, en));
    FFPA_TRY(check_view(q_out, any && Hq > 0, "q_out", eb, Hq, en));
    FFPA_TRY(check_view(k, any && Hkv > 0, "k", eb, Hkv, en));
    FFPA_TRY(check_view(k_out, any && Hkv > 0, "k_out", eb, Hkv, en));
    if (!any) return ok();
    ffpa::DeviceCtl ctl;
    FFPA_TRY(device_ctl(&ctl));
    ffpa::RopeArgs a{};
    a.bf16 = dt == FFPA_BF16;
    a.q = q.data;
    a.k = k.data;
    a.oq = q_out.data;
    a.ok = k_out.data;
    a.vq = to_view(q);
    a.vk = to_view(k);
    a.voq = to_view(q_out);
    a.vok = to_view(k_out);
    a.turns = reinterpret_cast<const unsigned long long*>(plan.turns);
    a.rot = plan.rot_dim;
    a.interleaved = plan.interleaved != 0;
    a.mscale = plan.mscale;
    a.sign = inverse ? -1.f : 1.f;
    a.zero_rest = zero_rest;
    a.start = start;
    a.pos = positions;
    a.cu = cu;
    a.B = B;
    a.Hq = Hq;
    a.Hk = Hkv;
    a.N = N;
    a.total = total;
    a.D = D;
    return launch_result(ffpa::launch_rope(a, reinterpret_cast<cudaStream_t>(stream)), "rotary launch");
}

// What the two decode forms over caches of different lengths have in common.
ffpa_status check_line(ffpa_dtype dt, const ffpa_view& q, const ffpa_view& k, const ffpa_view& v, const int* lens,
                       const ffpa_view& o, const float* lse, int B, int Hq, int Hkv, int Nq, int N, int D, int causal,
                       float scale, bool shared, int Np, ffpa::LineArgs* a)
{
    FFPA_TRY(check_common(dt, Hq, Hkv, D, scale));
    FFPA_TRY(check_dense_sizes(B, Hq, Nq, N));
    if (D % 64 != 0) return fail(FFPA_ERR_NOT_SUPPORTED, "decode path: D=%d must be a multiple of 64", D);
    if (Np < 0) return fail(FFPA_ERR_INVALID_VALUE, "negative prefix length %d", Np);
    if (static_cast<long long>(Np) + N > ffpa::kMaxTokens)
        return fail(FFPA_ERR_NOT_SUPPORTED, "prefix and cache hold %lld keys, above %d", static_cast<long long>(Np) + N,
                    ffpa::kMaxTokens);
    const long q_rows = static_cast<long>(B) * Hq * Nq;
    a->f.pb = dense_problem(B, Hq, Hkv, Nq, N, D, causal, scale);
    if (q_rows > 0 && !ffpa::line_fits(a->f.pb, shared, Np))
        return fail(FFPA_ERR_NOT_SUPPORTED, "B*Hq*Nq=%ld rows over N=%d keys exceed the launch's units", q_rows, N);
    FFPA_TRY(check_view(q, q_rows > 0, "q", B, Hq, Nq));
    FFPA_TRY(check_view(o, q_rows > 0, "o", B, Hq, Nq));
    FFPA_TRY(check_view(k, q_rows > 0 && N > 0, "k", B, Hkv, N));
    FFPA_TRY(check_view(v, q_rows > 0 && N > 0, "v", B, Hkv, N));
    FFPA_TRY(check_ptr(lse, q_rows > 0, "lse"));
    if (reinterpret_cast<uintptr_t>(lens) & 3u) return fail(FFPA_ERR_INVALID_VALUE, "lens must be 4-byte aligned");
    a->f.pb.vq = to_view(q);
    a->f.pb.vo = to_view(o);
    a->f.pb.vk = to_view(k);
    a->f.pb.vv = to_view(v);
    a->f.bf16 = dt == FFPA_BF16;
    a->f.q = q.data;
    a->f.k = k.data;
    a->f.v = v.data;
    a->f.o = o.data;
    a->f.lse = const_cast<float*>(lse);
    a->lens = lens;
    a->shared = shared;
    a->Np = Np;
    return FFPA_OK;
}

ffpa_status run_line(ffpa::LineArgs& a, void* workspace, size_t workspace_bytes, ffpa_stream_t stream)
{
    if (workspace_bytes > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return fail(FFPA_ERR_INVALID_VALUE, "decode workspace must be non-NULL and 256-byte aligned");
    ffpa_status st = device_ctl(&a.f.ctl);
    size_t need = 0;
    cudaError_t e = cudaSuccess;
    if (st == FFPA_OK)
        e = ffpa::launch_line(a, workspace, workspace_bytes, &need, reinterpret_cast<cudaStream_t>(stream));
    else
        need = ffpa::line_workspace_bytes(a.f.pb, a.shared, a.Np);
    if (workspace_bytes < need)
        return fail(FFPA_ERR_INVALID_VALUE, "decode workspace too small: %zu < %zu bytes", workspace_bytes, need);
    return st == FFPA_OK ? launch_result(e, "decode launch") : st;
}

// Workspace queries answer 0 for sizes outside the operation.
bool line_sizes_ok(ffpa_dtype dt, int B, int Hq, int Hkv, int Nq, int N, int D, int Np)
{
    return (dt == FFPA_BF16 || dt == FFPA_FP16) && B > 0 && Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && Nq > 0 && N >= 0 &&
           Np >= 0 && static_cast<long long>(Np) + N <= ffpa::kMaxTokens && D >= 64 && D <= 1024 && D % 64 == 0;
}

}  // namespace

extern "C" {

ffpa_status ffpa_rope(ffpa_dtype dt, ffpa_view q, ffpa_view k, ffpa_view q_out, ffpa_view k_out, ffpa_rope_plan plan,
                      const int* start, const int* positions, int B, int Hq, int Hkv, int N, int D, int inverse,
                      ffpa_stream_t stream)
{
    return run_rope(dt, q, k, q_out, k_out, plan, start, positions, nullptr, B, 0, Hq, Hkv, N, D, inverse, 0, stream);
}

ffpa_status ffpa_varlen_rope(ffpa_dtype dt, const void* q, const void* k, void* q_out, void* k_out,
                             ffpa_rope_plan plan, const int* cu_seqlens, const int* start, const int* positions,
                             int batch, int total, int Hq, int Hkv, int D, int flags, ffpa_stream_t stream)
{
    if (!cu_seqlens) return fail(FFPA_ERR_INVALID_VALUE, "cu_seqlens is NULL");
    if (flags & ~(FFPA_ROPE_INVERSE | FFPA_ROPE_ZERO_REST))
        return fail(FFPA_ERR_INVALID_VALUE, "flags=%d: FFPA_ROPE_INVERSE and FFPA_ROPE_ZERO_REST are known", flags);
    const int hq = Hq > 0 ? Hq : 1, hk = Hkv > 0 ? Hkv : 1;
    return run_rope(dt, packed_rows(const_cast<void*>(q), hq, D), packed_rows(const_cast<void*>(k), hk, D),
                    packed_rows(q_out, hq, D), packed_rows(k_out, hk, D), plan, start, positions, cu_seqlens, batch,
                    total, Hq, Hkv, total, D, flags & FFPA_ROPE_INVERSE, flags & FFPA_ROPE_ZERO_REST, stream);
}

size_t ffpa_decode_shared_workspace_bytes(ffpa_dtype dt, int B, int Hq, int Hkv, int Nq, int Np, int N, int D)
{
    if (!line_sizes_ok(dt, B, Hq, Hkv, Nq, N, D, Np)) return 0;
    const ffpa::Problem pb = dense_problem(B, Hq, Hkv, Nq, N, D, 0, 1.f);
    return ffpa::line_fits(pb, true, Np) ? ffpa::line_workspace_bytes(pb, true, Np) : 0;
}

ffpa_status ffpa_decode_fwd_shared(ffpa_dtype dt, ffpa_view q, ffpa_view k_prefix, ffpa_view v_prefix, ffpa_view k,
                                   ffpa_view v, const int* lens, ffpa_view o, float* lse, void* workspace,
                                   size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int Np, int N, int D,
                                   int causal, float scale, ffpa_stream_t stream)
{
    ffpa::LineArgs a{};
    FFPA_TRY(check_line(dt, q, k, v, lens, o, lse, B, Hq, Hkv, Nq, N, D, causal, scale, true, Np, &a));
    const long q_rows = static_cast<long>(B) * Hq * Nq;
    FFPA_TRY(check_view(k_prefix, q_rows > 0 && Np > 0, "k_prefix", 1, Hkv, Np));
    FFPA_TRY(check_view(v_prefix, q_rows > 0 && Np > 0, "v_prefix", 1, Hkv, Np));
    if (q_rows == 0) return ok();
    a.kp = k_prefix.data;
    a.vp = v_prefix.data;
    a.vkp = to_view(k_prefix);
    a.vvp = to_view(v_prefix);
    return run_line(a, workspace, workspace_bytes, stream);
}

size_t ffpa_decode_weights_workspace_bytes(ffpa_dtype dt, int B, int Hq, int Hkv, int Nq, int N, int D)
{
    if (!line_sizes_ok(dt, B, Hq, Hkv, Nq, N, D, 0)) return 0;
    const ffpa::Problem pb = dense_problem(B, Hq, Hkv, Nq, N, D, 0, 1.f);
    return ffpa::line_fits(pb, false, 0) ? ffpa::line_workspace_bytes(pb, false, 0) : 0;
}

ffpa_status ffpa_decode_fwd_weights(ffpa_dtype dt, ffpa_view q, ffpa_view k, ffpa_view v, const int* lens,
                                    const float* weights, float* weights_out, ffpa_view o, float* lse,
                                    void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int N,
                                    int D, int causal, float scale, ffpa_stream_t stream)
{
    ffpa::LineArgs a{};
    FFPA_TRY(check_line(dt, q, k, v, lens, o, lse, B, Hq, Hkv, Nq, N, D, causal, scale, false, 0, &a));
    const long q_rows = static_cast<long>(B) * Hq * Nq;
    FFPA_TRY(check_ptr(weights, q_rows > 0 && N > 0, "weights"));
    FFPA_TRY(check_ptr(weights_out, q_rows > 0 && N > 0, "weights_out"));
    if (q_rows == 0) return ok();
    a.weights = weights;
    a.oweights = weights_out;
    return run_line(a, workspace, workspace_bytes, stream);
}

ffpa_status ffpa_kv_evict(ffpa_dtype dt, ffpa_view k, ffpa_view v, const float* weights, const int* lens,
                          ffpa_view k_out, ffpa_view v_out, float* weights_out, int* lens_out, int* kept, int B,
                          int Hkv, int N, int N_out, int D, int keep, int recent, ffpa_stream_t stream)
{
    FFPA_TRY(check_common(dt, Hkv, Hkv, D, 1.f));
    if (B < 0 || N < 0 || N_out < 0) return fail(FFPA_ERR_INVALID_VALUE, "negative size B=%d N=%d N_out=%d", B, N, N_out);
    if (keep < 1 || recent < 0 || recent > keep)
        return fail(FFPA_ERR_INVALID_VALUE, "keep=%d must be positive and recent=%d in [0, keep]", keep, recent);
    if (N > ffpa::kMaxTokens || keep > ffpa::kMaxTokens)
        return fail(FFPA_ERR_NOT_SUPPORTED, "N=%d and keep=%d are limited to %d tokens", N, keep, ffpa::kMaxTokens);
    if (N_out < (keep < N ? keep : N))
        return fail(FFPA_ERR_INVALID_VALUE, "N_out=%d does not hold min(keep=%d, N=%d) tokens", N_out, keep, N);
    if (static_cast<long long>(B) * Hkv > INT_MAX / 2)
        return fail(FFPA_ERR_NOT_SUPPORTED, "B*Hkv=%lld exceeds %d", static_cast<long long>(B) * Hkv, INT_MAX / 2);
    const bool any = B > 0 && Hkv > 0;
    FFPA_TRY(check_view(k, any && N > 0, "k", B, Hkv, N));
    FFPA_TRY(check_view(v, any && N > 0, "v", B, Hkv, N));
    FFPA_TRY(check_view(k_out, any && N > 0, "k_out", B, Hkv, N_out));
    FFPA_TRY(check_view(v_out, any && N > 0, "v_out", B, Hkv, N_out));
    FFPA_TRY(check_ptr(weights, any && N > 0, "weights"));
    FFPA_TRY(check_ptr(weights_out, any && N > 0, "weights_out"));
    const void* ints[3] = {lens, lens_out, kept};
    const char* names[3] = {"lens", "lens_out", "kept"};
    for (int i = 0; i < 3; ++i) {
        if (any && !ints[i]) return fail(FFPA_ERR_INVALID_VALUE, "%s is NULL", names[i]);
        if (reinterpret_cast<uintptr_t>(ints[i]) & 3u)
            return fail(FFPA_ERR_INVALID_VALUE, "%s must be 4-byte aligned", names[i]);
    }
    auto same = [](const ffpa_view& x, const ffpa_view& y) {
        return x.data == y.data && x.stride_b == y.stride_b && x.stride_h == y.stride_h && x.stride_n == y.stride_n;
    };
    // in place is all of it in place: one tensor over another's storage would be read while it is written
    const bool in_place = k.data == k_out.data;
    if (any && N > 0) {
        if (in_place != (v.data == v_out.data) || in_place != (weights == weights_out) || k.data == v_out.data ||
            v.data == k_out.data)
            return fail(FFPA_ERR_INVALID_VALUE, "k, v and weights are cut all in place or all into other tensors");
        if (in_place && (!same(k, k_out) || !same(v, v_out) || N != N_out))
            return fail(FFPA_ERR_INVALID_VALUE, "in place, the outputs must be the inputs' own views");
    }
    if (!any) return ok();
    ffpa::DeviceCtl ctl;
    FFPA_TRY(device_ctl(&ctl));
    ffpa::EvictArgs a{};
    a.k = k.data;
    a.v = v.data;
    a.ok = k_out.data;
    a.ov = v_out.data;
    a.vk = to_view(k);
    a.vv = to_view(v);
    a.vok = to_view(k_out);
    a.vov = to_view(v_out);
    a.weights = weights;
    a.oweights = weights_out;
    a.lens = lens;
    a.olens = lens_out;
    a.kept = kept;
    a.B = B;
    a.Hkv = Hkv;
    a.N = N;
    a.Nout = N_out;
    a.D = D;
    a.keep = keep;
    a.recent = recent;
    a.in_place = in_place;
    a.status = ctl.status;
    return launch_result(ffpa::launch_evict(a, reinterpret_cast<cudaStream_t>(stream)), "eviction launch");
}

size_t ffpa_bwd_workspace_bytes_ds(ffpa_dtype dt, int B, int Hq, int Hkv, int Nq, int Nkv, int D, int causal)
{
    const size_t small = ffpa_bwd_workspace_bytes(dt, B, Hq, Hkv, Nq, Nkv, D);
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq <= 0 || Nkv <= 0 || Hq % Hkv != 0) return small;
    const ffpa::Problem pb = dense_problem(B, Hq, Hkv, Nq, Nkv, D, causal, 1.f);
    // dS^T, then P^T at the next 256-byte boundary
    return ffpa::dsq_supported(pb) ? small + align256(ffpa::dsq_ds_bytes(pb)) + ffpa::dsq_ds_bytes(pb) : small;
}

size_t ffpa_bwd_workspace_bytes_budget(ffpa_dtype dt, int B, int Hq, int Hkv, int Nq, int Nkv, int D, int causal,
                                       size_t budget)
{
    const size_t small = ffpa_bwd_workspace_bytes(dt, B, Hq, Hkv, Nq, Nkv, D);
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq <= 0 || Nkv <= 0 || Hq % Hkv != 0) return small;
    return budget_bytes(dense_problem(B, Hq, Hkv, Nq, Nkv, D, causal, 1.f), small, budget);
}

size_t ffpa_bwd_workspace_bytes(ffpa_dtype, int B, int Hq, int, int Nq, int, int)
{
    if (B < 0 || Hq < 0 || Nq < 0) return 0;
    return ws_bytes(static_cast<long>(B) * Hq * Nq);
}

ffpa_status ffpa_bwd(ffpa_dtype dt, const void* q, const void* k, const void* v, const void* o, const float* lse,
                     const void* dO, void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int B,
                     int Hq, int Hkv, int Nq, int Nkv, int D, int causal, float scale, ffpa_stream_t stream)
{
    FFPA_TRY(check_common(dt, Hq, Hkv, D, scale));
    FFPA_TRY(check_dense_sizes(B, Hq, Nq, Nkv));
    const long q_rows = static_cast<long>(B) * Hq * Nq;
    const long k_rows = static_cast<long>(B) * Hkv * Nkv;
    return run_bwd(dt, q, k, v, o, lse, dO, dq, dk, dv, workspace, workspace_bytes,
                   dense_problem(B, Hq, Hkv, Nq, Nkv, D, causal, scale), q_rows, k_rows, q_rows, 15u, stream);
}

ffpa_status ffpa_bwd_strided(ffpa_dtype dt, ffpa_view q, ffpa_view k, ffpa_view v, ffpa_view o, const float* lse,
                             ffpa_view dO, ffpa_view dq, ffpa_view dk, ffpa_view dv, void* workspace,
                             size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int Nkv, int D, int causal,
                             float scale, ffpa_stream_t stream)
{
    FFPA_TRY(check_common(dt, Hq, Hkv, D, scale));
    FFPA_TRY(check_dense_sizes(B, Hq, Nq, Nkv));
    const long q_rows = static_cast<long>(B) * Hq * Nq;
    const long k_rows = static_cast<long>(B) * Hkv * Nkv;
    FFPA_TRY(check_view(q, q_rows > 0, "q", B, Hq, Nq));
    FFPA_TRY(check_view(o, q_rows > 0, "o", B, Hq, Nq));
    FFPA_TRY(check_view(dO, q_rows > 0, "dO", B, Hq, Nq));
    FFPA_TRY(check_view(dq, q_rows > 0, "dq", B, Hq, Nq));
    FFPA_TRY(check_view(k, k_rows > 0, "k", B, Hkv, Nkv));
    FFPA_TRY(check_view(v, k_rows > 0, "v", B, Hkv, Nkv));
    FFPA_TRY(check_view(dk, k_rows > 0, "dk", B, Hkv, Nkv));
    FFPA_TRY(check_view(dv, k_rows > 0, "dv", B, Hkv, Nkv));
    ffpa::Problem pb = dense_problem(B, Hq, Hkv, Nq, Nkv, D, causal, scale);
    pb.vq = to_view(q);
    pb.vo = to_view(o);
    pb.vdo = to_view(dO);
    pb.vdq = to_view(dq);
    pb.vk = to_view(k);
    pb.vv = to_view(v);
    pb.vdk = to_view(dk);
    pb.vdv = to_view(dv);
    return run_bwd(dt, q.data, k.data, v.data, o.data, lse, dO.data, dq.data, dk.data, dv.data, workspace,
                   workspace_bytes, pb, q_rows, k_rows, q_rows, 15u, stream);
}

ffpa_status ffpa_bwd_stages(ffpa_dtype dt, const void* q, const void* k, const void* v, const void* o,
                            const float* lse, const void* dO, void* dq, void* dk, void* dv, void* workspace,
                            size_t workspace_bytes, int B, int Hq, int Hkv, int Nq, int Nkv, int D, int causal,
                            float scale, unsigned stages, ffpa_stream_t stream)
{
    FFPA_TRY(check_common(dt, Hq, Hkv, D, scale));
    FFPA_TRY(check_dense_sizes(B, Hq, Nq, Nkv));
    if (stages > 63u) return fail(FFPA_ERR_INVALID_VALUE, "stages mask %u: only bits 0..5", stages);
    const long q_rows = static_cast<long>(B) * Hq * Nq;
    const long k_rows = static_cast<long>(B) * Hkv * Nkv;
    return run_bwd(dt, q, k, v, o, lse, dO, dq, dk, dv, workspace, workspace_bytes,
                   dense_problem(B, Hq, Hkv, Nq, Nkv, D, causal, scale), q_rows, k_rows, q_rows, stages, stream);
}

ffpa_status ffpa_varlen_fwd(ffpa_dtype dt, const void* q, const void* k, const void* v, void* o, float* lse,
                            const int* cu_seqlens_q, const int* cu_seqlens_k, int batch, int total_q, int total_k,
                            int max_seqlen_q, int max_seqlen_k, int Hq, int Hkv, int D, int causal, float scale,
                            ffpa_stream_t stream)
{
    FFPA_TRY(check_common(dt, Hq, Hkv, D, scale));
    FFPA_TRY(check_varlen_sizes(batch, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, cu_seqlens_q, cu_seqlens_k));
    const long q_rows = batch > 0 ? static_cast<long>(total_q) * Hq : 0;
    const long k_rows = batch > 0 ? static_cast<long>(total_k) * Hkv : 0;
    return run_fwd(dt, q, k, v, o, lse,
                   varlen_problem(batch, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, D, causal, scale,
                                  cu_seqlens_q, cu_seqlens_k),
                   q_rows, k_rows, stream);
}

size_t ffpa_varlen_bwd_workspace_bytes(ffpa_dtype, int batch, int total_q, int, int, int, int Hq, int, int)
{
    if (batch <= 0 || total_q < 0 || Hq < 0) return 0;
    return ws_bytes(static_cast<long>(total_q) * Hq);
}

size_t ffpa_varlen_bwd_workspace_bytes_ds(ffpa_dtype dt, int batch, int total_q, int total_k, int max_seqlen_q,
                                          int max_seqlen_k, int Hq, int Hkv, int D, int causal)
{
    const size_t small =
        ffpa_varlen_bwd_workspace_bytes(dt, batch, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, D);
    if (batch <= 0 || total_q <= 0 || total_k <= 0 || max_seqlen_q <= 0 || max_seqlen_k <= 0 || Hq <= 0 ||
        Hkv <= 0 || Hq % Hkv != 0)
        return small;
    const ffpa::Problem pb = varlen_problem(batch, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, D, causal,
                                            1.f, nullptr, nullptr);
    // dS^T, then P^T at the next 256-byte boundary
    return ffpa::dsq_supported(pb) ? small + align256(ffpa::dsq_ds_bytes(pb)) + ffpa::dsq_ds_bytes(pb) : small;
}

size_t ffpa_varlen_bwd_workspace_bytes_budget(ffpa_dtype dt, int batch, int total_q, int total_k, int max_seqlen_q,
                                              int max_seqlen_k, int Hq, int Hkv, int D, int causal, size_t budget)
{
    const size_t small =
        ffpa_varlen_bwd_workspace_bytes(dt, batch, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, D);
    if (batch <= 0 || total_q <= 0 || total_k <= 0 || max_seqlen_q <= 0 || max_seqlen_k <= 0 || Hq <= 0 ||
        Hkv <= 0 || Hq % Hkv != 0)
        return small;
    return budget_bytes(varlen_problem(batch, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, D, causal, 1.f,
                                       nullptr, nullptr),
                        small, budget);
}

ffpa_status ffpa_varlen_bwd(ffpa_dtype dt, const void* q, const void* k, const void* v, const void* o,
                            const float* lse, const void* dO, void* dq, void* dk, void* dv, const int* cu_seqlens_q,
                            const int* cu_seqlens_k, int batch, int total_q, int total_k, int max_seqlen_q,
                            int max_seqlen_k, int Hq, int Hkv, int D, int causal, float scale, void* workspace,
                            size_t workspace_bytes, ffpa_stream_t stream)
{
    FFPA_TRY(check_common(dt, Hq, Hkv, D, scale));
    FFPA_TRY(check_varlen_sizes(batch, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, cu_seqlens_q, cu_seqlens_k));
    const long q_rows = batch > 0 ? static_cast<long>(total_q) * Hq : 0;
    const long k_rows = batch > 0 ? static_cast<long>(total_k) * Hkv : 0;
    return run_bwd(dt, q, k, v, o, lse, dO, dq, dk, dv, workspace, workspace_bytes,
                   varlen_problem(batch, total_q, total_k, max_seqlen_q, max_seqlen_k, Hq, Hkv, D, causal, scale,
                                  cu_seqlens_q, cu_seqlens_k),
                   q_rows, k_rows, q_rows, 15u, stream);
}

ffpa_status ffpa_get_status(ffpa_stream_t stream)
{
    cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(FFPA_ERR_CUDA, "stream error: %s", cudaGetErrorString(e));
    uint32_t word = 0;
    e = cudaMemcpyFromSymbol(&word, g_ffpa_status_word, sizeof(word));
    if (e != cudaSuccess) return fail(FFPA_ERR_CUDA, "reading the status word: %s", cudaGetErrorString(e));
    if (word == 0) return ok();
    const uint32_t zero = 0;
    cudaMemcpyToSymbol(g_ffpa_status_word, &zero, sizeof(zero));
    if ((word & 0xffu) == ffpa::DEV_TIMEOUT)
        return fail(FFPA_ERR_TIMEOUT, "a device wait timed out (site %u, block %u)", (word >> 8) & 0xffu, word >> 16);
    const uint32_t site = (word >> 8) & 0xffu;
    if ((word & 0xffu) == ffpa::DEV_INVALID && site >= ffpa::VS_KV4_WRITE && site <= ffpa::VS_KV4_DECODE)
        return fail(FFPA_ERR_INVALID_VALUE,
                    "4-bit cache: sequence %u breaks the contract of its lengths and block table (a negative length or "
                    "start, tokens past max_blocks * page_size or past the tensor's rows, or a page outside "
                    "[0, num_pages)); the outputs of that call are undefined for it (site 0x%02x)",
                    word >> 16, site);
    if ((word & 0xffu) == ffpa::DEV_INVALID && (site == ffpa::VS_LINE || site == ffpa::VS_EVICT))
        return fail(FFPA_ERR_INVALID_VALUE,
                    "cache: the length of sequence %u is negative or above the tokens that its cache holds; the outputs "
                    "of that call are undefined (site 0x%02x)",
                    word >> 16, site);
    if ((word & 0xffu) == ffpa::DEV_INVALID)
        return fail(FFPA_ERR_INVALID_VALUE,
                    "packed sequence %u breaks the varlen contract: its cu_seqlens entries are negative, decrease or "
                    "run past total_q / total_k, or its length exceeds max_seqlen_q / max_seqlen_k (which size the "
                    "launch); the outputs of that call are undefined (site 0x%02x)",
                    word >> 16, (word >> 8) & 0xffu);
    return fail(FFPA_ERR_CUDA, "device status word 0x%08x", word);
}

const char* ffpa_last_error(void) { return g_err.c_str(); }

void ffpa_set_wait_limit_ns(uint64_t ns) { g_limit_ns.store(ns ? ns : 2000000000ull); }

ffpa_status ffpa_selftest_wait_timeout(uint64_t limit_ns, ffpa_stream_t stream)
{
    bool cc_ok = false;
    uint32_t* st = nullptr;
    if (!device_state(&st, &cc_ok)) return fail(FFPA_ERR_CUDA, "no usable CUDA device");
    selftest_wait_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(st, limit_ns);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(FFPA_ERR_CUDA, "self-test launch: %s", cudaGetErrorString(e));
    return ffpa_get_status(stream);
}

int ffpa_num_sms(void) { return ffpa::num_sms(); }

}  // extern "C"
