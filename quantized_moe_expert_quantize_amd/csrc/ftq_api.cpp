// The C entry points of libftq: argument validation, path choice, workspace
// planning and dispatch.  No allocation, no synchronisation, no readback.
#include <cstdarg>
#include <mutex>

#include "ftq_internal.h"

namespace ftq {

namespace {
thread_local std::string g_error;
thread_local int g_forced_threads = 0;
thread_local int g_grouped_variant = kGroupedI8;

constexpr int kMaxDevices = 64;
std::mutex g_lim_mu;
DeviceLimits g_lim[kMaxDevices];

constexpr int64_t kMaxExperts = 4095;      // bucket tables live in LDS
constexpr int64_t kMaxPairs = INT32_MAX;   // pair ids are stored as int32

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
}  // namespace

void set_error(const char* fmt, ...)
{
    char buf[1024];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_error = buf;
}

void clear_error() { g_error.clear(); }

int forced_block_threads() { return g_forced_threads; }

int grouped_kernel_variant() { return g_grouped_variant; }
thread_local int g_route_split = 0;
int route_split_forced() { return g_route_split; }

int device_limits(DeviceLimits* out)
{
    int dev = -1;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess || dev < 0 || dev >= kMaxDevices) {
        set_error("hipGetDevice failed: %s", hipGetErrorString(err));
        return FTQ_ERR_HIP;
    }
    std::lock_guard<std::mutex> lock(g_lim_mu);
    DeviceLimits& l = g_lim[dev];
    if (l.device != dev) {
        int gx = 0, thr = 0, lds = 0, cus = 0;
        if (hipDeviceGetAttribute(&gx, hipDeviceAttributeMaxGridDimX, dev) != hipSuccess ||
            hipDeviceGetAttribute(&thr, hipDeviceAttributeMaxThreadsPerBlock, dev) != hipSuccess ||
            hipDeviceGetAttribute(&lds, hipDeviceAttributeMaxSharedMemoryPerBlock, dev) != hipSuccess ||
            hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) {
            set_error("hipDeviceGetAttribute failed on device %d", dev);
            return FTQ_ERR_HIP;
        }
        l.max_grid_x = gx;
        l.max_threads = thr;
        l.max_lds = lds;
        l.cu_count = cus;
        l.device = dev;
    }
    *out = l;
    return FTQ_OK;
}

int64_t stride_grid(int64_t needed, const DeviceLimits& lim, int per_cu)
{
    const int64_t cap = (int64_t)std::max(lim.cu_count, 1) * per_cu;
    return std::max<int64_t>(1, std::min(needed, std::min(cap, lim.max_grid_x)));
}

namespace {

int check_sizes(int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k)
{
    if (K <= 0 || K % kQK != 0) { set_error("K must be a positive multiple of 32 (got %lld)", (long long)K); return FTQ_ERR_INVALID_ARG; }
    if (E < 1 || N < 1 || top_k < 1 || T < 0) {
        set_error("need E >= 1, N >= 1, top_k >= 1, T >= 0 (got E=%lld N=%lld top_k=%lld T=%lld)",
                  (long long)E, (long long)N, (long long)top_k, (long long)T);
        return FTQ_ERR_INVALID_ARG;
    }
    if (top_k > E) { set_error("top_k (%lld) exceeds the number of experts (%lld)", (long long)top_k, (long long)E); return FTQ_ERR_INVALID_ARG; }
    if (T > kMaxPairs / top_k) {
        set_error("T*top_k = %lld*%lld exceeds the 2^31-1 pair limit", (long long)T, (long long)top_k);
        return FTQ_ERR_UNSUPPORTED;
    }
    if (E > kMaxExperts) { set_error("E = %lld exceeds the supported %lld experts", (long long)E, (long long)kMaxExperts); return FTQ_ERR_UNSUPPORTED; }
    // every byte offset must fit int64: E*N*(K/32)*18 and T*top_k*N*4
    const int64_t nb = K / kQK;
    if (N > INT64_MAX / 64 / E / nb || (T * top_k) > INT64_MAX / 64 / N) {
        set_error("tensor sizes overflow 64-bit byte offsets");
        return FTQ_ERR_UNSUPPORTED;
    }
    return FTQ_OK;
}

int select_path(int64_t E, int64_t T, int64_t top_k)
{
    const int64_t pairs = T * top_k;
    // few pairs per expert: stream each expert's rows once and serve its pairs
    // on the vector ALUs; otherwise sorted MFMA tiles.  The crossover, measured
    // on one MI355X: about 7 pairs per expert with 8 experts (14336 x 4096
    // rows), about 4 with 128 (1408 x 2816).
    const int64_t per_expert_x2 = E <= 16 ? 14 : 8;   // twice the pairs per expert
    if (pairs <= kGemvScanMaxPairs && 2 * pairs <= per_expert_x2 * E) return FTQ_PATH_GEMV;
    return FTQ_PATH_GROUPED;
}

int64_t tile_m_for(int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k)
{
    MoeArgs m{};
    m.E = E; m.N = N; m.K = K; m.T = T; m.top_k = top_k; m.wtype = FTQ_W_Q4_0;
    return grouped_tile_m(m);
}

// Workspace plan for a resolved path; `bucketed` tells whether the plan is used.
BucketPlan plan_for(int path, int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, bool* bucketed)
{
    const int64_t pairs = T * top_k;
    if (path == FTQ_PATH_GEMV && pairs <= kGemvScanMaxPairs) {
        *bucketed = false;
        return BucketPlan{};
    }
    *bucketed = true;
    const int64_t tm = path == FTQ_PATH_GROUPED ? tile_m_for(E, N, K, T, top_k) : 0;
    return make_bucket_plan(pairs, E, tm);
}

int resolve_path(int path, int64_t E, int64_t T, int64_t top_k)
{
    if (path == FTQ_PATH_AUTO) return select_path(E, T, top_k);
    if (path == FTQ_PATH_GEMV || path == FTQ_PATH_GROUPED) return path;
    return -1;
}

int check_workspace(int64_t need, const void* ws, size_t ws_bytes)
{
    if (!ws || (int64_t)ws_bytes < need) {
        set_error("workspace of %zu bytes is smaller than the %lld bytes needed", ws_bytes, (long long)need);
        return FTQ_ERR_WORKSPACE;
    }
    if (!aligned(ws, 256)) { set_error("workspace must be 256-byte aligned"); return FTQ_ERR_INVALID_ARG; }
    return FTQ_OK;
}

// kRoute: bucketing only; kMatmul: matmul only (pairs already routed); both: the full call.
enum Phase { kRoute = 1, kMatmul = 2 };

// act_per_pair: `a` holds one Q8_1 row per pair ([T*top_k][K/32]) instead of
// one per token ([T][K/32]).

int moe_common(const void* w, const void* a, const int32_t* ids, float* out, int32_t* partials,
               int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, void* ws, size_t ws_bytes,
               int path, hipStream_t stream, int phases, bool act_per_pair = false, int act = 0,
               int wtype = FTQ_W_Q4_0)
{
    clear_error();
    int st = check_sizes(E, N, K, T, top_k);
    if (st != FTQ_OK) return st;
    if (wtype != FTQ_W_Q4_0 && wtype != FTQ_W_Q4_1 && wtype != FTQ_W_Q5_0 && wtype != FTQ_W_Q5_1 && wtype != FTQ_W_Q8_0) {
        set_error("unknown weight type %d", wtype);
        return FTQ_ERR_INVALID_ARG;
    }
    if (wtype == FTQ_W_Q5_0 || wtype == FTQ_W_Q5_1) {
        // the five-bit types run on the GEMV path only
        if (path == FTQ_PATH_GROUPED) {
            set_error("weight type %d: the grouped path takes Q4_0, Q4_1 and Q8_0; use FTQ_PATH_GEMV or FTQ_PATH_AUTO", wtype);
            return FTQ_ERR_UNSUPPORTED;
        }
        if (path == FTQ_PATH_AUTO) path = FTQ_PATH_GEMV;
    }
    if (act != 0) {
        if (act != FTQ_ACT_SILU && act != FTQ_ACT_GELU_TANH) { set_error("unknown activation %d", act); return FTQ_ERR_INVALID_ARG; }
        if (N % 2 != 0) { set_error("a gated activation needs an even N (gate and up halves), got %lld", (long long)N); return FTQ_ERR_INVALID_ARG; }
    }
    const int rp = resolve_path(path, E, T, top_k);
    if (rp < 0) { set_error("unknown path %d", path); return FTQ_ERR_INVALID_ARG; }
    if (T == 0) return FTQ_OK;
    if (!ids || ((phases & kMatmul) && (!w || !a || (!out && !partials)))) {
        set_error("null pointer argument (w, a, topk_ids or the output)");
        return FTQ_ERR_INVALID_ARG;
    }
    if (!aligned(ids, 4) || ((phases & kMatmul) &&
        (!aligned(w, 2) || !aligned(a, 4) || !aligned(out ? (const void*)out : (const void*)partials, 4)))) {
        set_error("misaligned pointer (w needs 2-byte, a/topk_ids/out 4-byte alignment)");
        return FTQ_ERR_INVALID_ARG;
    }
    bool bucketed = false;
    const BucketPlan plan = plan_for(rp, E, N, K, T, top_k, &bucketed);
    if (bucketed) {
        // the workspace holds the bucket tables (both paths read the activations in place)
        st = check_workspace(plan.bytes, ws, ws_bytes);
        if (st != FTQ_OK) return st;
        if (phases & kRoute) {
            st = run_bucket(ids, E, plan, ws, stream);
            if (st != FTQ_OK) return st;
        }
    }
    if (!(phases & kMatmul)) return FTQ_OK;
    MoeArgs m{w, a, ids, out, partials, E, N, K, T, top_k, act_per_pair ? 1 : top_k, act, wtype};
    if (rp == FTQ_PATH_GEMV) return run_gemv(m, bucketed ? &plan : nullptr, ws, stream);
    return run_grouped(m, plan, ws, stream);
}

int64_t workspace_bytes(int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int path, bool act_per_pair)
{
    (void)act_per_pair;   // the workspace does not depend on how the activations are laid out
    clear_error();
    if (check_sizes(E, N, K, T, top_k) != FTQ_OK) return -1;
    const int rp = resolve_path(path, E, T, top_k);
    if (rp < 0) { set_error("unknown path %d", path); return -1; }
    if (T == 0) return 0;
    bool bucketed = false;
    const BucketPlan plan = plan_for(rp, E, N, K, T, top_k, &bucketed);
    if (!bucketed) return 0;
    return plan.bytes;
}

int64_t dtype_bytes(int dtype) { return dtype == FTQ_F32 ? 4 : (dtype == FTQ_F16 || dtype == FTQ_BF16) ? 2 : 0; }

// A [rows][K] array of `dtype` for the 8-bit floating-point quantisers: whole
// 16-byte runs of codes per row, offsets that fit int64.
int check_quantize_fp8(int dtype, int64_t rows, int64_t K, int64_t ld)
{
    if (!dtype_bytes(dtype)) { set_error("unknown element type %d", dtype); return FTQ_ERR_INVALID_ARG; }
    if (K <= 0 || K % 16 != 0) { set_error("K must be a positive multiple of 16 (got %lld)", (long long)K); return FTQ_ERR_INVALID_ARG; }
    if (rows < 0 || ld < K || ld > INT64_MAX / 16 || (ld * dtype_bytes(dtype)) % 16 != 0) {
        set_error("need rows >= 0 and a row stride of at least K elements and whole 16-byte units (got %lld rows, stride %lld)",
                  (long long)rows, (long long)ld);
        return FTQ_ERR_INVALID_ARG;
    }
    if (rows > INT64_MAX / 8 / ld) { set_error("tensor sizes overflow 64-bit byte offsets"); return FTQ_ERR_UNSUPPORTED; }
    return FTQ_OK;
}

// K of the 8-bit floating-point matmul is a multiple of 16, not of 32: the
// shared size rules are applied to K rounded up.
int check_sizes_fp8(int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k)
{
    if (K <= 0 || K % 16 != 0) { set_error("K must be a positive multiple of 16 (got %lld)", (long long)K); return FTQ_ERR_INVALID_ARG; }
    if (K > kFp8MaxK) { set_error("K = %lld exceeds the supported %lld", (long long)K, (long long)kFp8MaxK); return FTQ_ERR_UNSUPPORTED; }
    const int st = check_sizes(E, N, (K + 31) / 32 * 32, T, top_k);
    if (st != FTQ_OK) return st;
    if (T > 0 && K > INT64_MAX / 64 / (T * top_k)) { set_error("tensor sizes overflow 64-bit byte offsets"); return FTQ_ERR_UNSUPPORTED; }
    return FTQ_OK;
}

int resolve_path_fp8(int path, int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k)
{
    if (path == FTQ_PATH_AUTO) return fp8_select_path(E, N, K, T, top_k);
    if (path == FTQ_PATH_GEMV || path == FTQ_PATH_GROUPED) return path;
    return -1;
}

int fp8_common(const Fp8Args& m, bool per_pair, void* ws, size_t ws_bytes, int path, hipStream_t stream, int phases)
{
    clear_error();
    int st = check_sizes_fp8(m.E, m.N, m.K, m.T, m.top_k);
    if (st != FTQ_OK) return st;
    if (phases & kMatmul) {
        if (!dtype_bytes(m.out_dtype)) { set_error("unknown element type %d", m.out_dtype); return FTQ_ERR_INVALID_ARG; }
        if (m.act != 0) {
            if (m.act != FTQ_ACT_SILU && m.act != FTQ_ACT_GELU_TANH) { set_error("unknown activation %d", m.act); return FTQ_ERR_INVALID_ARG; }
            if (m.N % 2 != 0) { set_error("a gated activation needs an even N (gate and up halves), got %lld", (long long)m.N); return FTQ_ERR_INVALID_ARG; }
            if (m.N % 32 != 0) { set_error("a gated activation needs N %% 32 == 0 here, got %lld", (long long)m.N); return FTQ_ERR_UNSUPPORTED; }
        }
    }
    if (phases != (kRoute | kMatmul) && path == FTQ_PATH_AUTO) {
        set_error("a routing serves matmuls of several sizes: name the path (ftq_moe_fp8_select_path)");
        return FTQ_ERR_INVALID_ARG;
    }
    const int rp = resolve_path_fp8(path, m.E, m.N, m.K, m.T, m.top_k);
    if (rp < 0) { set_error("unknown path %d", path); return FTQ_ERR_INVALID_ARG; }
    const int64_t pairs = m.T * m.top_k;
    if (rp == FTQ_PATH_GEMV && pairs > kFp8GemvMaxPairs) {
        set_error("the GEMV path takes at most %lld pairs (got %lld)", (long long)kFp8GemvMaxPairs, (long long)pairs);
        return FTQ_ERR_UNSUPPORTED;
    }
    if (m.T == 0) return FTQ_OK;
    if (!m.ids || ((phases & kMatmul) && (!m.w || !m.w_scale || !m.a || !m.a_scale || !m.out))) {
        set_error("null pointer argument (w, w_scale, a, a_scale, topk_ids or out)");
        return FTQ_ERR_INVALID_ARG;
    }
    if (!aligned(m.ids, 4) || ((phases & kMatmul) &&
        (!aligned(m.w, 16) || !aligned(m.w_scale, 4) || !aligned(m.a, 16) || !aligned(m.a_scale, 4) ||
         !aligned(m.out, dtype_bytes(m.out_dtype))))) {
        set_error("misaligned pointer (w and a need 16-byte, scales and topk_ids 4-byte, out its element's alignment)");
        return FTQ_ERR_INVALID_ARG;
    }
    Fp8Args args = m;
    args.act_div = per_pair ? 1 : m.top_k;
    if (rp == FTQ_PATH_GEMV) return (phases & kMatmul) ? run_fp8_gemv(args, stream) : FTQ_OK;
    const BucketPlan plan = make_bucket_plan(pairs, m.E, fp8_tile_m(m.E, m.T, m.top_k));
    st = check_workspace(plan.bytes, ws, ws_bytes);
    if (st != FTQ_OK) return st;
    if (phases & kRoute) {
        st = run_bucket(m.ids, m.E, plan, ws, stream);
        if (st != FTQ_OK) return st;
    }
    return (phases & kMatmul) ? run_fp8_grouped(args, plan, ws, stream) : FTQ_OK;
}

}  // namespace

int moe_q4_0_q8_1_call(const void* w, const void* a, const int32_t* ids, float* out, int64_t E, int64_t N, int64_t K,
                       int64_t T, int64_t top_k, void* ws, size_t ws_bytes, int path, hipStream_t stream)
{
    return moe_common(w, a, ids, out, nullptr, E, N, K, T, top_k, ws, ws_bytes, path, stream, kRoute | kMatmul);
}

int64_t moe_workspace_need(int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int path, int* status)
{
    clear_error();
    *status = check_sizes(E, N, K, T, top_k);
    if (*status != FTQ_OK) return -1;
    const int rp = resolve_path(path, E, T, top_k);
    if (rp < 0) {
        set_error("unknown path %d", path);
        *status = FTQ_ERR_INVALID_ARG;
        return -1;
    }
    if (T == 0) return 0;
    bool bucketed = false;
    const BucketPlan plan = plan_for(rp, E, N, K, T, top_k, &bucketed);
    return bucketed ? plan.bytes : 0;
}

}  // namespace ftq

using namespace ftq;

extern "C" {

int ftq_quantize_q8_1(const float* x, int64_t T, int64_t K, void* y, hipStream_t stream)
{
    clear_error();
    if (K <= 0 || K % kQK != 0 || T < 0) { set_error("need K > 0, K %% 32 == 0, T >= 0"); return FTQ_ERR_INVALID_ARG; }
    if (T > INT64_MAX / K / 4) { set_error("T*K overflows"); return FTQ_ERR_UNSUPPORTED; }
    if (T == 0) return FTQ_OK;
    if (!x || !y) { set_error("null pointer argument"); return FTQ_ERR_INVALID_ARG; }
    if (!aligned(x, 16) || !aligned(y, 4)) { set_error("x must be 16-byte and y 4-byte aligned"); return FTQ_ERR_INVALID_ARG; }
    return run_quantize_q8_1(x, T, K, y, stream);
}

int ftq_quantize_q4_0(const float* w, int64_t rows, int64_t K, void* y, hipStream_t stream)
{
    clear_error();
    if (K <= 0 || K % kQK != 0 || rows < 0) { set_error("need K > 0, K %% 32 == 0, rows >= 0"); return FTQ_ERR_INVALID_ARG; }
    if (rows > INT64_MAX / K / 4) { set_error("rows*K overflows"); return FTQ_ERR_UNSUPPORTED; }
    if (rows == 0) return FTQ_OK;
    if (!w || !y) { set_error("null pointer argument"); return FTQ_ERR_INVALID_ARG; }
    if (!aligned(w, 16) || !aligned(y, 2)) { set_error("w must be 16-byte and y 2-byte aligned"); return FTQ_ERR_INVALID_ARG; }
    return run_quantize_q4_0(w, rows, K, y, stream);
}

int ftq_moe_select_path(int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k)
{
    clear_error();
    int st = check_sizes(E, N, K, T, top_k);
    if (st != FTQ_OK) return -st;
    return select_path(E, T, top_k);
}


int64_t ftq_moe_workspace_bytes(int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int path)
{
    return workspace_bytes(E, N, K, T, top_k, path, false);
}

int64_t ftq_moe_pairs_workspace_bytes(int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int path)
{
    return workspace_bytes(E, N, K, T, top_k, path, true);
}

int ftq_moe_q4_0_q8_1(const void* w, const void* a, const int32_t* topk_ids, float* out, int64_t E,
                      int64_t N, int64_t K, int64_t T, int64_t top_k, void* workspace,
                      size_t workspace_bytes, int path, hipStream_t stream)
{
    return moe_common(w, a, topk_ids, out, nullptr, E, N, K, T, top_k, workspace, workspace_bytes, path, stream,
                      kRoute | kMatmul);
}

int ftq_moe_route(const int32_t* topk_ids, int64_t E, int64_t T, int64_t top_k, void* workspace,
                  size_t workspace_bytes, int path, hipStream_t stream)
{
    // N and K do not enter the routing; any valid values pass the size checks
    return moe_common(nullptr, nullptr, topk_ids, nullptr, nullptr, E, 1, kQK, T, top_k, workspace,
                      workspace_bytes, path, stream, kRoute);
}

int ftq_moe_q4_0_q8_1_routed(const void* w, const void* a, const int32_t* topk_ids, float* out, int64_t E,
                             int64_t N, int64_t K, int64_t T, int64_t top_k, void* workspace,
                             size_t workspace_bytes, int path, hipStream_t stream)
{
    return moe_common(w, a, topk_ids, out, nullptr, E, N, K, T, top_k, workspace, workspace_bytes, path, stream,
                      kMatmul);
}

int ftq_moe_q4_0_q8_1_partials(const void* w, const void* a, const int32_t* topk_ids, int32_t* partials,
                               int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k,
                               void* workspace, size_t workspace_bytes, int path, hipStream_t stream)
{
    return moe_common(w, a, topk_ids, nullptr, partials, E, N, K, T, top_k, workspace, workspace_bytes, path, stream,
                      kRoute | kMatmul);
}

int ftq_moe_q4_0_q8_1_pairs(const void* w, const void* a_pairs, const int32_t* topk_ids, float* out, int64_t E,
                            int64_t N, int64_t K, int64_t T, int64_t top_k, void* workspace,
                            size_t workspace_bytes, int path, hipStream_t stream)
{
    return moe_common(w, a_pairs, topk_ids, out, nullptr, E, N, K, T, top_k, workspace, workspace_bytes, path,
                      stream, kRoute | kMatmul, true);
}

int ftq_moe_q4_0_q8_1_pairs_routed(const void* w, const void* a_pairs, const int32_t* topk_ids, float* out,
                                   int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, void* workspace,
                                   size_t workspace_bytes, int path, hipStream_t stream)
{
    return moe_common(w, a_pairs, topk_ids, out, nullptr, E, N, K, T, top_k, workspace, workspace_bytes, path,
                      stream, kMatmul, true);
}

int ftq_moe_q4_0_q8_1_pairs_partials(const void* w, const void* a_pairs, const int32_t* topk_ids,
                                     int32_t* partials, int64_t E, int64_t N, int64_t K, int64_t T,
                                     int64_t top_k, void* workspace, size_t workspace_bytes, int path,
                                     hipStream_t stream)
{
    return moe_common(w, a_pairs, topk_ids, nullptr, partials, E, N, K, T, top_k, workspace, workspace_bytes, path,
                      stream, kRoute | kMatmul, true);
}

int ftq_moe_combine_topk(const float* y, const float* gates, float* out, int64_t T, int64_t top_k, int64_t N,
                         hipStream_t stream)
{
    clear_error();
    if (T < 0 || top_k < 1 || N < 1) {
        set_error("need T >= 0, top_k >= 1, N >= 1 (got T=%lld top_k=%lld N=%lld)", (long long)T, (long long)top_k,
                  (long long)N);
        return FTQ_ERR_INVALID_ARG;
    }
    if (T > INT64_MAX / 8 / top_k / N) { set_error("T*top_k*N overflows 64-bit byte offsets"); return FTQ_ERR_UNSUPPORTED; }
    if (T == 0) return FTQ_OK;
    if (!y || !gates || !out) { set_error("null pointer argument (y, gates or out)"); return FTQ_ERR_INVALID_ARG; }
    if (!aligned(y, 4) || !aligned(gates, 4) || !aligned(out, 4)) {
        set_error("misaligned pointer (y, gates and out need 4-byte alignment)");
        return FTQ_ERR_INVALID_ARG;
    }
    return run_combine_topk(y, gates, out, T, top_k, N, stream);
}

int ftq_moe_q4_0_q8_1_act(const void* w, const void* a, const int32_t* topk_ids, float* out, int64_t E,
                          int64_t N, int64_t K, int64_t T, int64_t top_k, int act, void* workspace,
                          size_t workspace_bytes, int path, hipStream_t stream)
{
    return moe_common(w, a, topk_ids, out, nullptr, E, N, K, T, top_k, workspace, workspace_bytes, path, stream,
                      kRoute | kMatmul, false, act);
}

int ftq_moe_q4_0_q8_1_act_routed(const void* w, const void* a, const int32_t* topk_ids, float* out, int64_t E,
                                 int64_t N, int64_t K, int64_t T, int64_t top_k, int act, void* workspace,
                                 size_t workspace_bytes, int path, hipStream_t stream)
{
    return moe_common(w, a, topk_ids, out, nullptr, E, N, K, T, top_k, workspace, workspace_bytes, path, stream,
                      kMatmul, false, act);
}

int ftq_moe_gguf_q8_1(const void* w, int wtype, const void* a, const int32_t* topk_ids, float* out, int64_t E,
                      int64_t N, int64_t K, int64_t T, int64_t top_k, int act_per_pair, void* workspace,
                      size_t workspace_bytes, int path, hipStream_t stream)
{
    return moe_common(w, a, topk_ids, out, nullptr, E, N, K, T, top_k, workspace, workspace_bytes, path, stream,
                      kRoute | kMatmul, act_per_pair != 0, 0, wtype);
}

int ftq_moe_gguf_q8_1_partials(const void* w, int wtype, const void* a, const int32_t* topk_ids, int32_t* partials,
                               int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int act_per_pair,
                               void* workspace, size_t workspace_bytes, int path, hipStream_t stream)
{
    return moe_common(w, a, topk_ids, nullptr, partials, E, N, K, T, top_k, workspace, workspace_bytes, path, stream,
                      kRoute | kMatmul, act_per_pair != 0, 0, wtype);
}

int ftq_moe_topk(const void* logits, int dtype, int64_t ld, const float* bias, int32_t* topk_ids, float* gates,
                 int64_t T, int64_t E, int64_t top_k, int score, int64_t n_group, int64_t topk_group, int group_top,
                 int renorm, float scale, hipStream_t stream)
{
    clear_error();
    const int64_t esz = dtype_bytes(dtype);
    if (!esz) { set_error("unknown element type %d", dtype); return FTQ_ERR_INVALID_ARG; }
    if (score != FTQ_SCORE_SOFTMAX && score != FTQ_SCORE_SIGMOID) { set_error("unknown score function %d", score); return FTQ_ERR_INVALID_ARG; }
    if (T < 0 || E < 1 || top_k < 1 || ld < E) {
        set_error("need T >= 0, E >= 1, top_k >= 1, ld >= E (got T=%lld E=%lld top_k=%lld ld=%lld)", (long long)T,
                  (long long)E, (long long)top_k, (long long)ld);
        return FTQ_ERR_INVALID_ARG;
    }
    if (n_group < 1 || E % n_group != 0 || topk_group < 1 || topk_group > n_group || group_top < 1 ||
        group_top > 2 || group_top > E / n_group || top_k > topk_group * (E / n_group)) {
        set_error("n_group=%lld topk_group=%lld group_top=%d top_k=%lld do not fit %lld experts", (long long)n_group,
                  (long long)topk_group, group_top, (long long)top_k, (long long)E);
        return FTQ_ERR_INVALID_ARG;
    }
    if (E > kTopkMaxExperts || top_k > kTopkMaxK || n_group > kTopkMaxGroups) {
        set_error("the router takes at most %lld experts, %lld choices and %lld groups (got %lld, %lld, %lld)",
                  (long long)kTopkMaxExperts, (long long)kTopkMaxK, (long long)kTopkMaxGroups, (long long)E,
                  (long long)top_k, (long long)n_group);
        return FTQ_ERR_UNSUPPORTED;
    }
    if (ld > INT64_MAX / 16 || T > INT64_MAX / 16 / ld) { set_error("T*ld overflows 64-bit byte offsets"); return FTQ_ERR_UNSUPPORTED; }
    if (T == 0) return FTQ_OK;
    if (!logits || !topk_ids || !gates) { set_error("null pointer argument (logits, topk_ids or gates)"); return FTQ_ERR_INVALID_ARG; }
    if (!aligned(logits, esz) || !aligned(topk_ids, 4) || !aligned(gates, 4) || (bias && !aligned(bias, 4))) {
        set_error("misaligned pointer (logits need their element's alignment, bias, topk_ids and gates 4-byte alignment)");
        return FTQ_ERR_INVALID_ARG;
    }
    const TopkArgs m{logits, bias, topk_ids, gates, T, ld, dtype, (int32_t)E, (int32_t)top_k, score, (int32_t)n_group,
                     (int32_t)topk_group, group_top, renorm != 0, scale};
    return run_topk(m, stream);
}

int ftq_quantize_fp8(const void* x, int dtype, int64_t ld, int64_t T, int64_t K, void* y, float* scales,
                     hipStream_t stream)
{
    clear_error();
    int st = check_quantize_fp8(dtype, T, K, ld);
    if (st != FTQ_OK) return st;
    if (T == 0) return FTQ_OK;
    if (!x || !y || !scales) { set_error("null pointer argument (x, y or scales)"); return FTQ_ERR_INVALID_ARG; }
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(scales, 4)) { set_error("misaligned pointer (x and y need 16-byte, scales 4-byte alignment)"); return FTQ_ERR_INVALID_ARG; }
    return run_quantize_fp8(x, dtype, ld, T, K, y, scales, stream);
}

int ftq_quantize_fp8_weight(const void* w, int dtype, int64_t E, int64_t N, int64_t K, void* y, float* scales,
                            hipStream_t stream)
{
    clear_error();
    if (E < 0 || N < 0 || (N > 0 && E > INT64_MAX / N)) { set_error("need E >= 0 and N >= 0 (got E=%lld N=%lld)", (long long)E, (long long)N); return FTQ_ERR_INVALID_ARG; }
    int st = check_quantize_fp8(dtype, E * N, K, K);
    if (st != FTQ_OK) return st;
    if (E * N == 0) return FTQ_OK;
    if (!w || !y || !scales) { set_error("null pointer argument (w, y or scales)"); return FTQ_ERR_INVALID_ARG; }
    if (!aligned(w, 16) || !aligned(y, 16) || !aligned(scales, 4)) { set_error("misaligned pointer (w and y need 16-byte, scales 4-byte alignment)"); return FTQ_ERR_INVALID_ARG; }
    return run_quantize_fp8_weight(w, dtype, E, N, K, y, scales, stream);
}

int ftq_moe_fp8_select_path(int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k)
{
    clear_error();
    int st = check_sizes_fp8(E, N, K, T, top_k);
    if (st != FTQ_OK) return -st;
    return fp8_select_path(E, N, K, T, top_k);
}

int64_t ftq_moe_fp8_workspace_bytes(int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int path)
{
    clear_error();
    if (check_sizes_fp8(E, N, K, T, top_k) != FTQ_OK) return -1;
    const int rp = resolve_path_fp8(path, E, N, K, T, top_k);
    if (rp < 0) { set_error("unknown path %d", path); return -1; }
    if (T == 0 || rp == FTQ_PATH_GEMV) return 0;
    return make_bucket_plan(T * top_k, E, fp8_tile_m(E, T, top_k)).bytes;
}

int ftq_moe_fp8(const void* w, const float* w_scale, const void* a, const float* a_scale, const int32_t* topk_ids,
                void* out, int out_dtype, int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k,
                int act_per_pair, int act, void* workspace, size_t workspace_bytes, int path, hipStream_t stream)
{
    const Fp8Args m{static_cast<const uint8_t*>(w), w_scale, static_cast<const uint8_t*>(a), a_scale, topk_ids, out,
                    E, N, K, T, top_k, 0, act, out_dtype & ~FTQ_EXACT, (out_dtype & FTQ_EXACT) != 0};
    return fp8_common(m, act_per_pair != 0, workspace, workspace_bytes, path, stream, kRoute | kMatmul);
}

int ftq_moe_fp8_route(const int32_t* topk_ids, int64_t E, int64_t T, int64_t top_k, void* workspace,
                      size_t workspace_bytes, int path, hipStream_t stream)
{
    // N and K do not enter the routing; any valid values pass the size checks
    const Fp8Args m{nullptr, nullptr, nullptr, nullptr, topk_ids, nullptr, E, 1, kFp8Block, T, top_k, 0, 0, FTQ_F32, true};
    return fp8_common(m, false, workspace, workspace_bytes, path, stream, kRoute);
}

int ftq_moe_fp8_routed(const void* w, const float* w_scale, const void* a, const float* a_scale,
                       const int32_t* topk_ids, void* out, int out_dtype, int64_t E, int64_t N, int64_t K, int64_t T,
                       int64_t top_k, int act_per_pair, int act, void* workspace, size_t workspace_bytes, int path,
                       hipStream_t stream)
{
    const Fp8Args m{static_cast<const uint8_t*>(w), w_scale, static_cast<const uint8_t*>(a), a_scale, topk_ids, out,
                    E, N, K, T, top_k, 0, act, out_dtype & ~FTQ_EXACT, (out_dtype & FTQ_EXACT) != 0};
    return fp8_common(m, act_per_pair != 0, workspace, workspace_bytes, path, stream, kMatmul);
}

const char* ftq_last_error(void) { return g_error.c_str(); }

const char* ftq_version(void) { return "ftq 0.1.0 gfx950"; }

void ftq_debug_force_block_threads(int threads) { g_forced_threads = threads > 0 ? threads : 0; }

void ftq_debug_route_kernels(int split) { g_route_split = split ? 1 : 0; }

int ftq_debug_grouped_kernel(int variant)
{
    clear_error();
    if (variant < kGroupedI8 || variant > kGroupedF16Ws) {
        set_error("grouped kernel variant %d: expected 0 (int8), 1 (fp16) or 2 (fp16, warp-specialised)", variant);
        return FTQ_ERR_INVALID_ARG;
    }
    g_grouped_variant = variant;
    return FTQ_OK;
}

int ftq_debug_gemv_plan(int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k, int wtype, int act, int64_t* seg,
                        int64_t* pairs_per_pass, int64_t* wg_per_cu)
{
    clear_error();
    int st = check_sizes(E, N, K, T, top_k);
    if (st != FTQ_OK) return st;
    if (!seg || !pairs_per_pass || !wg_per_cu) { set_error("null output pointer"); return FTQ_ERR_INVALID_ARG; }
    MoeArgs m{};
    m.E = E; m.N = N; m.K = K; m.T = T; m.top_k = top_k; m.act = act; m.wtype = wtype;
    const GemvPlan g = plan_gemv(m, T * top_k > kGemvScanMaxPairs);
    if (!g.fits) { set_error("a fused activation row of K = %lld does not fit on chip", (long long)K); return FTQ_ERR_UNSUPPORTED; }
    *seg = g.seg;
    *pairs_per_pass = g.pc_cap;
    *wg_per_cu = g.per_cu;
    return FTQ_OK;
}

}  // extern "C"
