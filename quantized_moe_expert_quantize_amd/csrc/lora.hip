// Low-rank adapters of many requests beside a shared projection.  Pair p of adapter
// l (its id; others have none) with row x and scale s_l:
//
//   h[p] = A_l x,   out[p] = base[p] + s_l B_l h[p]
//
// and, from d_out, with g[p] = s_l B_l^T d_out[p],
//
//   d_x = sum over a row's pairs of A_l^T g[p],
//   dA_l = sum over the adapter's pairs of g[p] x^T,   dB_l = s_l * the same of d_out[p] h[p]^T.
#include "ftq_internal.h"

namespace ftq {
namespace {

constexpr int kThreads = 256;

template <int DT> __device__ __forceinline__ float load1(const void* p, int64_t i)
{
    if constexpr (DT == FTQ_F32) return static_cast<const float*>(p)[i];
    else return DT == FTQ_F16 ? f32_of_f16(static_cast<const uint16_t*>(p)[i]) : f32_of_bf16(static_cast<const uint16_t*>(p)[i]);
}
template <int DT> __device__ __forceinline__ void store1(void* p, int64_t i, float v)
{
    if constexpr (DT == FTQ_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = DT == FTQ_F16 ? f16_of_f32(v) : bf16_of_f32(v);
}
__device__ __forceinline__ bool adapter_ok(int32_t id, int64_t L) { return id >= 0 && id < L; }

// z[p][r] = f_l * sum_c w[l*w_l + r*w_r + c*w_c] * v[row][c]: a wave per pair.
template <int DT>
__global__ __launch_bounds__(kThreads) void lora_shrink_kernel(const void* v, int64_t ldv, int64_t div, const void* w, int64_t w_l,
                                                               int64_t w_r, int64_t w_c, const float* scale, const int32_t* ids,
                                                               float* z, int64_t L, int64_t R, int64_t C, int64_t pairs)
{
    const int lane = threadIdx.x % 64;
    for (int64_t p = (int64_t)blockIdx.x * 4 + threadIdx.x / 64; p < pairs; p += (int64_t)gridDim.x * 4) {
        const int32_t id = ids[p];
        for (int64_t r = 0; r < R; ++r) {
            float sum = 0.0f;
            if (adapter_ok(id, L)) {
                for (int64_t c = lane; c < C; c += 64) sum = __builtin_fmaf(load1<DT>(w, id * w_l + r * w_r + c * w_c), load1<DT>(v, p / div * ldv + c), sum);
                if (scale) sum *= scale[id];
            }
            for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
            if (lane == 0) z[p * R + r] = sum;
        }
    }
}

// out[row][c] = base[row][c] + sum over the row's `per` pairs of f_l * sum_r z[p][r] * w[l*w_l + r*w_r + c*w_c].
template <int DT, int OT>
__global__ __launch_bounds__(kThreads) void lora_expand_kernel(const float* z, const void* w, int64_t w_l, int64_t w_r, int64_t w_c,
                                                               const float* scale, const int32_t* ids, const void* base, int64_t ldb,
                                                               void* out, int64_t ldo, int64_t L, int64_t R, int64_t C, int64_t rows,
                                                               int64_t per)
{
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < rows * C; i += (int64_t)gridDim.x * kThreads) {
        const int64_t row = i / C, c = i - row * C;
        float sum = 0.0f;
        for (int64_t p = row * per; p < (row + 1) * per; ++p) {
            const int32_t id = ids[p];
            if (!adapter_ok(id, L)) continue;
            float part = 0.0f;
            for (int64_t r = 0; r < R; ++r) part = __builtin_fmaf(z[p * R + r], load1<DT>(w, id * w_l + r * w_r + c * w_c), part);
            sum += scale ? scale[id] * part : part;
        }
        store1<OT>(out, row * ldo + c, base ? load1<OT>(base, row * ldb + c) + sum : sum);
    }
}

// d[l*w_l + r*w_r + c*w_c] = f_l * sum over the adapter's pairs of z[p][r] * v[row][c].
template <int DT>
__global__ __launch_bounds__(kThreads) void lora_outer_kernel(const float* z, const void* v, int64_t ldv, int64_t div, const float* scale,
                                                              const int32_t* ids, float* d, int64_t w_l, int64_t w_r, int64_t w_c,
                                                              int64_t L, int64_t R, int64_t C, int64_t pairs)
{
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < L * R * C; i += (int64_t)gridDim.x * kThreads) {
        const int64_t l = i / (R * C), r = i / C % R, c = i % C;
        float sum = 0.0f;
        for (int64_t p = 0; p < pairs; ++p) {
            if (ids[p] == l) sum = __builtin_fmaf(z[p * R + r], load1<DT>(v, p / div * ldv + c), sum);
        }
        d[l * w_l + r * w_r + c * w_c] = scale ? scale[l] * sum : sum;
    }
}

constexpr int64_t kGrid = int64_t(1) << 20;
int64_t grid_of(int64_t items) { return std::min((items + kThreads - 1) / kThreads, kGrid); }

template <int DT, int OT>
int forward(const LoraArgs& m, float* z, hipStream_t s)
{
    const int64_t pairs = m.T * m.top_k;
    int st = launch("lora_shrink_kernel", lora_shrink_kernel<DT>, std::min((pairs + 3) / 4, kGrid), kThreads, 0, s, m.x, m.ldx, m.act_div,
                    m.a, m.R * m.K, m.K, int64_t(1), (const float*)nullptr, m.ids, z, m.L, m.R, m.K, pairs);
    if (st != FTQ_OK) return st;
    return launch("lora_expand_kernel", lora_expand_kernel<DT, OT>, grid_of(pairs * m.N), kThreads, 0, s, (const float*)z, m.b, m.N * m.R,
                  int64_t(1), m.R, m.scale, m.ids, m.base, m.ld_base, m.out, m.ld_out, m.L, m.R, m.N, pairs, int64_t(1));
}

template <int DT>
int backward(const LoraBackwardArgs& m, float* g, hipStream_t s)
{
    const int64_t pairs = m.T * m.top_k, rows = pairs / m.act_div;
    int st = FTQ_OK;
    if (pairs > 0 && (m.d_x || m.d_a)) {
        st = launch("lora_shrink_kernel", lora_shrink_kernel<DT>, std::min((pairs + 3) / 4, kGrid), kThreads, 0, s, m.d_out, m.ld_d, int64_t(1),
                    m.b, m.N * m.R, int64_t(1), m.R, m.scale, m.ids, g, m.L, m.R, m.N, pairs);
        if (st != FTQ_OK) return st;
    }
    if (pairs > 0 && m.d_x) {
        st = launch("lora_expand_kernel", lora_expand_kernel<DT, DT>, grid_of(rows * m.K), kThreads, 0, s, (const float*)g, m.a, m.R * m.K, m.K,
                    int64_t(1), (const float*)nullptr, m.ids, m.base, m.K, m.d_x, m.K, m.L, m.R, m.K, rows, m.act_div);
        if (st != FTQ_OK) return st;
    }
    if (m.d_a) {
        st = launch("lora_outer_kernel", lora_outer_kernel<DT>, grid_of(m.L * m.R * m.K), kThreads, 0, s, (const float*)g, m.x, m.ldx, m.act_div,
                    (const float*)nullptr, m.ids, m.d_a, m.R * m.K, m.K, int64_t(1), m.L, m.R, m.K, pairs);
        if (st != FTQ_OK) return st;
    }
    if (!m.d_b) return FTQ_OK;
    return launch("lora_outer_kernel", lora_outer_kernel<DT>, grid_of(m.L * m.R * m.N), kThreads, 0, s, m.h, m.d_out, m.ld_d, int64_t(1),
                  m.scale, m.ids, m.d_b, m.N * m.R, int64_t(1), m.R, m.L, m.R, m.N, pairs);
}

}  // namespace

int64_t lora_workspace(int64_t, int64_t R, int64_t, int64_t, int64_t T, int64_t top_k, int, int) { return (T * top_k * R * 4 + 255) / 256 * 256; }
int64_t lora_backward_workspace(int64_t, int64_t R, int64_t, int64_t, int64_t T, int64_t top_k, int) { return (T * top_k * R * 4 + 255) / 256 * 256; }
int lora_select_path(int64_t, int64_t) { return FTQ_PATH_GEMV; }

int run_lora(const LoraArgs& m, void* ws, int, hipStream_t s)
{
    float* z = m.h ? m.h : static_cast<float*>(ws);
    const auto by_out = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        if (m.out_dtype == FTQ_F32) return forward<DT, FTQ_F32>(m, z, s);
        if (m.out_dtype == FTQ_F16) return forward<DT, FTQ_F16>(m, z, s);
        return forward<DT, FTQ_BF16>(m, z, s);
    };
    if (m.dtype == FTQ_F32) return by_out(std::integral_constant<int, FTQ_F32>{});
    if (m.dtype == FTQ_F16) return by_out(std::integral_constant<int, FTQ_F16>{});
    return by_out(std::integral_constant<int, FTQ_BF16>{});
}

int run_lora_backward(const LoraBackwardArgs& m, void* ws, hipStream_t s)
{
    float* g = static_cast<float*>(ws);
    if (m.dtype == FTQ_F32) return backward<FTQ_F32>(m, g, s);
    if (m.dtype == FTQ_F16) return backward<FTQ_F16>(m, g, s);
    return backward<FTQ_BF16>(m, g, s);
}

}  // namespace ftq
