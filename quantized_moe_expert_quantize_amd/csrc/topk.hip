// Router: top-k experts and gate weights of every token from its router logits
// (scores, optional balance bias for the choice, optional groups, renormalised
// gates), in the layout the expert matmuls and the combine take.
//
// One row (token) is worked on by LPR lanes of a wave, LPR the power of two
// from 8 to 64 that holds the experts, so that a wave takes 64/LPR rows and a
// workgroup 256/LPR.  The choice is the one 64-bit arithmetic makes: scores are
// evaluated in 64 bits, kept in LDS, and the top_k taken by as many rounds of a
// maximum over the row's lanes (value, then lower index).
#include "ftq_internal.h"

namespace ftq {
namespace {

constexpr int kThreads = 256;

// The lanes of a row talk through LDS within one wave, whose LDS accesses the
// hardware keeps in order; the fence keeps the compiler from reordering them.
__device__ __forceinline__ void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront"); }

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i)
{
    if constexpr (DT == FTQ_F32) return static_cast<const float*>(p)[i];
    if constexpr (DT == FTQ_F16) return f32_of_f16(static_cast<const uint16_t*>(p)[i]);
    return f32_of_bf16(static_cast<const uint16_t*>(p)[i]);
}

template <int LPR, typename V>
__device__ __forceinline__ V row_sum(V v)
{
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor(v, o);
    return v;
}

template <int LPR>
__device__ __forceinline__ float row_max(float v)
{
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}

// LDS of one row: the choice values, the runs' scores, the chosen ids.
__host__ __device__ constexpr int64_t row_lds(int64_t E, int64_t n_group, int64_t top_k)
{
    return (E + n_group) * 8 + (top_k + 1) / 2 * 8;
}

template <int DT, int LPR>
__global__ __launch_bounds__(kThreads) void topk_kernel(TopkArgs m)
{
    extern __shared__ double lds[];
    constexpr int kRows = kThreads / LPR;
    const int sub = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const int base = (threadIdx.x & 63) / LPR * LPR;      // first lane of this row in its wave
    double* c = lds + slot * (row_lds(m.E, m.n_group, m.top_k) / 8);
    double* run_score = c + m.E;
    int32_t* picks = reinterpret_cast<int32_t*>(run_score + m.n_group);
    const int run = m.E / m.n_group;
    const double ninf = -__builtin_inf();

    for (int64_t row = (int64_t)blockIdx.x * kRows + slot; row < m.T; row += (int64_t)gridDim.x * kRows) {
        float mx = -__builtin_inff();
        bool bad = false;
        for (int e = sub; e < m.E; e += LPR) {
            const float l = load_logit<DT>(m.logits, row * m.ld + e);
            bad |= l != l || (m.score == FTQ_SCORE_SOFTMAX && l == __builtin_inff());
            mx = fmaxf(mx, l);
        }
        mx = row_max<LPR>(mx);
        bad = ((__ballot(bad) >> base) & (LPR == 64 ? ~0ull : (1ull << (LPR & 63)) - 1)) != 0;
        if (mx == -__builtin_inff()) mx = 0.0f;           // no expert is available
        double sum = 1.0;
        if (m.score == FTQ_SCORE_SOFTMAX) {
            sum = 0.0;
            for (int e = sub; e < m.E; e += LPR) sum += exp((double)load_logit<DT>(m.logits, row * m.ld + e) - (double)mx);
            sum = row_sum<LPR>(sum);
        }
        const auto score = [&](float l) -> double {
            return m.score == FTQ_SCORE_SOFTMAX ? exp((double)l - (double)mx) / sum : 1.0 / (1.0 + exp(-(double)l));
        };
        // by_score: the value is s (+ bias); else the logit, whose order is that of s
        const auto value = [&](int e, bool by_score) -> double {
            const float l = load_logit<DT>(m.logits, row * m.ld + e);
            double v = l;
            if (by_score) v = score(l) + (m.bias ? (double)m.bias[e] : 0.0);
            return (l == -__builtin_inff() || v != v) ? ninf : v;
        };
        uint64_t keep = ~0ull;                            // bit g: experts of run g may be chosen
        if (m.n_group > 1) {
            for (int e = sub; e < m.E; e += LPR) c[e] = value(e, m.bias || m.group_top > 1);
            wave_lds_fence();
            double mine = ninf;
            if (sub < m.n_group) {
                double a = ninf, b = ninf;                // the run's largest and second largest
                for (int i = sub * run; i < (sub + 1) * run; ++i) {
                    const double v = c[i];
                    b = fmax(b, fmin(a, v));
                    a = fmax(a, v);
                }
                mine = m.group_top == 2 ? a + b : a;
                if (mine != mine) mine = ninf;
                run_score[sub] = mine;
            }
            wave_lds_fence();
            int above = 0;
            for (int g = 0; g < m.n_group; ++g) {
                const double v = run_score[g];
                above += v > mine || (v == mine && g < sub);
            }
            keep = __ballot(sub < m.n_group && above < m.topk_group) >> base;
        }
        for (int e = sub; e < m.E; e += LPR) c[e] = ((keep >> (e / run)) & 1) || m.n_group == 1 ? value(e, m.bias != nullptr) : ninf;
        wave_lds_fence();
        for (int j = 0; j < m.top_k; ++j) {
            double best = ninf;
            int at = INT32_MAX;
            for (int e = sub; e < m.E; e += LPR) {
                if (c[e] > best) { best = c[e]; at = e; }
            }
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) {
                const double v = __shfl_xor(best, o);
                const int i = __shfl_xor(at, o);
                if (v > best || (v == best && i < at)) { best = v; at = i; }
            }
            const bool none = bad || best == ninf;
            if (sub == 0) {
                picks[j] = none ? -1 : at;
                if (!none) c[at] = ninf;
            }
            wave_lds_fence();
        }
        const int id = sub < m.top_k ? picks[sub] : -1;
        const double s = id >= 0 ? score(load_logit<DT>(m.logits, row * m.ld + id)) : 0.0;
        const double total = row_sum<LPR>(s);
        if (sub < m.top_k) {
            double g = m.renorm ? (total > 0.0 ? s / total : 0.0) : s;
            g = id >= 0 ? g * (double)m.scale : 0.0;
            m.ids[row * m.top_k + sub] = id;
            m.gates[row * m.top_k + sub] = bad ? __builtin_nanf("") : (float)g;
        }
        wave_lds_fence();                                 // the next row reuses this row's LDS
    }
}

template <int DT, int LPR>
int launch_topk(const TopkArgs& m, const DeviceLimits& lim, hipStream_t s)
{
    constexpr int kRows = kThreads / LPR;
    return launch("topk_kernel", topk_kernel<DT, LPR>, stride_grid((m.T + kRows - 1) / kRows, lim), kThreads,
                  (size_t)(kRows * row_lds(m.E, m.n_group, m.top_k)), s, m);
}

template <int DT>
int run_typed(const TopkArgs& m, const DeviceLimits& lim, hipStream_t s)
{
    if (m.E <= 8) return launch_topk<DT, 8>(m, lim, s);
    if (m.E <= 16) return launch_topk<DT, 16>(m, lim, s);
    if (m.E <= 32) return launch_topk<DT, 32>(m, lim, s);
    return launch_topk<DT, 64>(m, lim, s);
}

}  // namespace

int run_topk(const TopkArgs& m, hipStream_t s)
{
    DeviceLimits lim;
    int st = device_limits(&lim);
    if (st != FTQ_OK) return st;
    if (m.dtype == FTQ_F32) return run_typed<FTQ_F32>(m, lim, s);
    if (m.dtype == FTQ_F16) return run_typed<FTQ_F16>(m, lim, s);
    return run_typed<FTQ_BF16>(m, lim, s);
}

}  // namespace ftq
