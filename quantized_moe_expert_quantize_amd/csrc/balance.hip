// What trains the router: the balance loss of packed sequences with the experts'
// counts, and the gradient of gates and losses with respect to the logits.
//
// For a sequence of n counted tokens, with p_te the scores' share of their row's
// sum (softmax: the scores themselves) and c_e the pairs sent to expert e,
//
//   loss = E / (top_k n^2) * sum_e c_e * sum_t p_te.
//
// A row (token) is worked on by LPR lanes, each with runs of V consecutive experts,
// so that a wave takes 64/LPR rows.  The loss goes in two kernels: one workgroup per
// chunk of rows sums the probabilities and counts of each sequence that has rows in
// it, and one per sequence adds up its chunks, in a fixed order and without
// floating-point atomics.  Part (chunk c, sequence s) lies at index c + s: along the
// rows either c or s grows, so that no two parts meet.
#include "ftq_internal.h"

namespace ftq {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr float kInf = __builtin_inff();

template <int V> struct RunF { float v[V]; } __attribute__((packed, aligned(4)));
template <int V> struct RunH { uint16_t v[V]; } __attribute__((packed, aligned(2)));

// e^x for x <= 0: the base-2 product's rounding is carried along.
__device__ __forceinline__ float exp_neg(float x)
{
    constexpr float kLog2e = 1.4426950408889634f, kRest = 1.9259629911266175e-8f, kLn2 = 0.6931471805599453f;
    const float t = x * kLog2e;
    const float r = __builtin_fmaf(x, kRest, __builtin_fmaf(x, kLog2e, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return e == 0.0f ? e : __builtin_fmaf(e, r * kLn2, e);   // (-inf: its r is a NaN)
}

// Experts of a lane: run i is (i*LPR + sub)*V .. + V-1; past the last one -inf.
template <bool WIDE, int LPR, int G, int V>
__device__ __forceinline__ void load_row(const void* logits, int dtype, int64_t at, int sub, int E, float (&l)[G][V])
{
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const int e = (i * LPR + sub) * V;
        if (e < E) {                                   // E % V == 0: the whole run
            if constexpr (WIDE) {
                const RunF<V> r = *reinterpret_cast<const RunF<V>*>(static_cast<const float*>(logits) + at + e);
#pragma unroll
                for (int v = 0; v < V; ++v) l[i][v] = r.v[v];
            } else {
                const RunH<V> r = *reinterpret_cast<const RunH<V>*>(static_cast<const uint16_t*>(logits) + at + e);
#pragma unroll
                for (int v = 0; v < V; ++v) l[i][v] = dtype == FTQ_F16 ? f32_of_f16(r.v[v]) : f32_of_bf16(r.v[v]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) l[i][v] = -kInf;
        }
    }
}

template <int LPR> __device__ __forceinline__ float row_max(float x)
{
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) x = fmaxf(x, __shfl_xor(x, o));
    return x;
}
template <int LPR> __device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) x += __shfl_xor(x, o);
    return x;
}

// Scores up to a factor of the row's own, from the logit `top` (the row's largest, or the largest chosen one)
// on: softmax e^(l - top); sigmoid 1/(1 + e^-l) = e^min(l,0) / (1 + e^-|l|), divided by e^min(top,0).  No
// logit is too small for them; a NaN stays one, and a row without a finite logit has zeros.
__device__ __forceinline__ float weight_of(float l, float top, bool softmax)
{
    if (softmax) {
        const float d = l - (top == -kInf ? 0.0f : top);
        return exp_neg(d);
    }
    const float t = top < 0.0f && top != -kInf ? top : 0.0f;
    return exp_neg((l < 0.0f ? l : 0.0f) - t) / (1.0f + exp_neg(-__builtin_fabsf(l)));
}

// The sequence [begin, end) of rows that s is, within the T rows there are.
__device__ __forceinline__ void sequence(const int32_t* offsets, int64_t s, int64_t T, int64_t& begin, int64_t& end)
{
    begin = 0;
    end = T;
    if (offsets) {
        begin = max((int64_t)offsets[s], (int64_t)0);
        end = min((int64_t)offsets[s + 1], T);
    }
}

// The first sequence that ends after `row`, found by all threads of the workgroup (one barrier).
__device__ __forceinline__ int64_t first_sequence(const int32_t* offsets, int64_t S, int64_t row, int32_t* lds)
{
    if (!offsets) return 0;
    int before = 0;
    for (int64_t s = threadIdx.x; s < S; s += kThreads) before += offsets[s + 1] <= row;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) before += __shfl_xor(before, o);
    if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = before;
    __syncthreads();
    int64_t n = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) n += lds[w];
    return n;
}

struct Part { float p; int32_t c; };

// ---- loss: parts of a chunk of rows --------------------------------------------

template <int LPR, int G, int V, bool WIDE>
__global__ __launch_bounds__(kThreads) void balance_parts_kernel(BalanceArgs m, int64_t chunk, Part* __restrict__ parts,
                                                                 int32_t* __restrict__ part_n)
{
    constexpr int kRows = kThreads / LPR;             // rows at a time
    extern __shared__ int32_t lds[];                  // [E] counts, then [kRows][E] sums
    __shared__ int32_t found[kWaves];
    __shared__ int32_t rows_lds;
    int32_t* hist = lds;
    float* sums = reinterpret_cast<float*>(lds + m.E);
    const int sub = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const bool softmax = m.score == FTQ_SCORE_SOFTMAX;
    const int64_t r0 = (int64_t)blockIdx.x * chunk, r1 = min(m.T, r0 + chunk);
    for (int64_t s = first_sequence(m.offsets, m.S, r0, found); s < m.S; ++s) {
        int64_t begin, end;
        sequence(m.offsets, s, m.T, begin, end);
        if (begin >= r1) break;
        begin = max(begin, r0);
        end = min(end, r1);
        if (begin >= end) continue;
        __syncthreads();                              // the last part has been written
        for (int e = threadIdx.x; e < m.E; e += kThreads) hist[e] = 0;
        if (threadIdx.x == 0) rows_lds = 0;
        __syncthreads();
        float acc[G][V] = {};
        int32_t n = 0;
        for (int64_t t = begin + slot; t < end; t += kRows) {
            if (m.valid && !m.valid[t]) continue;
            ++n;
            float l[G][V], top = -kInf, sum = 0.0f;
            load_row<WIDE, LPR>(m.logits, m.dtype, t * m.ld, sub, m.E, l);
#pragma unroll
            for (int i = 0; i < G; ++i) {
#pragma unroll
                for (int v = 0; v < V; ++v) top = fmaxf(top, l[i][v]);
            }
            top = row_max<LPR>(top);
#pragma unroll
            for (int i = 0; i < G; ++i) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    l[i][v] = weight_of(l[i][v], top, softmax);
                    sum += l[i][v];
                }
            }
            sum = row_sum<LPR>(sum);
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int i = 0; i < G; ++i) {
#pragma unroll
                for (int v = 0; v < V; ++v) acc[i][v] = __builtin_fmaf(l[i][v], inv, acc[i][v]);
            }
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int e = (i * LPR + sub) * V;
            if (e < m.E) {
#pragma unroll
                for (int v = 0; v < V; ++v) sums[slot * m.E + e + v] = acc[i][v];
            }
        }
        if (sub == 0 && n) atomicAdd(&rows_lds, n);
        const int64_t ids = (end - begin) * m.top_k;
        for (int64_t i = threadIdx.x; i < ids; i += kThreads) {
            const int64_t t = begin + i / m.top_k;
            if (m.valid && !m.valid[t]) continue;
            const int32_t id = m.ids[begin * m.top_k + i];
            if (id >= 0 && id < m.E) atomicAdd(&hist[id], 1);
        }
        __syncthreads();
        const int64_t at = blockIdx.x + s;
        for (int e = threadIdx.x; e < m.E; e += kThreads) {
            float p = 0.0f;
            for (int q = 0; q < kRows; ++q) p += sums[q * m.E + e];
            parts[at * m.E + e] = Part{p, hist[e]};
        }
        if (threadIdx.x == 0) part_n[at] = rows_lds;
    }
}

// ---- loss: the parts of a sequence ---------------------------------------------

constexpr int kSumThreads = 1024;

__global__ __launch_bounds__(kSumThreads) void balance_sum_kernel(BalanceArgs m, int64_t chunk, const Part* __restrict__ parts,
                                                                  const int32_t* __restrict__ part_n)
{
    __shared__ double p_lds[kSumThreads];
    __shared__ int32_t c_lds[kSumThreads];
    __shared__ double wave_lds[kSumThreads / 64];
    __shared__ int32_t n_lds;
    const int64_t s = blockIdx.x;
    int64_t begin, end;
    sequence(m.offsets, s, m.T, begin, end);
    const int64_t c0 = begin / chunk, c1 = begin < end ? (end - 1) / chunk + 1 : c0;
    if (threadIdx.x == 0) n_lds = 0;
    __syncthreads();
    int32_t n = 0;
    for (int64_t c = c0 + threadIdx.x; c < c1; c += kSumThreads) n += part_n[c + s];
    if (n) atomicAdd(&n_lds, n);
    // E <= 1024: `ways` threads an expert, each every ways-th chunk
    const int ways = kSumThreads / m.E, e = threadIdx.x % m.E, way = threadIdx.x / m.E;
    double p = 0.0;
    int32_t c_sum = 0;
    if (way < ways) {
        for (int64_t c = c0 + way; c < c1; c += ways) {
            const Part x = parts[(c + s) * m.E + e];
            p += (double)x.p;
            c_sum += x.c;
        }
    }
    p_lds[threadIdx.x] = p;
    c_lds[threadIdx.x] = c_sum;
    __syncthreads();
    double loss = 0.0;
    if ((int)threadIdx.x < m.E) {
        for (int w = 1; w < ways; ++w) {
            p += p_lds[w * m.E + e];
            c_sum += c_lds[w * m.E + e];
        }
        m.counts[s * m.E + e] = c_sum;
        loss = c_sum == 0 ? 0.0 * p : p * c_sum;
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) loss += __shfl_xor(loss, o);
    if (threadIdx.x % 64 == 0) wave_lds[threadIdx.x / 64] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
        loss = 0.0;
        for (int w = 0; w < kSumThreads / 64; ++w) loss += wave_lds[w];
        const double nd = n_lds;
        m.tokens[s] = n_lds;
        m.loss[s] = n_lds == 0 ? 0.0f : (float)(loss * m.E / ((double)m.top_k * nd * nd));
    }
}

// ---- gradient of the logits ------------------------------------------------------
//
// With v_e = d_loss E/(top_k n^2) c_e, u_e the sum of scale * d_gates over the
// choices that are e, and m_e their number:
//   balance               dl_k += p_k (v_k - sum_e p_e v_e) [* (1 - s_k) for sigmoid scores]
//   gates, renormalised   D = sum m s, W = sum u s / D:  dl_k += s_k/D (u_k - m_k W) [* (1 - s_k)]
//   gates, softmax        dl_k += s_k (u_k - sum_e u_e s_e)
//   gates, sigmoid        dl_k += s_k (1 - s_k) u_k
// s/D is formed from scores relative to the largest chosen logit, so that choices far
// below the row's largest (a bias can choose them) keep their gradients.

template <int LPR, int G, int V, bool WIDE>
__global__ __launch_bounds__(kThreads) void topk_backward_kernel(TopkBackwardArgs m, int64_t chunk)
{
    constexpr int kRows = kThreads / LPR;
    __shared__ int32_t found[kWaves];
    const int sub = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const bool softmax = m.score == FTQ_SCORE_SOFTMAX, balance = m.d_loss != nullptr;
    const int64_t r0 = (int64_t)blockIdx.x * chunk, r1 = min(m.T, r0 + chunk);
    int64_t s = balance ? first_sequence(m.offsets, m.S, r0, found) : 0;
    for (int64_t t = r0 + slot; t < r1; t += kRows) {
        float grad[G][V] = {};
        if (!m.valid || m.valid[t]) {
            float l[G][V];
            load_row<WIDE, LPR>(m.logits, m.dtype, t * m.ld, sub, m.E, l);
            float top = -kInf;
#pragma unroll
            for (int i = 0; i < G; ++i) {
#pragma unroll
                for (int v = 0; v < V; ++v) top = fmaxf(top, l[i][v]);
            }
            top = row_max<LPR>(top);
            bool counted = false;
            float factor = 0.0f;
            if (balance) {
                while (s < m.S && m.offsets && m.offsets[s + 1] <= t) ++s;
                int64_t begin = 0, end = 0;
                if (s < m.S) sequence(m.offsets, s, m.T, begin, end);
                counted = t >= begin && t < end;
                if (counted) {
                    const double n = m.tokens[s];
                    factor = n > 0.0 ? (float)((double)m.d_loss[s] * m.E / ((double)m.top_k * n * n)) : 0.0f;
                }
            }
            float u[G][V] = {}, times[G][V] = {};
            if (m.d_gates) {
                for (int j = 0; j < m.top_k; ++j) {
                    const int32_t id = m.ids[t * m.top_k + j];
                    const float d = m.scale * m.d_gates[t * m.top_k + j];
#pragma unroll
                    for (int i = 0; i < G; ++i) {
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            const bool is = id == (i * LPR + sub) * V + v && id < m.E;
                            u[i][v] += is ? d : 0.0f;
                            times[i][v] += is ? 1.0f : 0.0f;
                        }
                    }
                }
            }
            if (counted || (m.d_gates && softmax && !m.renorm)) {   // sums over the whole row
                float w[G][V], sum = 0.0f, pv = 0.0f, us = 0.0f, c[G][V] = {};
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    const int e = (i * LPR + sub) * V;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if (counted && e < m.E) c[i][v] = (float)m.counts[s * m.E + e + v] * factor;
                        w[i][v] = weight_of(l[i][v], top, softmax);
                        sum += w[i][v];
                        pv = __builtin_fmaf(w[i][v], c[i][v], pv);
                        us = __builtin_fmaf(w[i][v], u[i][v], us);
                    }
                }
                sum = row_sum<LPR>(sum);
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                pv = row_sum<LPR>(pv) * inv;
                us = row_sum<LPR>(us) * inv;
#pragma unroll
                for (int i = 0; i < G; ++i) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float p = w[i][v] * inv;
                        if (counted) grad[i][v] = p * (c[i][v] - pv) * (softmax ? 1.0f : weight_of(-l[i][v], 0.0f, false));
                        if (m.d_gates && softmax && !m.renorm) grad[i][v] += p * (u[i][v] - us);
                    }
                }
            }
            if (m.d_gates && m.renorm) {
                float first = -kInf, w[G][V], sum = 0.0f, us = 0.0f;
#pragma unroll
                for (int i = 0; i < G; ++i) {
#pragma unroll
                    for (int v = 0; v < V; ++v) first = times[i][v] > 0.0f ? fmaxf(first, l[i][v]) : first;
                }
                first = row_max<LPR>(first);
#pragma unroll
                for (int i = 0; i < G; ++i) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        w[i][v] = times[i][v] > 0.0f ? weight_of(l[i][v], first, softmax) : 0.0f;
                        sum = __builtin_fmaf(times[i][v], w[i][v], sum);
                        us = __builtin_fmaf(u[i][v], w[i][v], us);
                    }
                }
                sum = row_sum<LPR>(sum);
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                us = row_sum<LPR>(us) * inv;
#pragma unroll
                for (int i = 0; i < G; ++i) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float d = w[i][v] * inv * (u[i][v] - times[i][v] * us);
                        if (times[i][v] > 0.0f) grad[i][v] += d * (softmax ? 1.0f : weight_of(-l[i][v], 0.0f, false));
                    }
                }
            } else if (m.d_gates && !softmax) {
#pragma unroll
                for (int i = 0; i < G; ++i) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if (times[i][v] > 0.0f) grad[i][v] += u[i][v] * weight_of(l[i][v], 0.0f, false) * weight_of(-l[i][v], 0.0f, false);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int e = (i * LPR + sub) * V;
            if (e >= m.E) continue;
            if constexpr (WIDE) {
                RunF<V> r;
#pragma unroll
                for (int v = 0; v < V; ++v) r.v[v] = grad[i][v];
                *reinterpret_cast<RunF<V>*>(static_cast<float*>(m.d_logits) + t * m.ld_d + e) = r;
            } else {
                RunH<V> r;
#pragma unroll
                for (int v = 0; v < V; ++v) r.v[v] = m.dtype == FTQ_F16 ? f16_of_f32(grad[i][v]) : bf16_of_f32(grad[i][v]);
                *reinterpret_cast<RunH<V>*>(static_cast<uint16_t*>(m.d_logits) + t * m.ld_d + e) = r;
            }
        }
    }
}

constexpr int64_t kChunkRows = 64, kMaxChunks = 512;

// Calls f<LPR, G, V>() for a row of E experts.
template <typename F>
int by_layout(int64_t E, F f)
{
    if (E % 4 == 0) {
        if (E <= 32) return f.template operator()<8, 1, 4>();
        if (E <= 64) return f.template operator()<16, 1, 4>();
        if (E <= 128) return f.template operator()<32, 1, 4>();
        if (E <= 256) return f.template operator()<64, 1, 4>();
        if (E <= 512) return f.template operator()<64, 2, 4>();
        return f.template operator()<64, 4, 4>();
    }
    if (E <= 8) return f.template operator()<8, 1, 1>();
    if (E <= 64) return f.template operator()<64, 1, 1>();
    if (E <= 128) return f.template operator()<64, 2, 1>();
    if (E <= 256) return f.template operator()<64, 4, 1>();
    if (E <= 512) return f.template operator()<64, 8, 1>();
    return f.template operator()<64, 16, 1>();
}

struct PartsCall {
    const BalanceArgs& m;
    int64_t chunk, chunks;
    Part* parts;
    int32_t* part_n;
    hipStream_t s;
    template <int LPR, int G, int V> int operator()() const
    {
        const size_t lds = sizeof(int32_t) * m.E * (1 + kThreads / LPR);
        if (m.dtype == FTQ_F32)
            return launch("balance_parts_kernel", balance_parts_kernel<LPR, G, V, true>, chunks, kThreads, lds, s, m, chunk, parts, part_n);
        return launch("balance_parts_kernel", balance_parts_kernel<LPR, G, V, false>, chunks, kThreads, lds, s, m, chunk, parts, part_n);
    }
};

struct TopkBackwardCall {
    const TopkBackwardArgs& m;
    int64_t chunk, chunks;
    hipStream_t s;
    template <int LPR, int G, int V> int operator()() const
    {
        if (m.dtype == FTQ_F32)
            return launch("topk_backward_kernel", topk_backward_kernel<LPR, G, V, true>, chunks, kThreads, 0, s, m, chunk);
        return launch("topk_backward_kernel", topk_backward_kernel<LPR, G, V, false>, chunks, kThreads, 0, s, m, chunk);
    }
};

struct BalancePlan { int64_t chunk, chunks, off_n, bytes; };

BalancePlan plan_balance(int64_t T, int64_t E, int64_t S)
{
    BalancePlan p;
    p.chunk = std::max(kChunkRows, (T + kMaxChunks - 1) / kMaxChunks);
    p.chunks = (T + p.chunk - 1) / p.chunk;
    p.off_n = (p.chunks + S) * E * (int64_t)sizeof(Part);
    p.bytes = (p.off_n + (p.chunks + S) * 4 + 255) / 256 * 256;
    return p;
}

}  // namespace

int64_t balance_workspace(int64_t T, int64_t E, int64_t S) { return plan_balance(T, E, S).bytes; }

int run_balance(const BalanceArgs& m, void* ws, hipStream_t s)
{
    const BalancePlan p = plan_balance(m.T, m.E, m.S);
    Part* parts = static_cast<Part*>(ws);
    int32_t* part_n = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + p.off_n);
    if (p.chunks > 0) {
        const int st = by_layout(m.E, PartsCall{m, p.chunk, p.chunks, parts, part_n, s});
        if (st != FTQ_OK) return st;
    }
    return launch("balance_sum_kernel", balance_sum_kernel, m.S, kSumThreads, 0, s, m, p.chunk, static_cast<const Part*>(parts),
                  static_cast<const int32_t*>(part_n));
}

int run_topk_backward(const TopkBackwardArgs& m, hipStream_t s)
{
    const int64_t chunk = std::max<int64_t>(32, (m.T + (int64_t(1) << 20) - 1) >> 20);
    return by_layout(m.E, TopkBackwardCall{m, chunk, (m.T + chunk - 1) / chunk, s});
}

}  // namespace ftq
