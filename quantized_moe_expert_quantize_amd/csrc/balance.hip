// What trains the router: the balance loss of packed sequences with the experts'
// counts, and the gradient of gates and losses with respect to the logits.
//
// For a sequence of n counted tokens, with p_te the scores' share of their row's
// sum (softmax: the scores themselves) and c_e the pairs sent to expert e,
//
//   loss = E / (top_k n^2) * sum_e c_e * sum_t p_te.
//
// A row (token) is worked on by LPR lanes, each with 16 experts in runs of V, so that
// a wave takes 64/LPR rows.  (64 lanes a row, with four experts each, were bound by the
// latency of the reductions: 32768 rows of 256 experts, loss 28 us, gradient 68 us.)
// The loss goes in two kernels: one workgroup per
// chunk of rows sums the probabilities and counts of each sequence that has rows in
// it, and one per sequence adds up its chunks, in a fixed order and without
// floating-point atomics.  Part (chunk c, sequence s) lies at index c + s: along the
// rows either c or s grows, so that no two parts meet.  A small batch is one
// chunk, whose workgroup writes the losses itself.
#include <algorithm>
#include <type_traits>

#include "ftq_internal.h"
#include "row_lanes.h"

namespace ftq {
namespace {

constexpr int kThreads = 256, kAloneThreads = 1024;
constexpr int kPerLane = 16;                          // experts of a lane
constexpr float kInf = __builtin_inff();

// The lanes of a row talk through LDS within one wave, whose LDS accesses the hardware
// keeps in order; the fence keeps the compiler from reordering them.
__device__ __forceinline__ void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront"); }

// N consecutive elements at any element address (the hardware takes unaligned accesses).
template <int N> struct RunF { float v[N]; } __attribute__((packed, aligned(4)));
template <int N> struct alignas(4 * N) LineF { float v[N]; };
template <int N> struct RunH { uint16_t v[N]; } __attribute__((packed, aligned(2)));

template <int DT> __device__ __forceinline__ float load_logit(const void* logits, int64_t i)
{
    if constexpr (DT == FTQ_F32) return static_cast<const float*>(logits)[i];
    const uint16_t h = static_cast<const uint16_t*>(logits)[i];
    return DT == FTQ_F16 ? f32_of_f16(h) : f32_of_bf16(h);
}

// Experts of a lane: run i is (i*LPR + sub)*V .. + V-1; past the last one -inf.
template <int DT, int LPR, int V>
__device__ __forceinline__ void load_row(const void* logits, int64_t at, int sub, int E, float (&l)[kPerLane])
{
#pragma unroll
    for (int i = 0; i < kPerLane / V; ++i) {
        const int e = (i * LPR + sub) * V;
        if (e < E) {                                   // E % V == 0: the whole run
            if constexpr (DT == FTQ_F32) {
                const RunF<V> r = *reinterpret_cast<const RunF<V>*>(static_cast<const float*>(logits) + at + e);
#pragma unroll
                for (int v = 0; v < V; ++v) l[i * V + v] = r.v[v];
            } else {
                const RunH<V> r = *reinterpret_cast<const RunH<V>*>(static_cast<const uint16_t*>(logits) + at + e);
#pragma unroll
                for (int v = 0; v < V; ++v) l[i * V + v] = DT == FTQ_F16 ? f32_of_f16(r.v[v]) : f32_of_bf16(r.v[v]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) l[i * V + v] = -kInf;
        }
    }
}

// e^x for x <= 0: within 1.25 |x| + 2 units of 2^-24 of its size (the base-2 exponent's and its factor's rounding), so that what is
// far off in its own size is small beside the row's largest.  -inf gives 0, a NaN itself.
__device__ __forceinline__ float exp_neg(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

// 1/(1 + e^-l), and 1 minus it, from one exponential of -|l| and one reciprocal (the hardware's, 1 unit off at most).
__device__ __forceinline__ float sigmoid(float l, float& rest)
{
    const float e = exp_neg(-__builtin_fabsf(l)), r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
    rest = l < 0.0f ? r : er;
    return l < 0.0f ? er : r;
}

constexpr float kLow = -60.0f;                        // sigmoids from here down are e^l
__device__ __forceinline__ float finite_top(float top) { return top == -kInf ? 0.0f : top; }

// Scores of a row up to a factor of its own, and their sum: softmax e^(l - top) with the
// row's largest logit; sigmoids as they are, or e^(l - top) where all lie so low that their
// sum would lose bits.  A NaN stays one; a row without a finite logit has zeros.
template <bool SOFT, int LPR>
__device__ __forceinline__ void row_scores(const float (&l)[kPerLane], float (&w)[kPerLane], float (&rest)[kPerLane], float& top, float& sum)
{
    const auto relative = [&] {
        top = -kInf;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) top = fmaxf(top, l[i]);
        top = finite_top(row_max<LPR>(top));
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) sum += w[i] = exp_neg(l[i] - top);
        sum = row_sum<LPR>(sum);
    };
    if constexpr (SOFT) {
        relative();
    } else {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) sum += w[i] = sigmoid(l[i], rest[i]);
        sum = row_sum<LPR>(sum);
        if (sum < 1e-26f) relative();                 // every logit is below kLow
    }
}

// The packed sequences around a wave's rows: lane i holds where sequence s0 + i begins
// (S: the end of the last one), so that finding a row's takes no further loads.
struct Sequences {
    const int32_t* offsets;    // or null: one sequence of all T rows
    int64_t S, T, s0;
    int32_t at;

    // The one that `row` lies in comes first, or the whole array if it fits: 64 probes a load.
    __device__ __forceinline__ void find(const int32_t* offsets_, int64_t S_, int64_t T_, int64_t row, int lane)
    {
        offsets = offsets_;
        S = S_;
        T = T_;
        s0 = 0;
        at = 0;
        if (!offsets) return;
        int64_t n = S;
        while (n > 63) {                              // those in [s0, s0 + n) that end after `row` are its last ones
            const int64_t step = (n + 63) / 64, s = s0 + (lane + 1) * step - 1;
            const int64_t before = __popcll(__ballot(s < s0 + n && offsets[min(s + 1, S)] <= row)) * step;
            s0 += before;
            n = min(step, n - before);
            if (step == 1) break;
        }
        at = offsets[min(s0 + lane, S)];
    }
    // The first sequence from s0 on that ends after `row` (S if none does), and its rows within the T there are.
    __device__ __forceinline__ int64_t of(int64_t row, int64_t& begin, int64_t& end) const
    {
        begin = 0;
        end = T;
        if (!offsets) return 0;
        int i = 0;                                    // entries 1 .. i of `at` are <= row
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const int32_t v = __shfl(at, min(i + o, 63));
            if (i + o < 64 && s0 + i + o <= S && v <= row) i += o;
        }
        begin = __shfl(at, i);
        end = __shfl(at, min(i + 1, 63));
        int64_t s = s0 + i;
        if (i == 63 && s < S) {                       // more sequences than lanes
            while (s < S && offsets[s + 1] <= row) ++s;
            begin = offsets[min(s, S - 1)];
            end = offsets[min(s + 1, S)];
        }
        if (s >= S) {
            begin = end = T;
            return S;
        }
        begin = max(begin, (int64_t)0);
        end = min(end, T);
        return s;
    }
};

struct Part { float p; int32_t c; };

__device__ __forceinline__ float loss_of(double sum, int32_t E, int32_t top_k, int32_t tokens)
{
    const double n = tokens;
    return tokens == 0 ? 0.0f : (float)(sum * E / ((double)top_k * n * n));
}

// ---- loss: parts of a chunk of rows --------------------------------------------

// ALONE: one workgroup takes all rows and writes the losses itself.
template <int DT, bool SOFT, int LPR, int V, bool ALONE>
__global__ __launch_bounds__(ALONE ? kAloneThreads : kThreads) void balance_parts_kernel(BalanceArgs m, int64_t chunk, Part* __restrict__ parts,
                                                                                         int32_t* __restrict__ part_n)
{
    constexpr int THREADS = ALONE ? kAloneThreads : kThreads, kWaves = THREADS / 64;
    constexpr int kRows = THREADS / LPR;              // rows at a time
    extern __shared__ int32_t lds[];                  // [E] counts, then [kWaves][E] sums
    __shared__ double sum_lds[kWaves];
    __shared__ int32_t rows_lds;
    int32_t* hist = lds;
    float* sums = reinterpret_cast<float*>(lds + m.E);
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int sub = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const int64_t r0 = (int64_t)blockIdx.x * chunk, r1 = min(m.T, r0 + chunk);
    Sequences seq;
    seq.find(m.offsets, m.S, m.T, ALONE ? -1 : r0, lane);
    int64_t s = 0, row = r0;
    for (int64_t next = 0;; ++next) {
        int64_t begin, end;
        if constexpr (ALONE) {                        // every sequence (there are few)
            if ((s = next) >= m.S) break;
            begin = m.offsets ? max((int64_t)__shfl(seq.at, (int)s), (int64_t)0) : 0;
            end = m.offsets ? min((int64_t)__shfl(seq.at, (int)s + 1), m.T) : m.T;
        } else {                                      // those that have rows in this chunk
            if (row >= r1 || (s = seq.of(row, begin, end)) >= m.S || begin >= r1 || end <= row) break;   // (end <= row: offsets that descend)
            if (begin > row) {                        // rows of no sequence
                row = begin;
                continue;
            }
            begin = row;
            row = end = min(end, r1);
        }
        const int count = (int)max(end - begin, (int64_t)0);
        float acc[kPerLane] = {}, ahead[kPerLane];
        int32_t n = 0;
        const auto load = [&](int t) {
            t = min(t, count - 1);
            load_row<DT, LPR, V>(m.logits, (begin + t) * m.ld, sub, m.E, ahead);
        };
        if (count > 0) load(slot);
        const int32_t* ids = m.ids + begin * m.top_k;
        const int pairs = count * m.top_k;            // (a chunk's fit 32 bits)
        int32_t next_id = (int)threadIdx.x < pairs ? ids[threadIdx.x] : -1;
        __syncthreads();                              // the last part has been written
        for (int e = threadIdx.x; e < m.E; e += THREADS) hist[e] = 0;
        if (threadIdx.x == 0) rows_lds = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < pairs; i += THREADS) {
            const int32_t id = next_id;
            next_id = i + THREADS < pairs ? ids[i + THREADS] : -1;
            if (id >= 0 && id < m.E && (!m.valid || m.valid[begin + (uint32_t)i / (uint32_t)m.top_k])) atomicAdd(&hist[id], 1);
        }
        for (int t0 = 0; t0 < count; t0 += kRows) {   // every lane goes round as often
            const bool live = t0 + slot < count && (!m.valid || m.valid[begin + t0 + slot]);
            float l[kPerLane], w[kPerLane], rest[kPerLane], top, sum;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) l[i] = ahead[i];
            if (t0 + kRows < count) load(t0 + kRows + slot);
            row_scores<SOFT, LPR>(l, w, rest, top, sum);
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            n += live;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) acc[i] = live ? __builtin_fmaf(w[i], inv, acc[i]) : acc[i];
        }
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int e = (i / V * LPR + sub) * V + i % V;
            acc[i] = sum_over_rows<LPR>(acc[i]);
            if (lane < LPR && e < m.E) sums[wave * m.E + e] = acc[i];
        }
        if (sub == 0 && n) atomicAdd(&rows_lds, n);
        __syncthreads();
        const int64_t at = blockIdx.x + s;
        double loss = 0.0;
        for (int e = threadIdx.x; e < m.E; e += THREADS) {
            float p = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) p += sums[w * m.E + e];
            if constexpr (ALONE) {
                m.counts[s * m.E + e] = hist[e];
                loss += (double)p * hist[e];
            } else {
                parts[at * m.E + e] = Part{p, hist[e]};
            }
        }
        if constexpr (ALONE) {
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) loss += __shfl_xor(loss, o);
            if (lane == 0) sum_lds[wave] = loss;
            __syncthreads();
            if (threadIdx.x == 0) {
                loss = 0.0;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) loss += sum_lds[w];
                m.tokens[s] = rows_lds;
                m.loss[s] = loss_of(loss, m.E, m.top_k, rows_lds);
            }
        } else {
            if (threadIdx.x == 0) part_n[at] = rows_lds;
        }
    }
}

// ---- loss: the parts of a sequence ---------------------------------------------

constexpr int kSumThreads = 1024;

__global__ __launch_bounds__(kSumThreads) void balance_sum_kernel(BalanceArgs m, int64_t chunk, const Part* __restrict__ parts,
                                                                  const int32_t* __restrict__ part_n, int64_t first)
{
    __shared__ double p_lds[kSumThreads];
    __shared__ int32_t c_lds[kSumThreads];
    __shared__ double wave_lds[kSumThreads / 64];
    __shared__ int32_t n_lds;
    const int64_t s = first + blockIdx.x;
    const int64_t begin = m.offsets ? max(m.offsets[s], 0) : 0, end = m.offsets ? min((int64_t)m.offsets[s + 1], m.T) : m.T;
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
#pragma unroll 8
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
        loss = p * c_sum;
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) loss += __shfl_xor(loss, o);
    if (threadIdx.x % 64 == 0) wave_lds[threadIdx.x / 64] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
        loss = 0.0;
        for (int w = 0; w < kSumThreads / 64; ++w) loss += wave_lds[w];
        m.tokens[s] = n_lds;
        m.loss[s] = loss_of(loss, m.E, m.top_k, n_lds);
    }
}

// ---- gradient of the logits ------------------------------------------------------
//
// With v_e = d_loss E/(top_k n^2) c_e, and for choice j of expert e_j, u_j = scale * d_gates_j:
//   balance               dl_k += p_k (v_k - sum_e p_e v_e) [* (1 - s_k) for sigmoid scores]
//   gates, renormalised   D = sum_j s, W = sum_j u s / D: choice j gives s/D (u - W) [* (1 - s)] to its expert
//   gates, softmax        choice j gives s u to its expert, and dl_k -= p_k sum_j s u
//   gates, sigmoid        choice j gives s (1 - s) u to its expert
// The first and third have a term for every expert, which the row's lanes form of their
// experts; what the choices give goes through LDS to the lanes that hold their experts.
// s/D is formed from scores relative to the largest chosen logit, so that choices far
// below the row's largest (a bias can choose them) keep their gradients.

template <int DT, bool SOFT, int LPR, int V>
__global__ __launch_bounds__(kThreads) void topk_backward_kernel(TopkBackwardArgs m, int64_t chunk)
{
    constexpr int kRows = kThreads / LPR;
    extern __shared__ __attribute__((aligned(16))) float row_lds[];                // [kRows][E + 4] gradients of the choices by expert, zero between
                                                      // rows, then [kRows][top_k] of them by choice, and the choices
    const int lane = threadIdx.x & 63, sub = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const int wide_e = m.E + 4;                       // rows of 256 floats would meet the same banks
    float* by_expert = row_lds + slot * wide_e;
    float* by_choice = row_lds + kRows * wide_e + slot * m.top_k;
    int32_t* id_of = reinterpret_cast<int32_t*>(row_lds + kRows * (wide_e + m.top_k)) + slot * m.top_k;
    const bool balance = m.d_loss != nullptr, spreads = SOFT && m.d_gates && !m.renorm;
    const int64_t r0 = (int64_t)blockIdx.x * chunk, r1 = min(m.T, r0 + chunk);
    if (m.d_gates) {
        for (int e = sub; e < m.E; e += LPR) by_expert[e] = 0.0f;
    }
    for (int64_t b = r0; b < r1; b += kRows) {        // every lane goes round as often
        // what a row reads is asked for at once: its logits, the lane's first choice and that choice's logit
        const int64_t t = min(b + slot, r1 - 1);
        const bool there = b + slot < r1, live = !m.valid || m.valid[t];
        float grad[kPerLane] = {}, l[kPerLane], c[kPerLane] = {};
        if (balance || spreads) load_row<DT, LPR, V>(m.logits, t * m.ld, sub, m.E, l);
        const int32_t* ids = m.ids + t * m.top_k;
        const float* d_gates = m.d_gates + t * m.top_k;
        int32_t id0 = -1;
        float u0 = 0.0f, x0 = 0.0f;
        const auto choice = [&](int j, int32_t& id, float& u, float& x) {   // its expert (or -1), scaled gradient and logit
            id = ids[j];
            u = m.scale * d_gates[j];
            if (id < 0 || id >= m.E) id = -1;
            x = id >= 0 ? load_logit<DT>(m.logits, t * m.ld + id) : -kInf;
        };
        if (m.d_gates && sub < m.top_k) choice(sub, id0, u0, x0);
        const auto recall = [&](int j, int32_t& id, float& u, float& x) {
            if (j == sub) {
                id = id0;
                u = u0;
                x = x0;
            } else {
                choice(j, id, u, x);
            }
        };
        bool counted = false;
        if (balance) {
            Sequences seq;
            seq.find(m.offsets, m.S, m.T, uniform(b + threadIdx.x / 64 * (64 / LPR)), lane);
            const int64_t mine = min(seq.s0 + lane, m.S - 1);   // lane i: n and d_loss of sequence s0 + i
            const int32_t tokens_at = m.tokens[mine];
            const float d_loss_at = m.d_loss[mine];
            int64_t begin, end;
            const int64_t s = seq.of(t, begin, end);
            float n = (float)__shfl(tokens_at, (int)min(s - seq.s0, (int64_t)63)), d = __shfl(d_loss_at, (int)min(s - seq.s0, (int64_t)63));
            counted = live && s < m.S && t >= begin && t < end;
            if (counted) {
                if (s - seq.s0 > 63) {
                    n = (float)m.tokens[s];
                    d = m.d_loss[s];
                }
                const float factor = n > 0.0f ? d * (float)m.E / (float)m.top_k / n / n : 0.0f;
#pragma unroll
                for (int i = 0; i < kPerLane / V; ++i) {
                    const int e = (i * LPR + sub) * V;
                    if (e < m.E) {
                        const RunF<V> r = *reinterpret_cast<const RunF<V>*>(reinterpret_cast<const float*>(m.counts) + s * m.E + e);
#pragma unroll
                        for (int v = 0; v < V; ++v) c[i * V + v] = (float)__builtin_bit_cast(int32_t, r.v[v]) * factor;
                    }
                }
            }
        }
        const bool spread = live && spreads, whole = counted || spread;   // whole: a term for every expert
        // the row's lanes over its experts
        float top = 0.0f, inv = 0.0f, pv = 0.0f, rest[kPerLane];
        if (whole) {
            float sum;
            row_scores<SOFT, LPR>(l, grad, rest, top, sum);
            inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) pv = __builtin_fmaf(grad[i], c[i], pv);
            pv = row_sum<LPR>(pv) * inv;
        }
        // the row's lanes over its choices
        float shared = pv;                            // what every expert's term is reduced by
        bool chose = false;
        if (live && m.d_gates) {
            float first = -kInf, sum = 0.0f, us = 0.0f;
            int32_t id;
            float u, x, tail = 1.0f;
            const auto score = [&](float x, float first) {   // up to a factor; tail: 1 - s of a sigmoid
                if constexpr (SOFT) return exp_neg(x - finite_top(first));
                const float s = sigmoid(x, tail);
                return first < kLow ? exp_neg(x - finite_top(first)) : s;
            };
            if (m.renorm) {
                for (int j = sub; j < m.top_k; j += LPR) {
                    recall(j, id, u, x);
                    first = fmaxf(first, x);
                }
                first = row_max<LPR>(first);
                for (int j = sub; j < m.top_k; j += LPR) {
                    recall(j, id, u, x);
                    const float w = score(x, first);       // (of -inf 0)
                    sum += w;
                    us = __builtin_fmaf(u, w, us);
                }
                sum = row_sum<LPR>(sum);
                sum = sum == 0.0f ? 0.0f : 1.0f / sum;
                us = row_sum<LPR>(us) * sum;
            }
            float given = 0.0f;
            for (int j = sub; j < m.top_k; j += LPR) {
                recall(j, id, u, x);
                float g = 0.0f;
                if (id >= 0) {
                    chose = true;
                    if (m.renorm) g = score(x, first) * sum * (u - us);
                    else g = SOFT ? score(x, top) * inv * u : score(x, 0.0f) * u;
                    g *= tail;
                    given += g;
                }
                by_choice[j] = g;
                id_of[j] = id;
            }
            if (spread) shared += row_sum<LPR>(given);
            wave_lds_fence();
            for (int j = sub; j < m.top_k; j += LPR) {   // an expert chosen more than once: the sum in the choices' order, by each
                id = id_of[j];
                if (id < 0) continue;
                float total = 0.0f;
                for (int i = 0; i < m.top_k; ++i) total += id_of[i] == id ? by_choice[i] : 0.0f;
                by_expert[id] = total;
            }
            wave_lds_fence();
        }
        const bool any = row_max<LPR>(chose ? 1.0f : 0.0f) > 0.0f;
        if (whole) {
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                const float d = grad[i] * inv * (c[i] - shared) * (SOFT ? 1.0f : rest[i]);
                grad[i] = counted || any ? d : 0.0f;
            }
        }
        if (any) {
#pragma unroll
            for (int i = 0; i < kPerLane / V; ++i) {
                const int e = (i * LPR + sub) * V;
                if (e < m.E) {
                    const LineF<V> r = *reinterpret_cast<const LineF<V>*>(by_expert + e);
#pragma unroll
                    for (int v = 0; v < V; ++v) grad[i * V + v] += r.v[v];
                }
            }
            wave_lds_fence();
            for (int j = sub; j < m.top_k; j += LPR) {
                if (id_of[j] >= 0) by_expert[id_of[j]] = 0.0f;
            }
            wave_lds_fence();
        }
#pragma unroll
        for (int i = 0; i < kPerLane / V; ++i) {
            const int e = (i * LPR + sub) * V;
            if (!there || e >= m.E) continue;
            if constexpr (DT == FTQ_F32) {
                RunF<V> r;
#pragma unroll
                for (int v = 0; v < V; ++v) r.v[v] = grad[i * V + v];
                *reinterpret_cast<RunF<V>*>(static_cast<float*>(m.d_logits) + t * m.ld_d + e) = r;
            } else {
                RunH<V> r;
#pragma unroll
                for (int v = 0; v < V; ++v) r.v[v] = DT == FTQ_F16 ? f16_of_f32(grad[i * V + v]) : bf16_of_f32(grad[i * V + v]);
                *reinterpret_cast<RunH<V>*>(static_cast<uint16_t*>(m.d_logits) + t * m.ld_d + e) = r;
            }
        }
    }
}

constexpr int64_t kMaxChunks = 512;

// Lanes of a row of E experts.  (Odd numbers of experts have two layouts, so that there are fewer kernels.)
int lanes_of(int64_t E)
{
    if (E % 4 != 0) return E <= 256 ? 16 : 64;
    return E <= 32 ? 2 : E <= 64 ? 4 : E <= 128 ? 8 : E <= 256 ? 16 : E <= 512 ? 32 : 64;
}

// Calls f<DT, SOFT, LPR, V>() for such rows.
template <typename F>
int by_layout(int dtype, int score, int64_t E, F f)
{
    const auto with = [&](auto dt, auto soft) {
        constexpr int DT = decltype(dt)::value;
        constexpr bool SOFT = decltype(soft)::value;
        const int lanes = lanes_of(E);
        if (E % 4 != 0) return lanes == 16 ? f.template operator()<DT, SOFT, 16, 1>() : f.template operator()<DT, SOFT, 64, 1>();
        if (lanes == 2) return f.template operator()<DT, SOFT, 2, 4>();
        if (lanes == 4) return f.template operator()<DT, SOFT, 4, 4>();
        if (lanes == 8) return f.template operator()<DT, SOFT, 8, 4>();
        if (lanes == 16) return f.template operator()<DT, SOFT, 16, 4>();
        if (lanes == 32) return f.template operator()<DT, SOFT, 32, 4>();
        return f.template operator()<DT, SOFT, 64, 4>();
    };
    const auto typed = [&](auto dt) { return score == FTQ_SCORE_SOFTMAX ? with(dt, std::true_type{}) : with(dt, std::false_type{}); };
    if (dtype == FTQ_F32) return typed(std::integral_constant<int, FTQ_F32>{});
    if (dtype == FTQ_F16) return typed(std::integral_constant<int, FTQ_F16>{});
    return typed(std::integral_constant<int, FTQ_BF16>{});
}

// Rows that a workgroup of so many threads works on at a time.
int64_t rows_at_once(int64_t E, int64_t threads) { return threads / lanes_of(E); }

struct BalancePlan { int64_t chunk, chunks, off_n, bytes; bool alone; };

// One workgroup does a small batch by itself: at most two rounds over the rows, and few sequences, which it takes one by one.
BalancePlan plan_balance(int64_t T, int64_t E, int64_t S)
{
    BalancePlan p;
    p.alone = S <= 4 && T <= 2 * rows_at_once(E, kAloneThreads);
    p.chunk = p.alone ? std::max<int64_t>(T, 1) : std::max(rows_at_once(E, kThreads), (T + kMaxChunks - 1) / kMaxChunks);
    p.chunks = p.alone ? 1 : (T + p.chunk - 1) / p.chunk;
    p.off_n = (p.chunks + S) * E * (int64_t)sizeof(Part);
    p.bytes = (p.off_n + (p.chunks + S) * 4 + 255) / 256 * 256;
    return p;
}

struct PartsCall {
    const BalanceArgs& m;
    const BalancePlan& p;
    Part* parts;
    int32_t* part_n;
    hipStream_t s;
    template <int DT, bool SOFT, int LPR, int V> int operator()() const
    {
        const auto go = [&](auto* kernel, int threads) {
            return launch("balance_parts_kernel", kernel, p.chunks, threads, sizeof(int32_t) * m.E * (1 + threads / 64), s, m, p.chunk, parts, part_n);
        };
        return p.alone ? go(balance_parts_kernel<DT, SOFT, LPR, V, true>, kAloneThreads) : go(balance_parts_kernel<DT, SOFT, LPR, V, false>, kThreads);
    }
};

struct TopkBackwardCall {
    const TopkBackwardArgs& m;
    int64_t chunk, chunks;
    hipStream_t s;
    template <int DT, bool SOFT, int LPR, int V> int operator()() const
    {
        const size_t lds = m.d_gates ? sizeof(float) * (kThreads / LPR) * (m.E + 4 + 2 * m.top_k) : 0;
        return launch("topk_backward_kernel", topk_backward_kernel<DT, SOFT, LPR, V>, chunks, kThreads, lds, s, m, chunk);
    }
};

}  // namespace

int64_t balance_workspace(int64_t T, int64_t E, int64_t S) { return plan_balance(T, E, S).bytes; }

int run_balance(const BalanceArgs& m, void* ws, hipStream_t s)
{
    const BalancePlan p = plan_balance(m.T, m.E, m.S);
    Part* parts = static_cast<Part*>(ws);
    int32_t* part_n = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + p.off_n);
    if (p.chunks > 0) {
        const int st = by_layout(m.dtype, m.score, m.E, PartsCall{m, p, parts, part_n, s});
        if (st != FTQ_OK || p.alone) return st;
    }
    return launch_in_turn(m.S, kSumThreads, [&](int64_t first, int64_t n) {
        return launch("balance_sum_kernel", balance_sum_kernel, n, kSumThreads, 0, s, m, p.chunk, static_cast<const Part*>(parts),
                      static_cast<const int32_t*>(part_n), first);
    });
}

int run_topk_backward(const TopkBackwardArgs& m, hipStream_t s)
{
    const int64_t rows = rows_at_once(m.E, kThreads);   // a workgroup goes round once, unless there are more than a launch takes
    const int64_t chunk = std::max(rows, (m.T + (int64_t(1) << 20) - 1) >> 20);
    return by_layout(m.dtype, m.score, m.E, TopkBackwardCall{m, chunk, (m.T + chunk - 1) / chunk, s});
}

}  // namespace ftq
