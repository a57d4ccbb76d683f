// Router: top-k experts and gate weights of every token from its router logits
// (scores, optional balance bias for the choice, optional groups, renormalised
// gates), in the layout the expert matmuls and the combine take.
//
// A row (token) is worked on by LPR lanes of a wave, EPL consecutive experts a
// lane, so that a wave takes 64/LPR rows.
//
// The choice is the one 64-bit arithmetic makes, without 64-bit scores of every
// expert: a lane turns its 32-bit values into ordered integers whose lowest bits
// give way to the expert's number (so that they are all different), a few more
// than top_k candidates are taken by as many rounds of a maximum, over the lane's
// entries and then over the row's lanes (DPP and lane swaps, no LDS), and the
// candidates, one a lane, are ranked by their 64-bit values.  What was not taken
// lies below the last candidate; a row in which that does not put it below the
// top_k with certainty (or whose runs are closer than 32 bits tell, or whose gates
// would lose bits) is done again in 64 bits throughout (exact_row).
//
// (exact_row for every row, the first form, took 127 us for 32768 rows of 256 experts
// in 8 runs with a bias, and 23 us for 8191 rows of 128 in bf16; this one takes 36
// and 5.7.)  It is bound by its instructions, about 150 a row and 64 experts, not by
// the 6.5 and 0.4 us that the logits take to read; a single row takes 3 to 7 us, the
// length of its chain of reductions.
#include "ftq_internal.h"
#include "row_lanes.h"

namespace ftq {
namespace {

constexpr int kThreads = 256;
constexpr float kInf = __builtin_inff();
constexpr float kUlp = 1.0f / 8388608.0f;             // 2^-23
constexpr int kSpare = 2;                             // candidates beyond top_k
constexpr float kTiny = 7.888609052210118e-31f;       // 2^-100

// The lanes of a row talk through LDS within one wave, whose LDS accesses the
// hardware keeps in order; the fence keeps the compiler from reordering them.
__device__ __forceinline__ void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront"); }

__device__ __forceinline__ float load_logit(const TopkArgs& m, int64_t i)
{
    if (m.dtype == FTQ_F32) return static_cast<const float*>(m.logits)[i];
    const uint16_t h = static_cast<const uint16_t*>(m.logits)[i];
    return m.dtype == FTQ_F16 ? f32_of_f16(h) : f32_of_bf16(h);
}

// N consecutive elements from any element address (the hardware takes unaligned 16-byte accesses).
template <int N> struct Run32 { float v[N]; } __attribute__((packed, aligned(4)));
template <int N> struct Run16 { uint16_t v[N]; } __attribute__((packed, aligned(2)));

template <bool WIDE, int EPL>
__device__ __forceinline__ void load_logits(const TopkArgs& m, int64_t i, float (&l)[EPL])
{
    if constexpr (WIDE) {
        const Run32<EPL> r = *reinterpret_cast<const Run32<EPL>*>(static_cast<const float*>(m.logits) + i);
#pragma unroll
        for (int j = 0; j < EPL; ++j) l[j] = r.v[j];
    } else {
        const Run16<EPL> r = *reinterpret_cast<const Run16<EPL>*>(static_cast<const uint16_t*>(m.logits) + i);
#pragma unroll
        for (int j = 0; j < EPL; ++j) l[j] = m.dtype == FTQ_F16 ? f32_of_f16(r.v[j]) : f32_of_bf16(r.v[j]);
    }
}

// ---- reductions over the LPR lanes of a row (row_lanes.h has the 32-bit ones) --------

template <int LPR> __device__ __forceinline__ double row_sum(double v)
{
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor(v, o);
    return v;
}

// The votes of this row's lanes, its first lane at bit 0.
template <int LPR> __device__ __forceinline__ uint64_t row_vote(bool b, int base)
{
    const uint64_t v = __ballot(b);
    return LPR == 64 ? v : (v >> base) & ((1ull << (LPR & 63)) - 1);
}

// ---- 64 bits ---------------------------------------------------------------------

// A double as an integer of the same order (-0 as +0); 0 stands for "not available".
__device__ __forceinline__ uint64_t order_of(double d)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, d + 0.0);
    return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}

// Bytes of LDS that exact_row works in: scores, choice values, runs' scores, chosen ids.
__host__ __device__ constexpr int64_t exact_lds(int64_t E, int64_t n_group, int64_t top_k)
{
    return (2 * E + n_group) * 8 + (top_k + 1) / 2 * 8;
}

// A row in 64 bits, by a whole wave: scores and choice values in LDS, top_k rounds
// of a maximum over the lanes (upper half, lower half, then lowest id).
__device__ void exact_row(const TopkArgs& m, int64_t row, int lane, double* s)
{
    uint64_t* c = reinterpret_cast<uint64_t*>(s + m.E);
    double* run_score = s + 2 * m.E;
    int32_t* picks = reinterpret_cast<int32_t*>(run_score + m.n_group);
    const int run = m.E / m.n_group;
    const bool softmax = m.score == FTQ_SCORE_SOFTMAX;
    const double ninf = -__builtin_inf();
    float mx = -kInf;
    bool nan = false;
    for (int e = lane; e < m.E; e += 64) {
        const float l = load_logit(m, row * m.ld + e);
        nan |= l != l || (softmax && l == kInf);
        mx = fmaxf(mx, l);
        s[e] = l;
    }
    mx = row_max<64>(mx);
    const bool bad = __ballot(nan) != 0;
    if (mx == -kInf) mx = 0.0f;                           // no expert is available
    // choice values by the logits first, where they decide; then s
    const bool by_logit = !m.bias && m.group_top == 1;
    double sum = 0.0;
    for (int e = lane; e < m.E; e += 64) {
        const double l = s[e];
        if (!m.bias) c[e] = l == ninf ? 0 : order_of(l);
        s[e] = softmax ? exp(l - (double)mx) : 1.0 / (1.0 + exp(-l));
        sum += s[e];
    }
    if (softmax) {
        sum = row_sum<64>(sum);
        for (int e = lane; e < m.E; e += 64) s[e] /= sum;
    }
    if (m.bias) {
        for (int e = lane; e < m.E; e += 64) {
            const double v = s[e] + (double)m.bias[e];
            c[e] = load_logit(m, row * m.ld + e) == -kInf || v != v || v == ninf ? 0 : order_of(v);
        }
    }
    wave_lds_fence();
    if (m.n_group > 1) {
        double mine = ninf;
        if (lane < m.n_group) {
            double a = ninf, b = ninf;                    // the run's largest and second largest
            for (int i = lane * run; i < (lane + 1) * run; ++i) {
                const uint64_t k = c[i];
                double v = s[i];
                if (by_logit || m.bias) v = __builtin_bit_cast(double, k ^ (~(uint64_t)((int64_t)k >> 63) | 0x8000000000000000ull));
                if (k == 0) v = ninf;
                b = fmax(b, fmin(a, v));
                a = fmax(a, v);
            }
            mine = m.group_top == 2 ? a + b : a;
            if (mine != mine) mine = ninf;
            run_score[lane] = mine;
        }
        wave_lds_fence();
        int above = 0;
        for (int g = 0; g < m.n_group; ++g) {
            const double v = run_score[g];
            above += v > mine || (v == mine && g < lane);
        }
        const uint64_t keep = __ballot(lane < m.n_group && above < m.topk_group);
        for (int e = lane; e < m.E; e += 64) {
            if (!((keep >> (e / run)) & 1)) c[e] = 0;
        }
        wave_lds_fence();
    }
    for (int j = 0; j < m.top_k; ++j) {
        uint64_t best = 0;
        int at = 0;
        for (int e = lane; e < m.E; e += 64) {
            if (c[e] > best) { best = c[e]; at = e; }
        }
        const uint32_t hi = row_max_u<64>((uint32_t)(best >> 32));
        const uint32_t lo = row_max_u<64>((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
        const uint64_t top = (uint64_t)hi << 32 | lo;
        const int id = (int)~row_max_u<64>(best == top ? ~(uint32_t)at : 0u);
        const bool none = bad || top == 0;
        if (lane == 0) {
            picks[j] = none ? -1 : id;
            if (!none) c[id] = 0;
        }
        wave_lds_fence();
    }
    const int id = lane < m.top_k ? picks[lane] : -1;
    const double g = id >= 0 ? s[id] : 0.0;
    const double total = row_sum<64>(g);
    if (lane < m.top_k) {
        const double v = m.renorm ? (total > 0.0 ? g / total : 0.0) : g;
        m.ids[row * m.top_k + lane] = id;
        m.gates[row * m.top_k + lane] = bad ? __builtin_nanf("") : id >= 0 ? (float)(v * (double)m.scale) : 0.0f;
    }
    wave_lds_fence();
}

// ---- 32 bits ---------------------------------------------------------------------

// fp32 to integers of the same order, -0 as +0; and back.
__device__ __forceinline__ uint32_t order_of(float f)
{
    const uint32_t u = as_u(f + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) { return as_f(k ^ (~(uint32_t)((int32_t)k >> 31) | 0x80000000u)); }

constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f, kLn2 = 0.693147181f;

// x of an exponential, brought to where e^x stays finite; the gates made of what is cut off are below kTiny.
__device__ __forceinline__ float clamped(float x) { return __builtin_amdgcn_fmed3f(x, -200.0f, 80.0f); }

// e^x by the base-2 exponential of a rounded product: relative error 1.5 |x| 2^-24 and a unit in the last place.
__device__ __forceinline__ float coarse_exp(float x) { return __builtin_amdgcn_exp2f(clamped(x) * kLog2e); }

// e^(x + rest), rest being small against x: what the product leaves out (its own rounding, that of log2 e, and rest)
// goes into a factor of its own, so that a unit in the last place and one rounding remain, 3 * 2^-24, whatever x is.
__device__ __forceinline__ float fine_exp(float x, float rest)
{
    const float c = clamped(x), t = c * kLog2e;
    const float left = __builtin_fmaf(rest, kLog2e, __builtin_fmaf(c, kLog2eRest, __builtin_fmaf(c, kLog2e, -t)));
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(e, left * kLn2, e);
}

// e^(v - mx): the difference with its rounding error (the sum of two values and what it lacks, after Knuth).
__device__ __forceinline__ float exp_below(float v, float mx)
{
    const float x = v - mx, back = x - v;
    const float rest = (v - (x - back)) + (-mx - back);
    return fine_exp(x, x > -200.0f ? rest : 0.0f);        // -inf and what is clamped has none
}

// Bytes of LDS of one row: candidates' values and ids, the lanes' two best values, runs' scores with their errors, logits.
__host__ __device__ constexpr int64_t quick_lds(int64_t E, int64_t n_group, int64_t lanes)
{
    return lanes * 8 + lanes * 4 + (n_group > 1 ? (lanes + n_group) * 8 : 0) + (E + 1) / 2 * 8;
}

// A row in 32 bits, its candidates in 64.  False (for all the row's lanes): the row needs exact_row.
template <int LPR, int EPL, bool WIDE>
__device__ __forceinline__ bool quick_row(const TopkArgs& m, int64_t row, int sub, int base, double* mem)
{
    double* cand = mem;
    float2* best_lds = reinterpret_cast<float2*>(cand + LPR);
    float2* run_lds = best_lds + (m.n_group > 1 ? LPR : 0);
    float* logit_lds = reinterpret_cast<float*>(run_lds + (m.n_group > 1 ? m.n_group : 0));
    int32_t* cand_id = reinterpret_cast<int32_t*>(logit_lds + (m.E + 1) / 2 * 2);
    constexpr uint32_t kPlace = LPR * EPL - 1;            // low bits of a key: kPlace - expert
    // this lane's experts: e0 + i for i >= first; the last lane's run is moved back to end with the row
    const int e0 = min(sub * EPL, m.E - EPL), first = sub * EPL < m.E ? sub * EPL - e0 : EPL;
    float l[EPL];
    load_logits<WIDE, EPL>(m, row * m.ld + e0, l);
    Run32<EPL> bias = {};
    if (m.bias) bias = *reinterpret_cast<const Run32<EPL>*>(m.bias + e0);
    const bool softmax = m.score == FTQ_SCORE_SOFTMAX;
    const float limit = softmax ? 3.4028235e38f : kInf;
    float mx = -3.4028235e38f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if (i >= first) logit_lds[e0 + i] = l[i];
        l[i] = i >= first ? l[i] : -kInf;
        nan |= !(l[i] <= limit);
        mx = fmaxf(mx, l[i]);
    }
    if (row_vote<LPR>(nan, base)) return false;
    // Scores: sigmoid, or e^(l - max) (the common divisor only where it matters); 0 for -inf.
    if (softmax) mx = row_max<LPR>(mx);
    const bool by_score = m.bias || (m.n_group > 1 && m.group_top > 1);
    float s[EPL];
    float inv = 1.0f;
    if (by_score || (softmax && !m.renorm)) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) s[i] = softmax ? exp_below(l[i], mx) : __builtin_amdgcn_rcpf(1.0f + coarse_exp(-l[i]));
        if (softmax) {
            // a balanced tree over the experts, whatever the lanes: a row's gates do not go by the launch's layout
            float part[EPL];
#pragma unroll
            for (int i = 0; i < EPL; ++i) part[i] = s[i];
            if (m.E % EPL != 0) {                         // the last lane's run was moved back: down to its places again
#pragma unroll
                for (int d = 1; d < EPL; d *= 2) {
#pragma unroll
                    for (int i = 0; i < EPL; ++i) part[i] = first & d ? (i + d < EPL ? part[i + d] : 0.0f) : part[i];
                }
            }
#pragma unroll
            for (int d = 1; d < EPL; d *= 2) {
#pragma unroll
                for (int i = 0; i < EPL; i += 2 * d) part[i] += part[i + d];
            }
            inv = 1.0f / row_sum<LPR>(part[0]);
        }
    }
    // `off` bounds the error of these scores, in units of 2^-23.  Sigmoid: s (1 - s) (0.75 |x| + 1) <= 0.6 from the
    // exponential, 0.5 from the sum, 1 from the reciprocal.  Softmax: 1.5 for the exponential, the same and half a
    // unit for each of the 10 additions that a term of the divisor goes through, 1 for the quotient.
    const float off = softmax ? 10 * kUlp : 2.5f * kUlp;
    uint32_t key[EPL];
    float a = -kInf, b = -kInf;                           // the lane's two largest values for its run's score
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        float c = l[i], r = l[i];
        if (by_score) r = s[i] * inv;
        if (m.bias) c = r = __builtin_fmaf(s[i], inv, bias.v[i]);
        const bool ok = l[i] > -kInf && c > -kInf;
        key[i] = ok ? (order_of(c) & ~kPlace) | (kPlace - (uint32_t)(e0 + i)) : 0u;
        if (m.n_group > 1) {
            r = ok ? r + 0.0f : -kInf;
            b = fmaxf(b, fminf(a, r));
            a = fmaxf(a, r);
        }
    }
    bool sure = true;
    if (m.n_group > 1) {
        // a lane's experts lie in one run (the launch sees to it): the run's two best over its lanes
        const int lanes = m.E / m.n_group / EPL;
        best_lds[sub] = float2{a, b};
        wave_lds_fence();
        // A run's score and a bound of its error.  Each of the two best values is off by its score's error and by a rounding
        // of its own size, which the sum of two large ones of opposite sign keeps; the sum adds one more rounding.
        // A run that lacks an available expert for it is -inf without error, and such runs go by their number: they get the
        // lowest finite values, in that order, and their rows need no exact_row (32768 x 256, 8 runs, 5 of them masked,
        // 4 kept: 170 us with it, 33 so).
        float mine = -kInf, err = 0.0f;
        if (sub < m.n_group) {
            a = b = -kInf;
#pragma unroll 4
            for (int i = 0; i < lanes; ++i) {
                const float2 v = best_lds[sub * lanes + i];
                b = fmaxf(fmaxf(b, v.y), fminf(a, v.x));
                a = fmaxf(a, v.x);
            }
            mine = m.group_top == 2 ? a + b : a;
            const float least = m.group_top == 2 ? b : a;
            if (by_score && least > -kInf) err = 2 * off + 2 * kUlp * (fabsf(a) + (m.group_top == 2 ? fabsf(b) : 0.0f));
            if (by_score && least == -kInf) mine = as_f(0xff7fffc0u + (uint32_t)sub);
            run_lds[sub] = float2{mine, err};
        }
        wave_lds_fence();
        int above = 0, near = 0;
#pragma unroll 4
        for (int g = 0; g < m.n_group; ++g) {
            const float v = run_lds[g].x, tol = err + run_lds[g].y;
            above += by_score ? v > mine + tol : v > mine || (v == mine && g < sub);
            near += !(v < mine - tol);                    // itself among them
        }
        const bool in = by_score ? near <= m.topk_group : above < m.topk_group;
        sure = row_vote<LPR>(by_score && sub < m.n_group && !in && above < m.topk_group, base) == 0;
        const uint64_t keep = row_vote<LPR>(sub < m.n_group && in, base);
        if (!((keep >> min(sub / lanes, 63)) & 1)) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = 0;
        }
    }
    // candidates: 16-bit logits without a bias have their lowest bits free, so that the keys decide alone
    const bool complete = !m.bias && !WIDE;
    const int count = complete ? m.top_k : min(m.top_k + kSpare, LPR);
    uint32_t mine = 0, best = 0;
    for (int j = 0; j < count; ++j) {
        best = key[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) best = max(best, key[i]);
        best = row_max_u<LPR>(best);
        mine = sub == j ? best : mine;
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = key[i] == best ? 0u : key[i];
    }
    if (count >= m.E) best = 0;                           // nothing is left
    wave_lds_fence();
    const int id = mine ? (int)(kPlace - (mine & kPlace)) : -1;
    const float logit = id >= 0 ? logit_lds[id] : -kInf;
    // The gate's score: sigmoid 3 * 2^-24 from the exponential, 1 and 2 from the sum and the reciprocal.
    float g = softmax ? exp_below(logit, mx) : __builtin_amdgcn_rcpf(1.0f + fine_exp(-logit, 0.0f));
    if (id < 0) g = 0.0f;
    int rank = sub;
    if (!complete) {
        double v = logit;
        if (m.bias && id >= 0) {
            const float be = m.bias[id];
            v = softmax ? (double)__builtin_fmaf(g, inv, be) : 1.0 / (1.0 + exp(-(double)logit)) + (double)be;
        }
        cand[sub] = v;
        cand_id[sub] = id;
        wave_lds_fence();
        // softmax scores with a bias stay 32-bit ones: neighbours among them have to be further apart than their error
        const double tol = m.bias && softmax ? 2 * off + 4 * kUlp * fabs(v) : -1.0;
        bool close = false;
        rank = 0;
#pragma unroll 2
        for (int j = 0; j < count; ++j) {
            const double o = cand[j];
            const int oid = cand_id[j];
            rank += oid >= 0 && (o > v || (o == v && oid < id));
            close = close || (oid >= 0 && oid != id && fabs(o - v) <= tol);
        }
        if (id < 0) rank = sub;                           // those that are none come last, in their places
        // every expert that is no candidate lies below this
        const double rest = best ? (double)value_of(best | kPlace) + (m.bias ? (double)off : 0.0) + (double)kUlp * fabs(v) : -__builtin_inf();
        const bool in = sub < count && id >= 0 && rank < m.top_k;
        sure = sure && row_vote<LPR>(in && (close || (best != 0 && !(v > rest))), base) == 0;
    }
    if (rank >= m.top_k || sub >= count) g = 0.0f;
    sure = sure && row_vote<LPR>(id >= 0 && sub < count && rank < m.top_k && g < kTiny, base) == 0;
    if (!sure) return false;
    const float total = row_sum<LPR>(g);
    if (sub < count && rank < m.top_k) {
        m.ids[row * m.top_k + rank] = id;
        m.gates[row * m.top_k + rank] = id < 0 ? 0.0f : (m.renorm ? g / total : g * inv) * m.scale;
    }
    return true;
}

__host__ __device__ constexpr int64_t wave_lds(int64_t E, int64_t n_group, int64_t top_k, int64_t lanes, int epl)
{
    const int64_t q = epl > 0 ? 64 / lanes * quick_lds(E, n_group, lanes) : 0, x = exact_lds(E, n_group, top_k);
    return q > x ? q : x;
}

// EPL == 0: every row in 64 bits.
template <int LPR, int EPL, bool WIDE>
__global__ __launch_bounds__(kThreads) void topk_kernel(TopkArgs m)
{
    extern __shared__ double lds[];
    constexpr int kRows = 64 / LPR;                       // rows of a wave
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int sub = lane % LPR, slot = lane / LPR;
    double* mem = lds + wave * (wave_lds(m.E, m.n_group, m.top_k, LPR, EPL) / 8);
    for (int64_t row0 = ((int64_t)blockIdx.x * (kThreads / 64) + wave) * kRows; row0 < m.T;
         row0 += (int64_t)gridDim.x * (kThreads / 64) * kRows) {
        bool done = row0 + slot >= m.T;
        if constexpr (EPL > 0) {
            if (!done) {
                done = quick_row<LPR, EPL, WIDE>(m, row0 + slot, sub, lane - sub,
                                                 mem + slot * (quick_lds(m.E, m.n_group, LPR) / 8));
            }
            wave_lds_fence();
        }
        // what needs 64 bits, one row after the other by the whole wave
        for (uint64_t todo = __ballot(!done && sub == 0); todo; todo &= todo - 1) {
            exact_row(m, row0 + (__ffsll((unsigned long long)todo) - 1) / LPR, lane, mem);
        }
        wave_lds_fence();                                 // the next rows reuse this wave's LDS
    }
}

template <int LPR, int EPL>
int launch_topk(const TopkArgs& m, const DeviceLimits& lim, hipStream_t s)
{
    constexpr int64_t kRows = kThreads / LPR;
    const int64_t grid = stride_grid((m.T + kRows - 1) / kRows, lim);
    const size_t lds = (size_t)(kThreads / 64 * wave_lds(m.E, m.n_group, m.top_k, LPR, EPL));
    if (m.dtype == FTQ_F32) return launch("topk_kernel", topk_kernel<LPR, EPL, true>, grid, kThreads, lds, s, m);
    return launch("topk_kernel", topk_kernel<LPR, EPL, false>, grid, kThreads, lds, s, m);
}

}  // namespace

int run_topk(const TopkArgs& m, hipStream_t s)
{
    DeviceLimits lim;
    int st = device_limits(&lim);
    if (st != FTQ_OK) return st;
    // Lanes and experts per lane: every run whole lanes, a lane for each run and choice.
    const int run = m.n_group > 1 ? m.E / m.n_group : 0;   // 0: no constraint
    const int need = std::max(m.n_group, std::min(m.top_k + kSpare, 64));
    const auto fits = [&](int lpr, int epl) { return lpr * epl >= m.E && m.E >= epl && lpr >= need && run % epl == 0; };
    if (m.E <= 64) {
        const int lanes = std::max(m.E, need);
        if (lanes <= 8) return launch_topk<8, 1>(m, lim, s);
        if (lanes <= 16) return launch_topk<16, 1>(m, lim, s);
        if (lanes <= 32) return launch_topk<32, 1>(m, lim, s);
        return launch_topk<64, 1>(m, lim, s);
    }
    // Many rows: more experts a lane, so that a reduction serves more rows (8191 x 128, bf16: 16 lanes of 8 take 5.7 us,
    // 64 of 2 9.5; 32768 x 256, groups: 16 of 16 take 36, 64 of 4 63).  Few: more lanes, a shorter chain (2048 x 128:
    // 4.9 against 4.7; 2048 x 256, groups: 12.0 against 10.1).  Both layouts of a size have the same product, and so the
    // same keys and the same bits of a row in either.  (More than 14 choices do not fit 16 lanes and keep the 64: 32768 x
    // 256, 16 of them 64 us and in bf16 20 of them 45; 32 lanes of 16, whose product is another, took 59 and 50.)
    const bool many = m.T >= 4096;
    if (fits(64, 2)) return many && fits(16, 8) ? launch_topk<16, 8>(m, lim, s) : launch_topk<64, 2>(m, lim, s);
    if (fits(64, 4)) return many && fits(16, 16) ? launch_topk<16, 16>(m, lim, s) : launch_topk<64, 4>(m, lim, s);
    if (fits(64, 8)) return many && fits(32, 16) ? launch_topk<32, 16>(m, lim, s) : launch_topk<64, 8>(m, lim, s);
    if (fits(64, 16)) return launch_topk<64, 16>(m, lim, s);
    return launch_topk<64, 0>(m, lim, s);                  // runs that no lane count splits evenly
}

}  // namespace ftq
