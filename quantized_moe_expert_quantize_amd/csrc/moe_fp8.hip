// The expert matmul on 8-bit floating-point (e4m3) weights and activations with
// one fp32 scale per 128 x 128 block of the weights and per 128 values of an
// activation row.  For pair p of expert e with activation row r:
//
//   y[p][n] = sum_b P_b * (a_scale[r][b] * w_scale[e][n/128][b]),
//   P_b     = sum over the 128 values of block b of w[e][n][.] * a[r][.]
//
// P_b of 16 weight rows x 16 activation rows is made on the matrix units from a
// zero accumulator, and one fp32 FMA per element and block adds it, scaled, to
// the sum.  The weights are the instructions' left operand, so that a lane holds
// four weight rows of ONE activation row: its scale is one value a lane, and its
// results four consecutive outputs.  Operand layout: lane l holds row l%16 of
// its side, and as k the 16-byte runs l/16 and l/16 + 4 of the block.  (The
// instructions' own order of k within the block does not matter while both sides
// use the same.)
//
// Two forms of P_b:
//   exact  the codes are converted to fp16, which holds every e4m3 value, and
//          multiplied by four v_mfma_f32_16x16x32_f16: exact products, fp32 sums
//          (measured 1e-8 relative to the result's norm on normal values).
//   fast   one v_mfma_f32_16x16x128_f8f6f4, twice the rate and no conversion.
//          It aligns each run of eight products to the largest one's exponent and
//          drops bits below 2^-13 of it (measured: 1.5e-5 relative to the result's
//          norm, 1.1e-5 of the sum of the terms' magnitudes at most).
// fp32 results take the exact form.  fp16 and bf16 results of the grouped path
// take the fast one, unless the caller asks for the exact one (FTQ_EXACT): what it
// drops is a hundredth of bf16's own rounding and a tenth of fp16's, but it is
// relative to the terms, so that a result which cancels loses more.  (8191 tokens
// evenly spread, bf16 results: first layer 736 us fast, 1192 exact; second 484 and
// 635.)  The GEMV, which waits for memory, takes the exact form always.
//
// Two kernels.  The GEMV splits K over the waves of a workgroup and reads each
// weight once for up to 16 pairs of its expert; it is bound by HBM (8 experts of
// 28672 x 4096, 8 tokens: 5.8 TB/s; a copy on this card moves 5.2 TB/s, reads and
// writes together).  The grouped one walks expert-sorted tiles (bucket.hip) with
// both operands copied into LDS.  Few pairs an expert: HBM again (512 tokens over
// 128 experts of 1408 x 2816, 4.1 TB/s).  Many: 1.4 PFLOP/s on evenly spread pairs
// and 1.8 to 2.0 on full tiles in the fast form (44 to 46% of the matrix units' time, the rest
// waits for copies and for the ends of ragged tiles), 0.7 to 1.1 in the exact one,
// where a library product of 8192^3 reaches 3.0 in 8 bits and 1.2 in bf16.
#include "ftq_internal.h"
#include "lds_copy.h"

namespace ftq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// One lane's 32 codes of a block, as the matrix instructions of a form take them.
template <bool EXACT> struct Operand;
template <> struct Operand<false> {
    i32x8 v;
    __device__ __forceinline__ explicit Operand(i32x8 codes) : v(codes) {}
    __device__ __forceinline__ Operand() {}
};
template <> struct Operand<true> {
    f16x8 v[4];
    __device__ __forceinline__ Operand() {}
    __device__ __forceinline__ explicit Operand(i32x8 codes)
    {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const int c = codes[2 * h + d];
                const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, false);
                const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, true);
                v[h][4 * d] = lo[0];
                v[h][4 * d + 1] = lo[1];
                v[h][4 * d + 2] = hi[0];
                v[h][4 * d + 3] = hi[1];
            }
        }
    }
};

// P_b of the NP weight tiles from i0 on with one activation tile.
template <int NW, int NP>
__device__ __forceinline__ void block_products(const Operand<false> (&w)[NW], int i0, const Operand<false>& a, f32x4 (&p)[NP])
{
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NP; ++i) p[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[i0 + i].v, a.v, zero, 0, 0, 0, 0, 0, 0);
}
template <int NW, int NP>
__device__ __forceinline__ void block_products(const Operand<true> (&w)[NW], int i0, const Operand<true>& a, f32x4 (&p)[NP])
{
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
#pragma unroll
        for (int i = 0; i < NP; ++i) p[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[i0 + i].v[h], a.v[h], h == 0 ? zero : p[i], 0, 0, 0);
    }
}

__device__ __forceinline__ i32x8 join(i32x4 lo, i32x4 hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }

// This lane's two 16-byte runs of block kb of a row of K codes, zeros past K.
__device__ __forceinline__ i32x8 load_block(const uint8_t* row, int64_t kb, int64_t K, int run)
{
    const int64_t k0 = kb * kFp8Block + run * 16, k1 = k0 + 64;
    i32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
    if (k0 < K) lo = *reinterpret_cast<const i32x4*>(row + k0);
    if (k1 < K) hi = *reinterpret_cast<const i32x4*>(row + k1);
    return join(lo, hi);
}

template <int OUT>
__device__ __forceinline__ void store1(void* out, int64_t i, float v)
{
    if constexpr (OUT == FTQ_F32) static_cast<float*>(out)[i] = v;
    else static_cast<uint16_t*>(out)[i] = OUT == FTQ_F16 ? f16_of_f32(v) : bf16_of_f32(v);
}

// 16 bytes of consecutive results at any element address (the hardware takes
// unaligned accesses), past the caches: results are written once, and kept in L2
// they drive out the weights that other workgroups are about to read (second
// layer, bf16 results: 420 us with plain stores, 346 us so).
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x8_any __attribute__((ext_vector_type(8), aligned(2)));
template <int OUT, int N>
__device__ __forceinline__ void store_run(void* out, int64_t i, const float (&v)[N])
{
    if constexpr (OUT == FTQ_F32) {
        static_assert(N == 4);
        const f32x4_any x = {v[0], v[1], v[2], v[3]};
        __builtin_nontemporal_store(x, reinterpret_cast<f32x4_any*>(static_cast<float*>(out) + i));
    } else {
        static_assert(N == 8);
        u16x8_any x;
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = OUT == FTQ_F16 ? f16_of_f32(v[q]) : bf16_of_f32(v[q]);
        __builtin_nontemporal_store(x, reinterpret_cast<u16x8_any*>(static_cast<uint16_t*>(out) + i));
    }
}

__device__ __forceinline__ bool expert_ok(int32_t id, int64_t E) { return id >= 0 && id < E; }

// ---- GEMV ---------------------------------------------------------------------

constexpr int kGemvWaves = 8;
constexpr int kGemvThreads = 64 * kGemvWaves;

// A workgroup takes 16*CT output columns of one expert: CT 16-row weight tiles, or
// with ACT the gate and the up tiles of the columns, and wave v every eighth block
// of K from block v on.  What keeps enough loads in flight is the number of waves:
// loading two or four blocks ahead in registers costs waves and lost 10 to 40%.
// by_pair: workgroups are laid out over the pairs, and the one of an expert's
// first pair serves all its pairs (few pairs: no workgroup for an expert that none
// takes); else over the experts and, last, the masked pairs.  More workgroups than
// a launch takes are several launches, each from workgroup `first` on.
constexpr int64_t kGemvWideFrom = 16 * 1024;   // columns over all experts from which a workgroup takes 32

template <int CT, int OUT, bool ACT>
__global__ __launch_bounds__(kGemvThreads) void moe_fp8_gemv_kernel(Fp8Args m, int64_t nb, int64_t nr, int64_t ntiles,
                                                                    int by_pair, int64_t first)
{
    constexpr int RT = ACT ? 2 * CT : CT, kCols = 16 * CT;
    __shared__ uint16_t list[kFp8GemvMaxPairs];
    __shared__ int count_lds;
    __shared__ f32x4 part[kGemvWaves][RT][64];
    const int lane = threadIdx.x & 63, wave = uniform((int32_t)(threadIdx.x >> 6));
    const int64_t item = first + blockIdx.x, slot = item / ntiles, n0 = (item - slot * ntiles) * kCols;
    const int pairs = (int)(m.T * m.top_k);
    const int64_t cols = ACT ? m.N / 2 : m.N;
    const int32_t e = by_pair ? uniform(m.ids[slot]) : slot < m.E ? (int32_t)slot : -1;
    const bool live = expert_ok(e, m.E);
    // the pairs of this expert (or the masked ones), ascending
    if (wave == 0) {
        int count = 0;
        for (int p0 = 0; p0 < pairs; p0 += 64) {
            const int p = p0 + lane;
            const int32_t id = p < pairs ? m.ids[p] : 0;
            const bool mine = p < pairs && (live ? id == e : by_pair ? p == (int)slot : !expert_ok(id, m.E));
            const uint64_t vote = __ballot(mine);
            if (mine) list[count + __popcll(vote & ((1ull << lane) - 1))] = (uint16_t)p;
            count += __popcll(vote);
        }
        if (lane == 0) count_lds = count;
    }
    __syncthreads();
    const int count = count_lds;
    if (count == 0 || (by_pair && list[0] != slot)) return;
    if (!live) {
        for (int i = threadIdx.x; i < count * kCols; i += kGemvThreads) {
            if (n0 + i % kCols < cols) store1<OUT>(m.out, list[i / kCols] * cols + n0 + i % kCols, 0.0f);
        }
        return;
    }
    const int r = lane & 15, run = lane >> 4;
    const uint8_t* wrow[RT];
    const float* wscale[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int64_t c = n0 + 16 * (i % CT), up = i / CT * cols;
        wrow[i] = m.w + ((int64_t)e * m.N + min(c + r, cols - 1) + up) * m.K;
        // a tile has one scale: it starts at a multiple of 16
        wscale[i] = m.w_scale + ((int64_t)e * nr + (min(c, cols - 1) + up) / kFp8Block) * nb;
    }
    for (int t0 = 0; t0 < count; t0 += 16) {
        const bool have = t0 + r < count;
        const int64_t arow = have ? list[t0 + r] / (int)m.act_div : 0;
        f32x4 acc[RT] = {};
        for (int64_t kb = wave; kb < nb; kb += kGemvWaves) {
            i32x8 a = {};
            float sa = 0.0f;
            if (have) {
                a = load_block(m.a + arow * m.K, kb, m.K, run);
                sa = m.a_scale[arow * nb + kb];
            }
            Operand<true> w[RT];
            f32x4 p[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) w[i] = Operand<true>(load_block(wrow[i], kb, m.K, run));
            block_products(w, 0, Operand<true>(a), p);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const float s = sa * wscale[i][kb];
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][q] = __builtin_fmaf(p[i][q], s, acc[i][q]);
            }
        }
        __syncthreads();   // the last pass has read part[]
#pragma unroll
        for (int i = 0; i < RT; ++i) part[wave][i][lane] = acc[i];
        __syncthreads();
        for (int h = threadIdx.x; h < 16 * kCols; h += kGemvThreads) {
            // column h%kCols of activation row h/kCols of this pass, its parts in wave order
            const int c = h % kCols, t = h / kCols;
            float y[ACT ? 2 : 1];
#pragma unroll
            for (int i = 0; i < (ACT ? 2 : 1); ++i) {
                y[i] = 0.0f;
#pragma unroll
                for (int v = 0; v < kGemvWaves; ++v) y[i] += part[v][i * CT + c / 16][c % 16 / 4 * 16 + t][c % 4];
            }
            if (t0 + t < count && n0 + c < cols) {
                float v = y[0];
                if constexpr (ACT) v = gated_act(m.act, y[0]) * y[ACT ? 1 : 0];
                store1<OUT>(m.out, list[t0 + t] * cols + n0 + c, v);
            }
        }
    }
}

// ---- grouped ------------------------------------------------------------------

constexpr int kGroups = 4;                             // groups of 64 weight rows (four 16-row tiles) per workgroup

constexpr int kXcds = 8;

struct GroupedTables {
    const int32_t* tiles;     // [E + 2] first tile of each bucket; the last entry is their number
    const int32_t* sorted;    // pair ids by expert
    const int4* tdesc;        // per tile {bucket, first slot, rows, 0}
    int64_t nb, nr, ntn;      // K blocks, weight row blocks per expert, column tiles
};

// A workgroup makes 16*TT*WT pairs x 256 weight rows: four groups of 64 rows, and
// WT waves a group, each with 16*TT of the pairs.  A wave keeps its weights of a
// block in registers and reads the activations a 16-pair tile at a time.  Both come
// by asynchronous copies into LDS, made one block ahead.  With NB == 1 the weights
// have one buffer, of the wave's own, refilled once they are in registers: two such
// workgroups of 64 pairs fit a CU and fill each other's waits.  With NB == 2 they
// have two, like the activations: 256 pairs by eight waves, for experts with many
// pairs (half the weight traffic a product), and 32 pairs by four, for experts with
// few, where the copies in flight are what counts.
// With ACT the wave has 32 columns, tiles 0 and 1 their gate and 2 and 3 their up
// rows.  Which row of a tile is which column is free; it is chosen so that a
// lane's results make whole 16-byte stores and the four lanes of a row 64 bytes
// side by side (8-byte stores at a stride, the first form, took 290 us for the
// 369 MB of a second layer's bf16 results that take 90 us so): fp32, row r of
// tile i is column 16*i + r, four columns a lane and tile; 16 bits, column
// 32*(i/2) + 8*(r/4) + 4*(i%2) + r%4, eight a lane and pair of tiles.
// A table tile of more than 16*TT pairs is made by `subs` items.
template <int TT, int WT, int NB, int OUT, bool ACT, bool EXACT>
__global__ __launch_bounds__(64 * kGroups * WT, 2) void moe_fp8_grouped_kernel(Fp8Args m, GroupedTables g, int subs)
{
    static_assert(NB == 2 || WT == 1);
    static_assert(EXACT || OUT != FTQ_F32);
    constexpr int kWaves = kGroups * WT, kThreads = 64 * kWaves;
    constexpr int BM = 16 * TT * WT;                   // pairs per workgroup
    constexpr int kShare = 8 / WT;                     // copies of its group's weight rows that a wave makes
    constexpr int kRuns = BM * 8 / kThreads;           // 16-byte runs of an activation tile per thread
    constexpr int kCols = ACT ? 32 : 64;               // output columns per wave
    constexpr bool kWide = OUT == FTQ_F32;
    constexpr int kRun = kWide ? 4 : 8;                // consecutive columns of a lane's store
    // weight scales per lane and block: 64 rows from a multiple of 64 on share one, 32 gate rows another, and
    // 32 up rows, which start at a multiple of 16, have at most one for each 16
    constexpr int kScales = ACT ? (kWide ? 3 : 2) : 1;
    constexpr int kScaleOf[4] = {0, 0, ACT ? 1 : 0, kScales - 1};
    __shared__ i32x4 act[2][BM][8];                    // run c of row x sits at c ^ (x % 8)
    __shared__ i32x4 weight[NB][kGroups][64][8];       // each group's rows, swizzled likewise
    __shared__ float act_scale[2][BM < 64 ? 64 : BM];
    __shared__ int32_t pair_of[BM];
    const int lane = threadIdx.x & 63, wave = uniform((int32_t)(threadIdx.x >> 6));
    const int group = wave % kGroups, half = wave / kGroups;   // weight rows, pairs
    const int r = lane & 15, run = lane >> 4;
    const int64_t cols = ACT ? m.N / 2 : m.N;
    const int64_t total = (int64_t)g.tiles[m.E + 1] * subs * g.ntn, full = m.K / kFp8Block;
    // each XCD takes a contiguous eighth of the items, so that what its workgroups share meets in its L2
    const int64_t per = (total + kXcds - 1) / kXcds, end = min(total, (int64_t)(blockIdx.x % kXcds + 1) * per);
    for (int64_t item = blockIdx.x % kXcds * per + blockIdx.x / kXcds; item < end; item += gridDim.x / kXcds) {
        const int64_t mt = item / g.ntn, c0 = (item - mt * g.ntn) * (kGroups * kCols) + group * kCols;
        const int sub = (int)(mt % subs) * BM;
        const int4 td = g.tdesc[mt / subs];
        const int4 desc{uniform(td.x), uniform(td.y) + sub, 0, 0};
        const int rows = min(uniform(td.z) - sub, BM);
        if (rows <= 0) continue;
        __syncthreads();                               // the last item's LDS has been read
        if (threadIdx.x < BM) pair_of[threadIdx.x] = g.sorted[desc.y + min((int)threadIdx.x, rows - 1)];
        __syncthreads();
        if (desc.x >= m.E) {                           // masked pairs: zero rows
            const int64_t first = c0 - group * kCols, n = min((int64_t)(kGroups * kCols), cols - first);
            for (int64_t i = threadIdx.x; i < rows * n; i += kThreads) store1<OUT>(m.out, pair_of[i / n] * cols + first + i % n, 0.0f);
            continue;
        }
        // weights: uniform bases, 32-bit lane offsets
        const int64_t cb = min(c0, cols - 1);
        const uint8_t* wbase[ACT ? 2 : 1];
        const float* wscale[kScales];
#pragma unroll
        for (int i = 0; i < (ACT ? 2 : 1); ++i) wbase[i] = m.w + ((int64_t)desc.x * m.N + cb + i * cols) * m.K;
#pragma unroll
        for (int i = 0; i < kScales; ++i) {
            const int64_t c = i == 0 ? c0 : kWide ? c0 + (i - 1) * 16 : c0 + run * 8;
            const int64_t n = min(c, cols - 1) + (i > 0 ? cols : 0);
            wscale[i] = m.w_scale + ((int64_t)desc.x * g.nr + n / kFp8Block) * g.nb;
        }
        // copies: instruction d of a wave brings LDS rows 8*d .. 8*d + 7, eight lanes a row, so that a row's 128
        // bytes are one request (lanes in operand order, one row each, read 16 bytes a cycle); lane l takes the
        // 16-byte run (l%8) ^ (l/8) of its row
        const int cr = lane / 8, cp = (lane % 8) ^ cr;
        uint32_t woff[kShare];
        static_assert(!ACT || kShare == 8 || kShare == 4);
#pragma unroll
        for (int e = 0; e < kShare; ++e) {
            const int d = half * kShare + e, i = d / 2, y = d % 2 * 8 + cr;   // tile and row of it
            const int t = ACT ? i & 1 : i;             // tile among those of its columns
            const int c = kWide ? 16 * t + y : 32 * (t / 2) + 8 * (y / 4) + 4 * (t & 1) + y % 4;
            woff[e] = (uint32_t)min((int64_t)c, cols - 1 - cb) * (uint32_t)m.K + cp * 16;
        }
        const uint8_t* arow[kRuns];                    // rows (i*4 + wave)*8 + l/8
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
            const int x = (i * kWaves + wave) * 8 + cr;
            arow[i] = m.a + (pair_of[x] / (int)m.act_div) * m.K + cp * 16;
        }
        const float* ascale = m.a_scale + (pair_of[threadIdx.x % BM] / (int)m.act_div) * g.nb;
        constexpr int kScaleWaves = BM < 64 ? 1 : BM / 64;
        float next[kScales];                           // weight scales of the block in flight
        const auto copy_block = [&](int64_t kb, int buf) {
#pragma unroll
            for (int i = 0; i < kScales; ++i) next[i] = wscale[i][kb];
#pragma unroll
            for (int e = 0; e < kShare; ++e) {
                const uint8_t* base = ACT ? (kShare == 8 ? wbase[e / 4] : half ? wbase[ACT ? 1 : 0] : wbase[0]) : wbase[0];
                copy16(lds_address(&weight[NB == 2 ? buf : 0][group][8 * (half * kShare + e)][0]), base + kb * kFp8Block, woff[e]);
            }
#pragma unroll
            for (int i = 0; i < kRuns; ++i) copy16(lds_address(&act[buf][(i * kWaves + wave) * 8][0]), arow[i] + kb * kFp8Block);
            if (wave < kScaleWaves) copy4(lds_address(&act_scale[buf][wave * 64]), ascale + kb);
        };
        i32x8 wv[4];
        float sw[kScales];
        const auto read_weights = [&](int buf) {
#pragma unroll
            for (int i = 0; i < 4; ++i) wv[i] = join(weight[buf][group][16 * i + r][run ^ (r % 8)], weight[buf][group][16 * i + r][(run + 4) ^ (r % 8)]);
        };
        f32x4 acc[4][TT] = {};
        const auto multiply = [&](int buf) {
            Operand<EXACT> w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = Operand<EXACT>(wv[i]);
            // Two weight tiles at a time: their products are made while the last two's are added up, and the next
            // activation tile is read meanwhile.  (The scheduling barriers keep the compiler from making all products
            // first, which takes registers that are not there.)
            const auto tile = [&](int j) {
                const int x = half * 16 * TT + j * 16 + r;
                return join(act[buf][x][run ^ (r % 8)], act[buf][x][(run + 4) ^ (r % 8)]);
            };
            f32x4 p[2][2];
            i32x8 codes = tile(0), ahead = codes;
            float sa = act_scale[buf][half * 16 * TT + r], last = 0.0f, sa_ahead = 0.0f;
#pragma unroll
            for (int h = 0; h <= 2 * TT; ++h) {
                const int j = h / 2, i0 = h % 2 * 2;
                if (i0 == 0 && j + 1 < TT) {
                    ahead = tile(j + 1);
                    sa_ahead = act_scale[buf][half * 16 * TT + (j + 1) * 16 + r];
                }
                if (h < 2 * TT) {
                    const Operand<EXACT> b(codes);
                    block_products(w, i0, b, p[h & 1]);
                }
                if (h > 0) {
                    const int l0 = 2 - i0, lj = (h - 1) / 2;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float s = (i0 == 0 ? last : sa) * sw[kScaleOf[l0 + i]];
#pragma unroll
                        for (int q = 0; q < 4; ++q) acc[l0 + i][lj][q] = __builtin_fmaf(p[(h - 1) & 1][i][q], s, acc[l0 + i][lj][q]);
                    }
                }
                if (i0 == 2) {
                    last = sa;
                    sa = sa_ahead;
                    codes = ahead;
                }
                if constexpr (!EXACT) {               // a product, then the four sums of one made two products ago
                    __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (full > 0) copy_block(0, 0);
        for (int64_t kb = 0; kb < full; ++kb) {
            const int buf = kb & 1;
            wait_copies();
            block_barrier();                           // every wave's copies of block kb are there, block kb - 1 has been read
            if constexpr (NB == 2) {
#pragma unroll
                for (int i = 0; i < kScales; ++i) sw[i] = next[i];
                if (kb + 1 < full) copy_block(kb + 1, buf ^ 1);
                read_weights(buf);
            } else {
                read_weights(0);
                wait_lds();                            // a wave's weights have one buffer: read before the next copy
#pragma unroll
                for (int i = 0; i < kScales; ++i) sw[i] = next[i];
                if (kb + 1 < full) copy_block(kb + 1, buf ^ 1);
            }
            if (WT == 1 || half * 16 * TT < rows) multiply(buf);
        }
        if (full < g.nb) {                             // the last block is cut short: zeros past K on both sides
            const int buf = full & 1;
            const int64_t k0 = full * kFp8Block;
            const bool in = k0 + cp * 16 < m.K;
#pragma unroll
            for (int e = 0; e < kShare; ++e) {
                const uint8_t* base = ACT ? (kShare == 8 ? wbase[e / 4] : half ? wbase[ACT ? 1 : 0] : wbase[0]) : wbase[0];
                i32x4 v = {0, 0, 0, 0};
                if (in) v = *reinterpret_cast<const i32x4*>(base + k0 + woff[e]);
                weight[NB == 2 ? buf : 0][group][8 * (half * kShare + e) + cr][lane % 8] = v;
            }
#pragma unroll
            for (int i = 0; i < kRuns; ++i) {
                i32x4 v = {0, 0, 0, 0};
                if (in) v = *reinterpret_cast<const i32x4*>(arow[i] + k0);
                act[buf][(i * kWaves + wave) * 8 + cr][lane % 8] = v;
            }
            if (threadIdx.x < BM) act_scale[buf][threadIdx.x] = ascale[full];
#pragma unroll
            for (int i = 0; i < kScales; ++i) sw[i] = wscale[i][full];
            block_barrier();
            read_weights(NB == 2 ? buf : 0);
            multiply(buf);
        }
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            const int x = half * 16 * TT + j * 16 + r;
            if (x >= rows) continue;
            const int64_t o = pair_of[x] * cols;
#pragma unroll
            for (int t = 0; t < kCols / 16; t += kRun / 4) {
                const int64_t c = c0 + 16 * t + kRun * run;
                float v[kRun];
#pragma unroll
                for (int q = 0; q < kRun; ++q) {
                    v[q] = acc[t + q / 4][j][q % 4];
                    if constexpr (ACT) v[q] = gated_act(m.act, v[q]) * acc[t + q / 4 + 2][j][q % 4];
                }
                if (c + kRun <= cols) {
                    store_run<OUT>(m.out, o + c, v);
                } else {
#pragma unroll
                    for (int q = 0; q < kRun; ++q) {
                        if (c + q < cols) store1<OUT>(m.out, o + c + q, v[q]);
                    }
                }
            }
        }
    }
}

constexpr int64_t kMaxGrid = int64_t(1) << 22;         // workgroups of a launch

template <int CT, int OUT, bool ACT>
int launch_gemv_tile(const Fp8Args& m, hipStream_t s)
{
    const int64_t cols = ACT ? m.N / 2 : m.N;
    const int64_t pairs = m.T * m.top_k, ntiles = (cols + 16 * CT - 1) / (16 * CT);
    const int by_pair = pairs <= m.E + 1;
    const int64_t nb = (m.K + kFp8Block - 1) / kFp8Block, nr = (m.N + kFp8Block - 1) / kFp8Block;
    const int64_t items = (by_pair ? pairs : m.E + 1) * ntiles;
    for (int64_t first = 0; first < items; first += kMaxGrid) {
        const int st = launch("moe_fp8_gemv_kernel", moe_fp8_gemv_kernel<CT, OUT, ACT>, std::min(items - first, kMaxGrid),
                              kGemvThreads, 0, s, m, nb, nr, ntiles, by_pair, first);
        if (st != FTQ_OK) return st;
    }
    return FTQ_OK;
}

template <int OUT, bool ACT>
int launch_gemv(const Fp8Args& m, hipStream_t s)
{
    const int64_t cols = ACT ? m.N / 2 : m.N;
    if (std::min(m.T * m.top_k, m.E) * cols >= kGemvWideFrom) return launch_gemv_tile<2, OUT, ACT>(m, s);
    return launch_gemv_tile<1, OUT, ACT>(m, s);
}

// Tables of tile_m pairs a tile, walked in parts of 16*TT*WT, with a stride if there are more than a launch takes.
template <int TT, int WT, int NB, int OUT, bool ACT, bool EXACT>
int launch_tile(const Fp8Args& m, const GroupedTables& g, int64_t tile_m, int64_t max_tiles, hipStream_t s)
{
    const int subs = (int)(tile_m / (16 * TT * WT));
    const int64_t grid = std::min((max_tiles * subs * g.ntn + kXcds - 1) / kXcds * kXcds, kMaxGrid);
    return launch("moe_fp8_grouped_kernel", moe_fp8_grouped_kernel<TT, WT, NB, OUT, ACT, EXACT>, grid, 64 * kGroups * WT, 0, s, m, g, subs);
}

template <int OUT, bool ACT, bool EXACT>
int launch_grouped(const Fp8Args& m, const GroupedTables& g, int64_t tile_m, int64_t max_tiles, hipStream_t s)
{
    if (tile_m == 32) return launch_tile<2, 1, 2, OUT, ACT, EXACT>(m, g, tile_m, max_tiles, s);
    // The exact form walks tall tiles in parts of 64 pairs (second layer, 8191 tokens uniform: 754 us, 803 in parts
    // of 128 by two waves a weight group).
    if constexpr (!EXACT) {
        if (tile_m == 256) return launch_tile<8, 2, 2, OUT, ACT, EXACT>(m, g, tile_m, max_tiles, s);
    }
    return launch_tile<4, 1, 1, OUT, ACT, EXACT>(m, g, tile_m, max_tiles, s);
}

// Calls f<OUT, ACT>() for the output type and activation of m.
template <typename F>
int dispatch(const Fp8Args& m, F f)
{
    if (m.act != 0) {
        if (m.out_dtype == FTQ_F32) return f.template operator()<FTQ_F32, true>();
        if (m.out_dtype == FTQ_F16) return f.template operator()<FTQ_F16, true>();
        return f.template operator()<FTQ_BF16, true>();
    }
    if (m.out_dtype == FTQ_F32) return f.template operator()<FTQ_F32, false>();
    if (m.out_dtype == FTQ_F16) return f.template operator()<FTQ_F16, false>();
    return f.template operator()<FTQ_BF16, false>();
}

struct GemvCall {
    const Fp8Args& m;
    hipStream_t s;
    template <int OUT, bool ACT> int operator()() const { return launch_gemv<OUT, ACT>(m, s); }
};
struct GroupedCall {
    const Fp8Args& m;
    const GroupedTables& g;
    int64_t tile_m, max_tiles;
    hipStream_t s;
    template <int OUT, bool ACT> int operator()() const
    {
        if constexpr (OUT != FTQ_F32) {
            if (!m.exact) return launch_grouped<OUT, ACT, false>(m, g, tile_m, max_tiles, s);
        }
        return launch_grouped<OUT, ACT, true>(m, g, tile_m, max_tiles, s);
    }
};

}  // namespace

// The GEMV needs no routing tables, which cost the grouped path about 12 us, and
// reads the weights as fast; the grouped path makes the products three to twenty
// times as fast, which counts sooner when the pairs crowd on few experts.  GEMV
// against grouped, pairs evenly spread (all on the same top_k experts), in us:
// 128 experts of 1408 x 2816, 2 pairs an expert 88 / 102 (21 / 30), 4 pairs 106 /
// 108 (39 / 31), 8 pairs 126 / 113; 8 of 28672 x 4096, 2 pairs 162 / 170 (42 / 44),
// 8 pairs 167 / 171 (89 / 50).  Little work in all: 16 of 300 x 512, pairs*N*K =
// 1.6e8, 12 / 22 (24 / 22); 8 of 704 x 1024, 3.7e8, 14 / 25 (30 / 25), 3e9, 94 / 34.
int fp8_select_path(int64_t E, int64_t N, int64_t K, int64_t T, int64_t top_k)
{
    const int64_t pairs = T * top_k;
    if (pairs > kFp8GemvMaxPairs) return FTQ_PATH_GROUPED;
    return pairs <= 2 * E || pairs * N <= 200000000 / K ? FTQ_PATH_GEMV : FTQ_PATH_GROUPED;
}

// Pairs per tile, from the average pairs per expert.  1408 x 2816 weights, 128
// experts, bf16, evenly spread pairs (all on 8 experts): 32 an expert, tiles of 32
// / 64 / 256: 129 (51) / 120 (40) / 139 (53) us; 16 an expert 114 (33) / 114 (34) /
// 134 (52); 96 an expert, 64 / 256: 161 (91) / 161 (104); 128: 187 (106) / 171
// (111); 256: 290 (192) / 269 (165).
int64_t fp8_tile_m(int64_t E, int64_t T, int64_t top_k)
{
    const int64_t per_expert = T * top_k / E;
    return per_expert >= 112 ? 256 : per_expert >= 24 ? 64 : 32;
}

int run_fp8_gemv(const Fp8Args& m, hipStream_t s) { return dispatch(m, GemvCall{m, s}); }

int run_fp8_grouped(const Fp8Args& m, const BucketPlan& plan, const void* ws, hipStream_t s)
{
    const uint8_t* base = static_cast<const uint8_t*>(ws);
    const int64_t cols = m.act ? m.N / 2 : m.N, tile = kGroups * (m.act ? 32 : 64);
    const GroupedTables g{reinterpret_cast<const int32_t*>(base + plan.off_tiles),
                          reinterpret_cast<const int32_t*>(base + plan.off_sorted),
                          reinterpret_cast<const int4*>(base + plan.off_tdesc),
                          (m.K + kFp8Block - 1) / kFp8Block, (m.N + kFp8Block - 1) / kFp8Block, (cols + tile - 1) / tile};
    return dispatch(m, GroupedCall{m, g, plan.tile_m, plan.max_tiles, s});
}

}  // namespace ftq
