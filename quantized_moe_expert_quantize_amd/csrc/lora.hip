// Low-rank adapters of many requests beside a shared projection.  Pair p of adapter
// l (its id; others have none) with row x and scale s_l:
//
//   h[p] = A_l x,   out[p] = base[p] + s_l B_l h[p]
//
// and, from d_out, with g[p] = s_l B_l^T d_out[p],
//
//   d_x = sum over a row's pairs of A_l^T g[p],
//   dA_l = sum over the adapter's pairs of g[p] x^T,   dB_l = s_l * the same of d_out[p] h[p]^T.
//
// Everything is bound by the long rows (x, base, out, d_out, d_x), which are read or
// written once each but for d_out, read for g and for dB; the rank-sized values between
// are small.  Three products, each on the matrix units:
//
//   shrink   [R x C] times a row: rows and weights come through LDS in 128-byte pieces
//            by asynchronous copies several pieces ahead; the row's length is split over
//            workgroups, whose parts the reader adds up in their order;
//   expand   [C x R] times an R-vector, added to base: one pass over the columns;
//   outer    sums over an adapter's pairs of R-vector times row: pairs sorted by adapter
//            (bucket.hip) in tiles of 32, each workgroup a run of tiles and 512 bytes of columns.
//
// A tile of rows may hold several adapters: shrink and expand go through them one by
// one, each time for the whole tile, and keep each row's results of its own adapter
// alone, so that no row ever sees another's weights.  An adapter's R-vectors are fp32.
// As operands beside 16-bit weights or rows they are the sum of three bf16 pieces of 8 bits
// each, which have fp32's range and, together, its 24 bits whatever else lies in the
// vector.  bf16 weights and rows are multiplied by every piece; fp16 ones are the sum of two bf16
// operands (8 bits and the remaining 3), six products in all.  Each product is exact and
// summed in fp32.  (fp16 with two fp16 pieces under one power of two: gradients of 8192 rows at rank 64 in 128 us,
// 151 so, 8191 rows at rank 32 in 58, 60 so; but ranks or pairs at 2^-24 of the largest beside
// them were 1e-4 of their size off, and an infinity took the bits of the others.)
#include <type_traits>

#include "ftq_internal.h"
#include "lds_copy.h"

namespace ftq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kLine = 128;                             // bytes of a row in one piece

template <int DT> constexpr int kSize = DT == FTQ_F32 ? 4 : 2;
template <int DT> constexpr int kPieces = DT == FTQ_F32 ? 1 : 3;   // of an R-vector's value
template <int DT> constexpr int kParts = DT == FTQ_F16 ? 2 : 1;     // of a weight or a row's value beside them

__device__ const u32x4 kZeros = {0u, 0u, 0u, 0u};      // what a copy reads in place of what is not there

__device__ __forceinline__ bool adapter_ok(int32_t id, int32_t L) { return id >= 0 && id < L; }

// 16 rows x 16 columns += 64 bytes of 16 rows on either side.  Lane l holds 16 bytes of
// row l%16 of each operand, and results 4*(l/16) .. +3 of the left's rows for row l%16
// of the right.  (fp32: four instructions, one element of every lane's each; the order
// of the products within the 64 bytes does not matter while both sides have the same.)
template <int DT>
__device__ __forceinline__ f32x4 multiply(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (DT == FTQ_F16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    } else if constexpr (DT == FTQ_BF16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    } else {
        const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], c, 0, 0, 0);
        return c;
    }
}

// Of 16 lanes, each naming 8 bytes (four 16-bit values), four lanes a row: lane l gets value l of the four rows.
__device__ __forceinline__ u32x2 read_transposed(const uint8_t* lds)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)lds));
}

// The next bf16 piece of v: its first 8 significant bits; v becomes what is left of it.
__device__ __forceinline__ uint32_t take_piece(float& v)
{
    const uint32_t top = __builtin_bit_cast(uint32_t, v) & 0xffff0000u;
    v -= __builtin_bit_cast(float, top);
    return top >> 16;
}

// An operand of weights or rows as those that the pieces are multiplied by: itself, or, of fp16, two of bf16 whose
// sum it is.  (Of an infinity the second is a NaN.)
template <int DT>
__device__ __forceinline__ void split_operand(u32x4 w, u32x4 (&part)[kParts<DT>])
{
    if constexpr (DT != FTQ_F16) {
        part[0] = w;
    } else {
        const auto two = [](f16x2 h) {                 // values of at most 8 significant bits: the upper halves of their floats
            return __builtin_bit_cast(uint32_t, (float)h[0]) >> 16 | (__builtin_bit_cast(uint32_t, (float)h[1]) & 0xffff0000u);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f16x2 top = __builtin_bit_cast(f16x2, w[i] & 0xfff8fff8u);
            part[0][i] = two(top);
            part[1][i] = two(__builtin_bit_cast(f16x2, (uint32_t)w[i]) - top);
        }
    }
}

// 16 rows x 16 columns += weights or rows (their parts) times 64 bytes of R-vectors (their pieces).
template <int DT>
__device__ __forceinline__ f32x4 multiply_pieces(const u32x4 (&part)[kParts<DT>], const u32x4 (&piece)[kPieces<DT>], f32x4 c)
{
#pragma unroll
    for (int i = 0; i < kPieces<DT>; ++i) {
#pragma unroll
        for (int h = 0; h < kParts<DT>; ++h) c = multiply<DT == FTQ_F16 ? FTQ_BF16 : DT>(part[h], piece[i], c);
    }
    return c;
}

// ---- tiles of pairs --------------------------------------------------------------
//
// Without tables a tile is BM pairs in their order, of whatever adapters.  With the tables of
// pairs sorted by adapter (bucket.hip) it is `span` table tiles in a row, each of one adapter.

struct TileList {
    const int32_t* sorted;     // or null: no tables
    const int4* tdesc;         // per table tile {adapter (L: none), first slot, pairs, 0}
    const int32_t* count;      // number of table tiles
    int32_t span;
    int32_t rows;              // pairs of a tile at most
    int64_t most;              // tiles at most
};

// First slot and pairs of tile i (no pairs behind the last tile).
template <int BM>
__device__ __forceinline__ void find_tile(const TileList& t, int64_t i, int64_t pairs, int64_t& slot0, int& rows)
{
    if (!t.sorted) {
        slot0 = i * BM;
        rows = (int)min((int64_t)BM, pairs - slot0);
        return;
    }
    const int64_t n = uniform(*t.count), t0 = i * t.span;
    slot0 = 0;
    rows = 0;
    if (t0 >= n) return;
    const int4 d0 = t.tdesc[t0], d1 = t.tdesc[min(t0 + t.span, n) - 1];
    slot0 = uniform(d0.y);
    rows = uniform(d1.y) + uniform(d1.z) - uniform(d0.y);
}

// ---- shrink: z[p] = W_l v[row of p] ---------------------------------------------

struct ShrinkArgs {
    const uint8_t* v;          // rows
    int64_t ldv;               // bytes from row to row
    const uint8_t* w;          // [L][R][C], or [L][C][R] (by_column)
    const int32_t* ids;        // [pairs]
    TileList tiles;
    float* part;               // [splits][pairs][R]
    int64_t pairs, row_bytes;  // bytes of C elements
    int32_t div, L, R;
    int32_t splits, steps;     // 128-byte steps of a split
    int32_t groups;            // workgroups that share a tile's adapters
};

constexpr int kDepth = 4;      // pieces in LDS: one is multiplied while three are on their way

// A workgroup takes 16 rows a wave.  LDS: run c (16 bytes) of row x sits at c ^ (x % 8).
// COLS: the weights lie by column, [C][R].  A piece of them is then as many rows of R values
// as it has columns (rows padded to 16*RT), and a lane collects its columns' values of one
// rank, in 16 bits by transposing reads of four columns x 16 ranks.  The columns' places and
// runs are permuted so that the 16 columns of such a read lie side by side and meet no bank twice.
template <int DT, int WAVES, int RT, bool COLS>
__global__ __launch_bounds__(64 * WAVES) void lora_shrink_kernel(ShrinkArgs m, int64_t first_item)
{
    constexpr int kRuns = RT * kSize<DT>;                          // 16-byte runs of a column's ranks
    constexpr int kSpread = RT == 8 ? 0 : RT == 4 ? 1 : RT == 2 ? 2 : 3;
    static_assert(kLine / kSize<DT> * kRuns == 128 * RT);
    const auto run_at = [](int place, int run) { return DT == FTQ_F32 ? run : run ^ (((place >> kSpread) & (RT - 1)) << 1); };
    constexpr int BM = 16 * WAVES;
    constexpr int kW = 2 * RT, kShare = (kW + WAVES - 1) / WAVES;   // copies of the weights' rows: in all, and a wave's
    constexpr int kPer = 2 + kShare;                               // copies of a wave and step
    __shared__ u32x4 xs[kDepth][BM][8];
    __shared__ u32x4 ws[kDepth][16 * RT][8];
    const int lane = threadIdx.x & 63, wave = uniform((int32_t)(threadIdx.x >> 6));
    const int r16 = lane & 15, q = lane >> 4;
    const int64_t item = first_item + blockIdx.x, at = item / m.splits;
    const int ks = (int)(item - at * m.splits), g = (int)(at % m.groups);
    int64_t slot0;
    int rows;
    find_tile<BM>(m.tiles, at / m.groups, m.pairs, slot0, rows);
    if (rows == 0) return;
    // lane i: row i of the tile
    int32_t pair = 0, id = -1;
    if (lane < rows) {
        pair = m.tiles.sorted ? m.tiles.sorted[slot0 + lane] : (int32_t)(slot0 + lane);
        id = m.ids[pair];
        if (!adapter_ok(id, m.L)) id = -1;
    }
    uint64_t todo = __ballot(id >= 0);
    const int cr = lane >> 3, run = (lane & 7) ^ cr;               // row of eight and 16-byte run that this lane copies
    const uint8_t* xsrc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = (wave * 2 + i) * 8 + cr;
        xsrc[i] = m.v + (int64_t)(__shfl(pair, min(row, rows - 1)) / m.div) * m.ldv;
        if (row >= rows) xsrc[i] = nullptr;
    }
    const int64_t total = (m.row_bytes + kLine - 1) / kLine, first = (int64_t)ks * m.steps, columns = m.row_bytes / kSize<DT>;
    const int n = (int)max((int64_t)0, min((int64_t)m.steps, total - first));
    const int32_t my_pair = __shfl(pair, wave * 16 + r16);
    for (int index = 0; todo; ++index) {
        const int32_t l = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
        const uint64_t mine = __ballot(id == l);
        todo &= ~mine;
        if (index % m.groups != g) continue;
        const uint8_t* wsrc[kShare];
        int col[kShare];                                           // COLS: the column of a step's that this lane copies a run of, or none (a large one)
#pragma unroll
        for (int i = 0; i < kShare; ++i) {
            const int part = (wave + i * WAVES) % kW;
            if constexpr (COLS) {
                const int at = part * 64 + lane, place = at / kRuns, run_w = run_at(place, at % kRuns);
                // place = 32h + 16a + 4b + c of 16-bit columns 32h + 8b + 4a + c, 16h + 4b + a of 32-bit ones 16h + 4a + b
                col[i] = DT == FTQ_F32 ? (place & 16) + 4 * (place & 3) + ((place >> 2) & 3) : (place & 32) + 8 * ((place >> 2) & 3) + 4 * ((place >> 4) & 1) + (place & 3);
                wsrc[i] = m.w + ((int64_t)l * columns + col[i]) * m.R * kSize<DT> + run_w * 16;
                if (run_w * 16 >= m.R * kSize<DT>) col[i] = INT32_MAX;
            } else {
                wsrc[i] = m.w + ((int64_t)l * m.R + min(part * 8 + cr, m.R - 1)) * m.row_bytes;
            }
        }
        const auto copy_step = [&](int s) {
            const int64_t byte = (first + s) * kLine + run * 16;
            const bool in = byte < m.row_bytes;
            const uint8_t* none = reinterpret_cast<const uint8_t*>(&kZeros);
            const int buf = s % kDepth;
#pragma unroll
            for (int i = 0; i < 2; ++i) copy16(lds_address(&xs[buf][(wave * 2 + i) * 8][0]), in && xsrc[i] ? xsrc[i] + byte : none);
#pragma unroll
            for (int i = 0; i < kShare; ++i) {
                const uint8_t* src = in ? wsrc[i] + byte : none;
                if constexpr (COLS) {
                    const int64_t c = (first + s) * (kLine / kSize<DT>);
                    src = col[i] < columns - c ? wsrc[i] + c * m.R * kSize<DT> : none;
                }
                copy16(lds_address(&ws[buf][(wave + i * WAVES) % kW * 8][0]), src);
            }
        };
        f32x4 acc[RT] = {};
        block_barrier();                                           // the last adapter's pieces have been read
        settle();
        for (int s = 0; s < kDepth - 1 && s < n; ++s) copy_step(s);
        for (int s = 0; s < n; ++s) {
            if (n - 1 - s >= 2) wait_copies_but<2 * kPer>();
            else if (n - 1 - s == 1) wait_copies_but<kPer>();
            else wait_copies();
            block_barrier();                                       // all waves' copies of step s are there, step s - 1 has been read
            if (s + kDepth - 1 < n) copy_step(s + kDepth - 1);
            const int buf = s % kDepth;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4 x = xs[buf][wave * 16 + r16][(4 * h + q) ^ (r16 & 7)];
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    u32x4 w;
                    if constexpr (!COLS) {
                        w = ws[buf][16 * i + r16][(4 * h + q) ^ (r16 & 7)];
                    } else {
                        const uint8_t* base = reinterpret_cast<const uint8_t*>(&ws[buf][0][0]);
                        if constexpr (DT == FTQ_F32) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const uint32_t*>(base + ((16 * h + 4 * e + q) * kRuns * 16 + (16 * i + r16) * 4));
                        } else {
#pragma unroll
                            for (int a = 0; a < 2; ++a) {
                                const int place = 32 * h + 16 * a + 4 * q + (r16 >> 2);
                                const u32x2 t = read_transposed(base + (place * kRuns + run_at(place, 2 * i + ((r16 & 3) >> 1))) * 16 + (r16 & 1) * 8);
                                w[2 * a] = t[0];
                                w[2 * a + 1] = t[1];
                            }
                        }
                    }
                    acc[i] = multiply<DT>(w, x, acc[i]);
                }
            }
        }
        if (mine >> (wave * 16 + r16) & 1) {
            float* z = m.part + ((int64_t)ks * m.pairs + my_pair) * m.R;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                if (16 * i + 4 * q < m.R) *reinterpret_cast<f32x4*>(z + 16 * i + 4 * q) = acc[i];
            }
        }
    }
}

// ---- expand: out[row] = base[row] + f_l * W_l z[p] ---------------------------------

struct ExpandArgs {
    const float* part;         // [splits][pairs][R]
    const uint8_t* w;          // [L][C][R], or [L][R][C] (by rank)
    const float* scale;        // [L] or null
    const int32_t* ids;
    TileList tiles;
    const void* base;          // or null
    void* out;
    float* h;                  // [pairs][R] or null: the sum of the parts
    int64_t ld_base, ld_out, pairs, C;
    int32_t L, R, splits, groups;
    int64_t col_items;         // workgroups along the columns
    int32_t cols;              // columns of a workgroup, whole steps
};

template <int DT> __device__ __forceinline__ float load1(const void* p, int64_t i)
{
    if constexpr (DT == FTQ_F32) return static_cast<const float*>(p)[i];
    else return DT == FTQ_F16 ? f32_of_f16(static_cast<const uint16_t*>(p)[i]) : f32_of_bf16(static_cast<const uint16_t*>(p)[i]);
}

// N consecutive results v added to 16 bytes of base, rounded to OT and stored; PAST: past the caches, as long results
// are that would drive out the rows other workgroups are about to read (8191 rows of 4096 in bf16, their shrink and expand
// 62 us, 60 so).
template <int OT, bool PAST, int N>
__device__ __forceinline__ void add_and_store(void* out, int64_t i, u32x4 base, const float (&v)[N])
{
    if constexpr (OT == FTQ_F32) {
        static_assert(N == 4);
        f32x4 b = __builtin_bit_cast(f32x4, base);
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] += v[e];
        f32x4* to = reinterpret_cast<f32x4*>(static_cast<float*>(out) + i);
        if constexpr (PAST) __builtin_nontemporal_store(b, to);
        else *to = b;
    } else {
        static_assert(N == 8);
        u32x4 r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint16_t lo = (uint16_t)base[e], hi = (uint16_t)(base[e] >> 16);
            if constexpr (OT == FTQ_F16) {
                r[e] = f16_of_f32(f32_of_f16(lo) + v[2 * e]) | (uint32_t)f16_of_f32(f32_of_f16(hi) + v[2 * e + 1]) << 16;
            } else {
                r[e] = bf16_of_f32(f32_of_bf16(lo) + v[2 * e]) | (uint32_t)bf16_of_f32(f32_of_bf16(hi) + v[2 * e + 1]) << 16;
            }
        }
        u32x4* to = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + i);
        if constexpr (PAST) __builtin_nontemporal_store(r, to);
        else *to = r;
    }
}

// The value of the lane beside this one (0 and 1, 2 and 3, ...).
__device__ __forceinline__ float swap_pair(float v)
{
    const int i = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, 0xB1, 0xF, 0xF, false));   // quad_perm 1 0 3 2
}

// A wave takes 16 pairs, whose R-vectors it holds in registers as operands, and streams 64
// columns at a time: base (the next columns' is on its way), results, and the weights.  WR == 4:
// the waves of a workgroup have 16 pairs each and the same columns, whose weights they bring
// into LDS in the order they lie, a step ahead in registers.  WR == 1: the same 16 pairs and 64
// columns of 256 each, and every wave loads its weights as operands: for few pairs, which
// cost time by the length of their chain of loads.  (Weights loaded so by each wave of many, a column a lane, took as many
// address cycles as base and results together: 34 to 46 us where a copy of the same rows takes 21.)
// W is the left operand, so that a lane holds four columns of one row; which row of a 16-row tile is
// which column is free and chosen so that a lane's results are whole 16-byte runs and
// the four lanes of a row have 64 bytes side by side: 32-bit results, row r of tile i is column
// 16*i + r; 16-bit ones, column 32*(i/2) + 8*(r/4) + 4*(i%2) + r%4.  Lanes of neighbouring
// rows then trade a run each, so that eight lanes read and write the 128 bytes of a line of one row.
// KST: 64-byte steps of an R-vector.  RANKS: the weights lie by rank, [R][C], also in LDS, and
// 16-bit ones are read by transposing reads of four ranks x 16 columns.
template <int DT, int OT, int KST, bool RANKS, int WR>
__global__ __launch_bounds__(kThreads) void lora_expand_kernel(ExpandArgs m, int64_t first_item)
{
    constexpr int kElems = 64 / kSize<DT>, kOwn = 16 / kSize<DT>;  // ranks of a step, and a lane's of them
    constexpr bool kWide = OT == FTQ_F32;
    constexpr int kRun = kWide ? 4 : 8, kLines = 64 / (8 * kRun);  // columns of a lane's store, 128-byte lines of a row and wave
    constexpr int BM = 16 * WR, kCols = 256 / WR;                  // pairs of a workgroup, columns of its step
    // LDS rows: a column's ranks or a rank's columns, set apart by 16 bytes where they would meet the same banks
    constexpr int kRow = RANKS ? kCols * kSize<DT> : 64 * KST, kPitch = kRow + (RANKS || KST > 1 ? 16 : 0);
    constexpr int kRowsLds = RANKS ? kElems * KST : kCols, kPlane = kRowsLds * kPitch;   // a part's bytes
    constexpr int kUnits = kRow / 16 * kRowsLds / kThreads;        // 16-byte runs of a thread
    static_assert(kRow / 16 * kRowsLds % kThreads == 0);
    constexpr bool kLds = WR == 4;
    static_assert(kLds || !RANKS);
    __shared__ __attribute__((aligned(16))) uint8_t wl[kLds ? kParts<DT> * kPlane : 16];
    const int lane = threadIdx.x & 63, wave = uniform((int32_t)(threadIdx.x >> 6)), r16 = lane & 15, q = lane >> 4;
    const bool odd = r16 & 1;
    const int64_t item = first_item + blockIdx.x, at = item / m.col_items;
    const int64_t c_first = (item - at * m.col_items) * m.cols, c_end = min(c_first + m.cols, m.C);
    const int g = (int)(at % m.groups);
    int64_t slot0;
    int rows;
    find_tile<BM>(m.tiles, at / m.groups, m.pairs, slot0, rows);
    if (rows == 0) return;
    // lane i: row i of the tile
    int32_t tile_pair = 0, tile_id = INT32_MIN;                    // rows that are not there
    if (lane < rows) {
        tile_pair = m.tiles.sorted ? m.tiles.sorted[slot0 + lane] : (int32_t)(slot0 + lane);
        tile_id = m.ids[tile_pair];
        if (!adapter_ok(tile_id, m.L)) tile_id = -1;
    }
    const int row0 = WR == 1 ? 0 : 16 * wave, col0 = WR == 1 ? 64 * wave : 0;   // of this wave
    const int32_t pair = __shfl(tile_pair, row0 + r16);
    // this lane's row and its neighbour's, the even one first
    const uint8_t* from[2];
    uint8_t* to[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        const int64_t p = __shfl(tile_pair, row0 + (r16 & 14) + z);
        from[z] = static_cast<const uint8_t*>(m.base) + (p * m.ld_base + col0 + odd * 4 * kRun + q * kRun) * kSize<OT>;
        to[z] = static_cast<uint8_t*>(m.out) + (p * m.ld_out + col0 + odd * 4 * kRun + q * kRun) * kSize<OT>;
    }
    // runs of the weights that this thread brings: of rank or column `row` the run `part`; ranks from R on stay zero
    const int per_row = RANKS ? kRow / 16 : m.R * kSize<DT> / 16, have = RANKS ? m.R * per_row : kCols * per_row;
    int row_of[kUnits], part_of[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits && kLds; ++i) {
        const int u = i * kThreads + threadIdx.x;
        row_of[i] = u < have ? u / per_row : INT32_MAX;
        part_of[i] = u % per_row;
    }
    if (kLds && have < kUnits * kThreads) {
        for (int i = threadIdx.x; i < kParts<DT> * kPlane / 16; i += kThreads) *reinterpret_cast<u32x4*>(wl + 16 * i) = u32x4{0u, 0u, 0u, 0u};
    }
    uint64_t todo = __ballot(tile_id != INT32_MIN);
    for (int index = 0; todo; ++index) {
        const int32_t l = __builtin_amdgcn_readlane(tile_id, __builtin_ctzll(todo));
        const uint64_t all = __ballot(tile_id == l);
        todo &= ~all;
        if (index % m.groups != g) continue;
        const uint32_t mine = (uint32_t)(all >> row0) & 0xffff;    // of this wave's rows
        const bool own[2] = {(mine >> (r16 & 14) & 1) != 0, (mine >> (r16 | 1) & 1) != 0};
        // line t: the even lanes of a pair take its first half, the odd ones its second, of the even row, then the odd one
        const auto there = [&](int64_t c0, int t) { return c0 + col0 + (2 * t + odd) * 4 * kRun + q * kRun < c_end; };
        const auto load_base = [&](int64_t c0, u32x4 (&b)[kLines][2]) {
#pragma unroll
            for (int t = 0; t < kLines; ++t) {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    if (m.base && own[z] && there(c0, t)) b[t][z] = *reinterpret_cast<const u32x4*>(from[z] + (c0 + t * 8 * kRun) * kSize<OT>);
                }
            }
        };
        const auto column = [&](int i) { return col0 + (kWide ? 16 * i + r16 : 32 * (i / 2) + 8 * (r16 / 4) + 4 * (i % 2) + r16 % 4); };   // of a weight tile's row
        u32x4 ahead[kLds ? kUnits : 4 * KST] = {};
        const auto load_weights = [&](int64_t c0) {
            if (l < 0) return;
            if constexpr (!kLds) {                                 // each lane its own operand
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t c = min(c0 + column(i), m.C - 1);
#pragma unroll
                    for (int k = 0; k < KST; ++k) {
                        const int r = k * kElems + q * kOwn;
                        if (r >= m.R) continue;                    // (R is a multiple of 8: all of a lane's ranks are there or none)
                        ahead[i * KST + k] = *reinterpret_cast<const u32x4*>(m.w + (((int64_t)l * m.C + c) * m.R + r) * kSize<DT>);
                    }
                }
                return;
            }
#pragma unroll
            for (int i = 0; i < (kLds ? kUnits : 0); ++i) {
                if constexpr (RANKS) {
                    if (row_of[i] < m.R && c0 + part_of[i] * kOwn < m.C)
                        ahead[i] = *reinterpret_cast<const u32x4*>(m.w + (((int64_t)l * m.R + row_of[i]) * m.C + c0) * kSize<DT> + part_of[i] * 16);
                } else {
                    if (row_of[i] < m.C - c0) ahead[i] = *reinterpret_cast<const u32x4*>(m.w + (((int64_t)l * m.C + c0 + row_of[i]) * m.R) * kSize<DT> + part_of[i] * 16);
                }
            }
        };
        u32x4 base[kLines][2] = {}, base_next[kLines][2] = {};
        load_weights(c_first);
        load_base(c_first, base);
        // the R-vectors of this adapter's rows (zeros for others) as operands
        u32x4 z[KST][kPieces<DT>];
        {
            const float scale = l >= 0 && m.scale ? m.scale[l] : 1.0f;
            const bool take = mine >> r16 & 1;
            f32x4 v[KST][kOwn / 4];
#pragma unroll
            for (int k = 0; k < KST; ++k) {
#pragma unroll
                for (int h = 0; h < kOwn / 4; ++h) {
                    const int r = k * kElems + q * kOwn + 4 * h;
                    v[k][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                    if (take && r < m.R) {
                        const int64_t o = (int64_t)pair * m.R + r;
                        if (l >= 0) {
#pragma unroll(WR == 1 ? 8 : 1)
                            for (int i = 0; i < m.splits; ++i) v[k][h] += *reinterpret_cast<const f32x4*>(m.part + i * m.pairs * m.R + o);
                        }
                        if (m.h && c_first == 0 && (WR == 4 || wave == 0)) *reinterpret_cast<f32x4*>(m.h + o) = v[k][h];
                        v[k][h] *= scale;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < KST; ++k) {
                if constexpr (DT == FTQ_F32) {
                    z[k][0] = __builtin_bit_cast(u32x4, v[k][0]);
                } else {
#pragma unroll
                    for (int c = 0; c < kPieces<DT>; ++c) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float lo = v[k][e / 2][e % 2 * 2], hi = v[k][e / 2][e % 2 * 2 + 1];
                            const uint32_t piece = take_piece(lo);
                            z[k][c][e] = piece | take_piece(hi) << 16;
                            v[k][e / 2][e % 2 * 2] = lo;
                            v[k][e / 2][e % 2 * 2 + 1] = hi;
                        }
                    }
                }
            }
        }
        for (int64_t c0 = c_first; c0 < c_end; c0 += kCols) {
            if constexpr (kLds) {
                block_barrier();                                   // the last step's weights have been read
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    if (row_of[i] == INT32_MAX) continue;
                    u32x4 w[kParts<DT>];
                    split_operand<DT>(ahead[i], w);                // once for the workgroup (by each wave: 8192 rows, rank 64, 4096 columns 58 us, 46 so)
#pragma unroll
                    for (int h = 0; h < kParts<DT>; ++h) *reinterpret_cast<u32x4*>(wl + h * kPlane + row_of[i] * kPitch + part_of[i] * 16) = w[h];
                }
                if (c0 + kCols < c_end) load_weights(c0 + kCols);
            }
            if (c0 + kCols < c_end) load_base(c0 + kCols, base_next);
            if constexpr (kLds) block_barrier();
            if (mine && c0 + col0 < c_end && (l >= 0 || m.base != m.out)) {   // (in place, rows without an adapter stay as they are)
                f32x4 acc[4] = {};
#pragma unroll
                for (int k = 0; k < KST; ++k) {
                    if (l < 0) continue;                           // no adapter, no weights: what LDS holds may be anything
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        u32x4 w[kParts<DT>];
                        if constexpr (!kLds) split_operand<DT>(ahead[i * KST + k], w);
#pragma unroll
                        for (int p = 0; p < (kLds ? kParts<DT> : 0); ++p) {
                            const uint8_t* plane = wl + p * kPlane;
                            if constexpr (!RANKS || DT == FTQ_F32) {
                                const int c = column(i);
                                if constexpr (!RANKS) {
                                    w[p] = *reinterpret_cast<const u32x4*>(plane + c * kPitch + k * 64 + q * 16);
                                } else {
#pragma unroll
                                    for (int e = 0; e < 4; ++e) w[p][e] = *reinterpret_cast<const uint32_t*>(plane + (k * kElems + 4 * q + e) * kPitch + c * 4);
                                }
                            } else {
                                // columns four by four, as lanes 4j .. 4j+3 of a result hold them
                                const int c = col0 + (kWide ? 16 * i + 4 * (r16 & 3) : 32 * (i / 2) + 8 * (r16 & 3) + 4 * (i % 2));
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const u32x2 t = read_transposed(plane + (k * kElems + 8 * q + 4 * h + (r16 >> 2)) * kPitch + c * 2);
                                    w[p][2 * h] = t[0];
                                    w[p][2 * h + 1] = t[1];
                                }
                            }
                        }
                        acc[i] = multiply_pieces<DT>(w, z[k], acc[i]);
                    }
                }
#pragma unroll
                for (int t = 0; t < kLines; ++t) {
                    float v[2][kRun];                              // of the even row, of the odd one
#pragma unroll
                    for (int e = 0; e < kRun; ++e) {
                        const float first = kWide ? acc[2 * t][e % 4] : acc[e / 4][e % 4];
                        const float second = kWide ? acc[2 * t + 1][e % 4] : acc[2 + e / 4][e % 4];
                        const float got = swap_pair(odd ? first : second);
                        v[0][e] = odd ? got : first;
                        v[1][e] = odd ? second : got;
                    }
#pragma unroll
                    for (int z2 = 0; z2 < 2; ++z2) {
                        if (own[z2] && there(c0, t)) add_and_store<OT, WR == 4>(to[z2] + (c0 + t * 8 * kRun) * kSize<OT>, 0, base[t][z2], v[z2]);
                    }
                }
            }
            if (!kLds && c0 + kCols < c_end) load_weights(c0 + kCols);
#pragma unroll
            for (int t = 0; t < kLines; ++t) {
#pragma unroll
                for (int z2 = 0; z2 < 2; ++z2) base[t][z2] = base_next[t][z2];
            }
        }
    }
}

// ---- d_x of rows that several pairs share -----------------------------------------
//
// d_x[t] = base[t] + sum over the pairs of t of A_l^T g[p]: a pair's adapter is its own, so
// nothing is shared but A in the caches, and the vector units do it: a wave takes a
// token and 16 bytes of columns a lane, g comes in scalar registers.  Workgroups of an XCD
// work on the same columns, so that its L2 holds them of all adapters.

struct GatherArgs {
    const float* g;            // [T*k][R]
    const uint8_t* a;          // [L][R][C]
    const int32_t* ids;
    const uint8_t* base;       // or null
    uint8_t* out;
    int64_t T, C, slices, groups;
    int32_t L, R, k;
};

constexpr int kXcds = 8, kGatherTokens = 4;            // tokens of a workgroup, one a wave

template <int DT>
__global__ __launch_bounds__(kThreads) void lora_gather_kernel(GatherArgs m, int64_t first_item)
{
    constexpr int kCols = 16 / kSize<DT>;
    const int lane = threadIdx.x & 63, wave = uniform((int32_t)(threadIdx.x >> 6));
    const int64_t total = m.slices * m.groups, per = (total + kXcds - 1) / kXcds;
    const int64_t at = first_item + blockIdx.x, item = at % kXcds * per + at / kXcds;   // (first_item: whole rounds of the XCDs)
    if (item >= total || at / kXcds >= per) return;
    const int64_t slice = item / m.groups, t = (item - slice * m.groups) * kGatherTokens + wave;
    const int64_t c = slice * 64 * kCols + lane * kCols;
    if (t >= m.T || c >= m.C) return;
    float acc[kCols] = {};
    for (int j = 0; j < m.k; ++j) {
        const int64_t p = t * m.k + j;
        const int32_t l = uniform(m.ids[p]);
        if (!adapter_ok(l, m.L)) continue;
        const float* g = m.g + p * m.R;
        const uint8_t* a = m.a + ((int64_t)l * m.R * m.C + c) * kSize<DT>;
        for (int r = 0; r < m.R; r += 8) {
            u32x4 row[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) row[e] = *reinterpret_cast<const u32x4*>(a + (r + e) * m.C * kSize<DT>);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = g[r + e];
#pragma unroll
                for (int i = 0; i < kCols; ++i) acc[i] = __builtin_fmaf(f, load1<DT>(&row[e], i), acc[i]);
            }
        }
    }
    u32x4 base = {0u, 0u, 0u, 0u};
    const int64_t o = (t * m.C + c) * kSize<DT>;
    if (m.base) base = *reinterpret_cast<const u32x4*>(m.base + o);
    add_and_store<DT, false>(m.out + o, 0, base, acc);
}

// ---- outer: d[l] = sum over its pairs of u[p] v[row of p]^T -----------------------------
//
// The pairs are sorted by adapter and cut into tiles of 32 of one adapter.  lora_pieces
// writes the R-vectors of a tile in the order that the products take them, u^T in its
// pieces: [tile][piece][16*RT][32].  A workgroup takes `run` tiles in a row and 512 bytes
// of columns; where the adapter changes it writes its sums: to the result if all the
// adapter's tiles are its own, else to part 2c (the adapter began before run c) or
// 2c + 1, and lora_reduce adds an adapter's parts in their order.

constexpr int kTile = 32;

struct OuterTables {
    const int32_t* tiles;      // [L + 2] first tile of each adapter; the last entry is their number
    const int32_t* sorted;
    const int4* tdesc;         // per tile {adapter (L: none), first slot, pairs, 0}
};

struct PiecesArgs {
    const float* part;         // [splits][pairs][R]
    const float* scale;        // [L] or null
    float* sum;                // [pairs][R] or null: the sum of the parts
    void* u;                   // [tiles][kPieces][16*RT][32]
    int64_t pairs, max_tiles;
    int32_t L, R, splits;
};

// One workgroup per tile (of either set of vectors): thread h has pair h%32 and every eighth group of four ranks from h/32 on.
template <int DT, int RT>
__global__ __launch_bounds__(kThreads) void lora_pieces_kernel(OuterTables tab, PiecesArgs a0, PiecesArgs a1, int64_t first_item)
{
    constexpr int kQuads = 4 * RT, kMine = (kQuads + 7) / 8;
    const int64_t item = first_item + blockIdx.x;
    const bool second = item >= a0.max_tiles;
    const PiecesArgs m = second ? a1 : a0;
    const int64_t t = second ? item - a0.max_tiles : item;
    if (t >= tab.tiles[m.L + 1]) return;
    const int4 d = tab.tdesc[t];
    const int s = threadIdx.x % kTile, q0 = threadIdx.x / kTile;
    const bool have = s < d.z;
    const int64_t p = have ? tab.sorted[d.y + s] : 0;
    const bool none = d.x >= m.L;
    const float scale = !none && m.scale ? m.scale[d.x] : 1.0f;
    f32x4 z[kMine] = {};
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int r = (q0 + 8 * i) * 4;
        if (have && r < m.R) {
            if (!none) {
#pragma unroll 4
                for (int k = 0; k < m.splits; ++k) z[i] += *reinterpret_cast<const f32x4*>(m.part + (k * m.pairs + p) * m.R + r);
            }
            z[i] *= scale;
            if (m.sum) *reinterpret_cast<f32x4*>(m.sum + p * m.R + r) = z[i];
        }
    }
    if (none || !m.u) return;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int r = (q0 + 8 * i) * 4;
        if (r >= 16 * RT) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (DT == FTQ_F32) {
                static_cast<float*>(m.u)[(t * 16 * RT + r + e) * kTile + s] = z[i][e];
            } else {
                float v = z[i][e];
#pragma unroll
                for (int c = 0; c < kPieces<DT>; ++c) static_cast<uint16_t*>(m.u)[((t * kPieces<DT> + c) * 16 * RT + r + e) * kTile + s] = (uint16_t)take_piece(v);
            }
        }
    }
}

struct OuterArgs {
    const uint8_t* u;          // as lora_pieces writes it
    const uint8_t* v;          // rows
    int64_t ldv;               // bytes
    float* part;               // [2 * runs][16*RT * C] (or C * R, as the result)
    float* d;                  // result: [L][R][C], or [L][C][R] with by_column
    int64_t C, col_items, items;
    int32_t div, L, R, by_column;
    int32_t run;               // tiles of a workgroup
    const float* scale;        // [L]: what an adapter's sums are multiplied by, or null (1)
};

constexpr int kBatch = 32;                             // tiles listed in LDS
// Tiles in LDS: as many as let two workgroups onto a CU, or one of the highest ranks.  (8192 rows of 4096 columns, rank
// 64: 41 us with two tiles and two workgroups, 48 to 56 with four or five tiles and one.)
template <int RT> constexpr int kOuterDepth = RT == 4 ? 2 : 3;

// Waits until at most `left` (uniform, below D - 1) of the steps copied after the next one are in flight, PER copies each.
template <int PER, int D>
__device__ __forceinline__ void wait_step(int left)
{
    if constexpr (D > 0) {
        if (left >= D) wait_copies_but<PER * D>();
        else wait_step<PER, D - 1>(left);
    } else {
        wait_copies();
    }
}

template <int DT, int RT>
__global__ __launch_bounds__(kThreads) void lora_outer_kernel(OuterTables tab, OuterArgs a0, OuterArgs a1, int64_t first_item)
{
    constexpr int kCols = 512 / kSize<DT>, kTiles = kCols / 64;    // columns of a workgroup, 16-column tiles of a wave
    constexpr int kULine = kTile * kSize<DT>;                      // bytes of a rank's row of u
    constexpr int kUBytes = kPieces<DT> * 16 * RT * kULine;        // of a tile, whole copies of 1024
    constexpr int kDeep = kOuterDepth<RT>;
    constexpr int kU = kUBytes / 1024, kUShare = (kU + 3) / 4, kPer = 4 + kUShare;
    static_assert(kUBytes % 1024 == 0);
    __shared__ __attribute__((aligned(16))) uint8_t vs[kDeep][kTile][512];
    __shared__ __attribute__((aligned(16))) uint8_t us[kDeep][kUBytes];
    __shared__ int32_t row_lds[kBatch * kTile], id_lds[kBatch + 1];
    __shared__ float scale_lds[kBatch];
    const int64_t at_item = first_item + blockIdx.x;
    const bool second = at_item >= a0.items;
    // (field by field: a selected struct would be read from memory in the loop, and such a read waits for the copies)
    const struct { const uint8_t *u, *v; float *part, *d; int64_t ldv, C, col_items; int32_t div, L, R, by_column, run; const float* scale; } m = {
        second ? a1.u : a0.u, second ? a1.v : a0.v, second ? a1.part : a0.part, second ? a1.d : a0.d,
        second ? a1.ldv : a0.ldv, second ? a1.C : a0.C, second ? a1.col_items : a0.col_items, second ? a1.div : a0.div, a0.L, a0.R,
        second ? a1.by_column : a0.by_column, a0.run, second ? a1.scale : a0.scale};
    const int64_t item = second ? at_item - a0.items : at_item;
    const int lane = threadIdx.x & 63, wave = uniform((int32_t)(threadIdx.x >> 6));
    const int r16 = lane & 15, q = lane >> 4;
    const int64_t chunk = item / m.col_items, col0 = (item - chunk * m.col_items) * kCols;
    const int64_t t0 = chunk * m.run, t1 = min(t0 + m.run, (int64_t)uniform(tab.tiles[m.L]));   // (the pairs without adapter are last)
    if (t0 >= t1) return;
    // copies: instruction i of a wave brings rows 2*(4*i + wave), +1; a lane's position in its row holds another run (below)
    const int cr = lane >> 5, pos = lane & 31;
    const uint8_t* none = reinterpret_cast<const uint8_t*>(&kZeros);
    const auto swizzle = [](int row) { return ((row & 3) | ((row >> 1) & 4)) << 1; };
    f32x4 acc[kTiles][RT] = {};
    // a batch of tiles at a time: its rows are listed in LDS, since a load in the loop below would wait for the copies too
    for (int64_t b0 = t0; b0 < t1; b0 += kBatch) {
    const int count = (int)min((int64_t)kBatch, t1 - b0);
    block_barrier();                                               // the last batch's lists have been read
    for (int i = threadIdx.x; i < count * kTile; i += kThreads) {
        const int4 d = tab.tdesc[b0 + i / kTile];
        const int s = i % kTile;
        row_lds[i] = s < d.z ? tab.sorted[d.y + s] / m.div : -1;
        if (s == 0) {
            id_lds[i / kTile] = d.x;
            scale_lds[i / kTile] = m.scale ? m.scale[d.x] : 1.0f;
        }
    }
    if (threadIdx.x == 0) id_lds[count] = b0 + count < t1 ? tab.tdesc[b0 + count].x : -1;
    block_barrier();
    const auto copy_tile = [&](int i0) {
        const int buf = i0 % kDeep;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = 2 * (4 * i + wave) + cr;
            const int32_t row = row_lds[i0 * kTile + at];
            const int64_t c = col0 + (pos ^ swizzle(at)) * (16 / kSize<DT>);
            copy16(lds_address(&vs[buf][2 * (4 * i + wave)][0]), row >= 0 && c < m.C ? m.v + (int64_t)row * m.ldv + c * kSize<DT> : none);
        }
#pragma unroll
        for (int i = 0; i < kUShare; ++i) {
            const int part = (wave + 4 * i) % kU;
            copy16(lds_address(&us[buf][part * 1024]), m.u + (b0 + i0) * kUBytes + part * 1024 + lane * 16);
        }
    };
    settle();
    for (int i0 = 0; i0 < count && i0 < kDeep - 1; ++i0) copy_tile(i0);
    for (int i0 = 0; i0 < count; ++i0) {
        const int buf = i0 % kDeep;
        wait_step<kPer, kDeep - 2>(count - 1 - i0);
        block_barrier();                                           // all waves' copies of the tile are there, the last one has been read
        const int32_t l = uniform(id_lds[i0]), after = uniform(id_lds[i0 + 1]);
        const float scale = scale_lds[i0];
        if (i0 + kDeep - 1 < count) copy_tile(i0 + kDeep - 1);
        if constexpr (DT == FTQ_F32) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float x[kTiles];
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    const int row = 4 * k + q, c = wave * (kCols / 4) + 16 * i + r16;
                    x[i] = *reinterpret_cast<const float*>(&vs[buf][row][((c >> 2) ^ swizzle(row)) * 16 + (c & 3) * 4]);
                }
#pragma unroll
                for (int j = 0; j < RT; ++j) {
                    const float u = *reinterpret_cast<const float*>(&us[buf][(16 * j + r16) * kULine + (4 * k + q) * 4]);
#pragma unroll
                    for (int i = 0; i < kTiles; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], u, acc[i][j], 0, 0, 0);
                }
            }
        } else {
            // columns as the left operand: a transposing read gives a lane four rows of its column
            u32x4 x[kTiles][kParts<DT>];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                u32x2 half[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = 8 * q + 4 * h + (r16 >> 2), c = wave * (kCols / 4) + 16 * i + (r16 & 3) * 4;
                    const uint8_t* src = &vs[buf][row][((c >> 3) ^ swizzle(row)) * 16 + (c & 7) * 2];
                    half[h] = read_transposed(src);
                }
                split_operand<DT>(u32x4{half[0][0], half[0][1], half[1][0], half[1][1]}, x[i]);
            }
#pragma unroll
            for (int j = 0; j < RT; ++j) {
#pragma unroll
                for (int c = 0; c < kPieces<DT>; ++c) {
                    const u32x4 u = *reinterpret_cast<const u32x4*>(&us[buf][((c * RT + j) * 16 + r16) * kULine + q * 16]);
#pragma unroll
                    for (int h = 0; h < kParts<DT>; ++h) {
#pragma unroll
                        for (int i = 0; i < kTiles; ++i) acc[i][j] = multiply<FTQ_BF16>(x[i][h], u, acc[i][j]);
                    }
                }
            }
        }
        if (after == l) continue;
        // the adapter's last tile here: its sums
        const int64_t f0 = uniform(tab.tiles[l]), f1 = uniform(tab.tiles[l + 1]);
        float* to = m.d + (int64_t)l * m.R * m.C;
        if (f0 < t0 || f1 > t1) to = m.part + (2 * chunk + (f0 < t0 ? 0 : 1)) * m.R * m.C;
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            const int64_t c = col0 + wave * (kCols / 4) + 16 * i + 4 * q;   // this lane's four columns
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const int r = 16 * j + r16;
                if (c < m.C && r < m.R) {
                    if (m.by_column) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) to[(c + e) * m.R + r] = acc[i][j][e] * scale;
                    } else {
                        *reinterpret_cast<f32x4*>(to + r * m.C + c) = acc[i][j] * scale;
                    }
                }
                acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
        }
    }
    }
}

// Adapters whose tiles lie in several runs: their parts added up; adapters without a pair: zeros.
struct ReduceArgs {
    const float* part;
    float* d;
    int64_t size;              // R * C
    int32_t L, run;
    int64_t blocks;            // workgroups of an adapter
};

__global__ __launch_bounds__(kThreads) void lora_reduce_kernel(const int32_t* tiles, ReduceArgs a0, ReduceArgs a1)
{
    const bool second = (int64_t)blockIdx.x >= a0.blocks * a0.L;
    const ReduceArgs m = second ? a1 : a0;
    const int64_t item = second ? blockIdx.x - a0.blocks * a0.L : blockIdx.x;
    const int64_t l = item / m.blocks, i0 = (item - l * m.blocks) * kThreads + threadIdx.x;
    const int64_t t0 = tiles ? tiles[l] : 0, t1 = tiles ? tiles[l + 1] : 0;
    const int64_t c0 = t0 / m.run, c1 = t1 > t0 ? (t1 - 1) / m.run : c0;
    if (t1 > t0 && c0 == c1) return;
    for (int64_t i = i0; i < m.size / 4; i += m.blocks * kThreads) {
        f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
        if (t1 > t0) {
            sum = *reinterpret_cast<const f32x4*>(m.part + (2 * c0 + 1) * m.size + 4 * i);
            for (int64_t c = c0 + 1; c <= c1; ++c) sum += *reinterpret_cast<const f32x4*>(m.part + 2 * c * m.size + 4 * i);
        }
        *reinterpret_cast<f32x4*>(m.d + l * m.size + 4 * i) = sum;
    }
}

// ---- host ---------------------------------------------------------------------------

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t size_of(int dtype) { return dtype == FTQ_F32 ? 4 : 2; }
int rank_tiles(int64_t R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }

// Parts that a row's length is split into: by the sizes alone, so that a pair's bits do not go by the path.
int64_t shrink_splits(int64_t pairs, int64_t C, int64_t R, int dtype)
{
    const int64_t steps = ceil_div(C * size_of(dtype), kLine), tiles = ceil_div(pairs, 64);
    const int64_t want = tiles <= 16 ? 16 : std::max<int64_t>(1, 512 / tiles);
    return std::max<int64_t>(1, std::min({want, int64_t(16), steps / 2}));
}

// Pairs of an adapter side by side that a table tile takes, by the average.
int64_t table_tile(int64_t pairs, int64_t L) { return pairs / L >= 48 ? 64 : pairs / L >= 12 ? 32 : 16; }

// Few pairs in their order: tiles of 16, whose adapters several workgroups share.
bool few(int64_t pairs) { return pairs <= 256; }

TileList in_order(int64_t pairs)
{
    const int32_t rows = few(pairs) ? 16 : 64;
    return TileList{nullptr, nullptr, nullptr, 1, rows, ceil_div(pairs, rows)};
}

// The tables' plan; a tile holds a pair at least (ten pairs of 4095 adapters: ten tiles, not a partly filled one of each adapter).
BucketPlan plan_tables(int64_t pairs, int64_t L, int64_t tile)
{
    BucketPlan p = make_bucket_plan(pairs, L, tile);
    p.max_tiles = std::min(p.max_tiles, pairs);
    return p;
}

TileList from_tables(const BucketPlan& plan, const uint8_t* mem, int64_t L, int64_t span)
{
    return TileList{reinterpret_cast<const int32_t*>(mem + plan.off_sorted), reinterpret_cast<const int4*>(mem + plan.off_tdesc),
                    reinterpret_cast<const int32_t*>(mem + plan.off_tiles) + L + 1, (int32_t)span, (int32_t)(plan.tile_m * span),
                    ceil_div(plan.max_tiles, span)};
}

// Calls f(type constant).
template <typename F>
int by_type(int dtype, F f)
{
    if (dtype == FTQ_F32) return f(std::integral_constant<int, FTQ_F32>{});
    if (dtype == FTQ_F16) return f(std::integral_constant<int, FTQ_F16>{});
    return f(std::integral_constant<int, FTQ_BF16>{});
}

template <int DT, int WAVES, bool COLS>
int launch_shrink(const ShrinkArgs& m, int64_t grid, hipStream_t s)
{
    const auto go = [&](auto* kernel) {
        return launch_in_turn(grid, 64 * WAVES, [&](int64_t first, int64_t n) { return launch("lora_shrink_kernel", kernel, n, 64 * WAVES, 0, s, m, first); });
    };
    switch (rank_tiles(m.R)) {
        case 1: return go(lora_shrink_kernel<DT, WAVES, 1, COLS>);
        case 2: return go(lora_shrink_kernel<DT, WAVES, 2, COLS>);
        case 4: return go(lora_shrink_kernel<DT, WAVES, 4, COLS>);
        default: return go(lora_shrink_kernel<DT, WAVES, 8, COLS>);
    }
}

template <bool COLS>
int run_shrink(int dtype, ShrinkArgs m, hipStream_t s)
{
    const bool small = m.tiles.rows <= 16;
    const int64_t tiles = m.tiles.most;
    m.groups = !m.tiles.sorted && small ? (int32_t)std::min<int64_t>(16, m.L) : 1;
    m.steps = (int32_t)ceil_div(ceil_div(m.row_bytes, kLine), m.splits);
    return by_type(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const int64_t grid = tiles * m.groups * m.splits;
        if constexpr (!COLS) {                                     // (the gradients' tiles are of 32 pairs and more)
            if (small) return launch_shrink<DT, 1, COLS>(m, grid, s);
        }
        return launch_shrink<DT, 4, COLS>(m, grid, s);
    });
}

template <int DT, int OT, bool RANKS, int WR>
int launch_expand(const ExpandArgs& m, int64_t grid, hipStream_t s)
{
    const auto go = [&](auto* kernel) {
        return launch_in_turn(grid, kThreads, [&](int64_t first, int64_t n) { return launch("lora_expand_kernel", kernel, n, kThreads, 0, s, m, first); });
    };
    const int rt = rank_tiles(m.R);
    if constexpr (DT == FTQ_F32) {
        if (rt == 1) return go(lora_expand_kernel<DT, OT, 1, RANKS, WR>);
        if (rt == 2) return go(lora_expand_kernel<DT, OT, 2, RANKS, WR>);
        if (rt == 4) return go(lora_expand_kernel<DT, OT, 4, RANKS, WR>);
        return go(lora_expand_kernel<DT, OT, 8, RANKS, WR>);
    } else {
        if (rt <= 2) return go(lora_expand_kernel<DT, OT, 1, RANKS, WR>);
        if (rt == 4) return go(lora_expand_kernel<DT, OT, 2, RANKS, WR>);
        return go(lora_expand_kernel<DT, OT, 4, RANKS, WR>);
    }
}

template <bool RANKS>
int run_expand(int dtype, int out_dtype, ExpandArgs m, hipStream_t s)
{
    const bool small = m.tiles.rows <= 16;
    m.groups = !m.tiles.sorted && small ? (int32_t)std::min<int64_t>(16, m.L) : 1;
    // the columns in even shares of whole steps, for about four workgroups a CU; many tiles are not shared (1009 tiles of up
    // to 32 pairs, 2816 columns: 90 us, 98 in two shares)
    const int64_t step = small ? 256 : 64, lots = ceil_div(m.C, step), tiles = m.tiles.most * m.groups;
    const int64_t shares = tiles >= 512 ? 1 : std::min(lots, ceil_div(1024, tiles));
    m.cols = (int32_t)(ceil_div(lots, shares) * step);
    m.col_items = ceil_div(m.C, m.cols);
    const int64_t grid = tiles * m.col_items;
    return by_type(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const auto with = [&](auto ot) {
            constexpr int OT = decltype(ot)::value;
            if constexpr (!RANKS) {
                if (small) return launch_expand<DT, OT, RANKS, 1>(m, grid, s);
            }
            return launch_expand<DT, OT, RANKS, 4>(m, grid, s);
        };
        if constexpr (RANKS) return with(dt);                      // d_x has the rows' type
        else return by_type(out_dtype, with);
    });
}

struct ForwardPlan {
    BucketPlan bucket;
    int64_t splits, off_part, bytes;
};

ForwardPlan plan_forward(int64_t L, int64_t R, int64_t K, int64_t pairs, int dtype, int path)
{
    ForwardPlan p;
    if (path == FTQ_PATH_GROUPED) p.bucket = plan_tables(pairs, L, table_tile(pairs, L));
    p.splits = shrink_splits(pairs, K, R, dtype);
    p.off_part = p.bucket.bytes;
    p.bytes = p.off_part + align256(p.splits * pairs * R * 4);
    return p;
}

struct BackwardPlan {
    BucketPlan bucket;
    int64_t splits, run, runs_max;
    int64_t off_part, off_g, off_ug, off_uh, off_pa, off_pb, bytes;
};

BackwardPlan plan_backward(int64_t L, int64_t R, int64_t K, int64_t N, int64_t pairs, int dtype)
{
    BackwardPlan p;
    const int64_t es = size_of(dtype), rt = 16 * rank_tiles(R), pieces = dtype == FTQ_F32 ? 2 : 3;   // (of 16 bits)
    p.bucket = plan_tables(pairs, L, kTile);
    p.splits = shrink_splits(pairs, N, R, dtype);
    // runs of tiles for as many workgroups as fit the chip at once (by LDS two on a CU, one of high ranks), at most a part
    // for every four tiles
    const int64_t col_items = ceil_div(K * es, 512) + ceil_div(N * es, 512), tiles = std::max<int64_t>(p.bucket.max_tiles, 1);
    p.run = std::max<int64_t>(4, ceil_div(tiles * col_items, R <= 64 ? 512 : 256));
    p.runs_max = ceil_div(tiles, p.run);
    int64_t off = p.bucket.bytes;
    const auto take = [&](int64_t bytes) {
        const int64_t at = off;
        off += align256(bytes);
        return at;
    };
    p.off_part = take(p.splits * pairs * R * 4);
    p.off_g = take(pairs * R * 4);
    p.off_ug = take(tiles * rt * kTile * 2 * pieces);
    p.off_uh = take(tiles * rt * kTile * 2 * pieces);
    p.off_pa = take(2 * p.runs_max * R * K * 4);
    p.off_pb = take(2 * p.runs_max * R * N * 4);
    p.bytes = off;
    return p;
}

int launch_pieces(int dtype, int rt, const OuterTables& tab, const PiecesArgs& a, const PiecesArgs& b, hipStream_t s)
{
    return by_type(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const auto go = [&](auto* kernel) {
            return launch_in_turn(a.max_tiles + b.max_tiles, kThreads,
                                  [&](int64_t first, int64_t n) { return launch("lora_pieces_kernel", kernel, n, kThreads, 0, s, tab, a, b, first); });
        };
        if (rt == 1) return go(lora_pieces_kernel<DT, 1>);
        if (rt == 2) return go(lora_pieces_kernel<DT, 2>);
        if (rt == 4) return go(lora_pieces_kernel<DT, 4>);
        return go(lora_pieces_kernel<DT, 8>);
    });
}

int launch_outer(int dtype, int rt, const OuterTables& tab, const OuterArgs& a, const OuterArgs& b, hipStream_t s)
{
    return by_type(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const auto go = [&](auto* kernel) {
            return launch_in_turn(a.items + b.items, kThreads,
                                  [&](int64_t first, int64_t n) { return launch("lora_outer_kernel", kernel, n, kThreads, 0, s, tab, a, b, first); });
        };
        if (rt == 1) return go(lora_outer_kernel<DT, 1>);
        if (rt == 2) return go(lora_outer_kernel<DT, 2>);
        if (rt == 4) return go(lora_outer_kernel<DT, 4>);
        return go(lora_outer_kernel<DT, 8>);
    });
}

}  // namespace

int64_t lora_workspace(int64_t L, int64_t R, int64_t K, int64_t, int64_t T, int64_t top_k, int dtype, int path)
{
    return plan_forward(L, R, K, T * top_k, dtype, path).bytes;
}

int64_t lora_backward_workspace(int64_t L, int64_t R, int64_t K, int64_t N, int64_t T, int64_t top_k, int dtype)
{
    return T == 0 ? 0 : plan_backward(L, R, K, N, T * top_k, dtype).bytes;
}

// In order where a tile holds few adapters: rows of requests (top_k 1), by what a call can know, or few pairs.  In order /
// sorted, us, rank 16, 4096 x 4096, bf16: 8192 rows of 8 adapters, each one's together, 49 / 59, at random 181 / 60; 512 of
// 64 together 92 / 19, at random 288 / 20; 256 of 8 together 16 / 21, at random 20 / 21.
int lora_select_path(int64_t T, int64_t top_k) { return top_k == 1 || T * top_k <= 256 ? FTQ_PATH_GEMV : FTQ_PATH_GROUPED; }

int run_lora(const LoraArgs& m, void* ws, int path, hipStream_t s)
{
    const int64_t pairs = m.T * m.top_k;
    uint8_t* mem = static_cast<uint8_t*>(ws);
    const ForwardPlan plan = plan_forward(m.L, m.R, m.K, pairs, m.dtype, path);
    TileList tiles = in_order(pairs);
    if (path == FTQ_PATH_GROUPED) {
        const int st = run_bucket(m.ids, m.L, plan.bucket, ws, s);
        if (st != FTQ_OK) return st;
        tiles = from_tables(plan.bucket, mem, m.L, 1);
    }
    ShrinkArgs shrink{};
    shrink.v = static_cast<const uint8_t*>(m.x);
    shrink.ldv = m.ldx * size_of(m.dtype);
    shrink.w = static_cast<const uint8_t*>(m.a);
    shrink.ids = m.ids;
    shrink.tiles = tiles;
    shrink.part = reinterpret_cast<float*>(mem + plan.off_part);
    shrink.pairs = pairs;
    shrink.row_bytes = m.K * size_of(m.dtype);
    shrink.div = (int32_t)m.act_div;
    shrink.L = (int32_t)m.L;
    shrink.R = (int32_t)m.R;
    shrink.splits = (int32_t)plan.splits;
    const int st = run_shrink<false>(m.dtype, shrink, s);
    if (st != FTQ_OK) return st;
    ExpandArgs expand{};
    expand.part = shrink.part;
    expand.w = static_cast<const uint8_t*>(m.b);
    expand.scale = m.scale;
    expand.ids = m.ids;
    expand.tiles = tiles;
    expand.base = m.base;
    expand.out = m.out;
    expand.h = m.h;
    expand.ld_base = m.ld_base;
    expand.ld_out = m.ld_out;
    expand.pairs = pairs;
    expand.C = m.N;
    expand.L = shrink.L;
    expand.R = shrink.R;
    expand.splits = shrink.splits;
    return run_expand<false>(m.dtype, m.out_dtype, expand, s);
}

int run_lora_backward(const LoraBackwardArgs& m, void* ws, hipStream_t s)
{
    const int64_t pairs = m.T * m.top_k, es = size_of(m.dtype);
    const int rt = rank_tiles(m.R);
    const auto reduce = [&](const int32_t* tiles, int64_t run, const float* pa, const float* pb) {
        const auto args = [&](float* d, int64_t C, const float* part) {
            return ReduceArgs{part, d, m.R * C, d ? (int32_t)m.L : 0, (int32_t)run, std::min<int64_t>(ceil_div(m.R * C / 4, kThreads), std::max<int64_t>(8, 2048 / m.L))};
        };
        const ReduceArgs a = args(m.d_a, m.K, pa), b = args(m.d_b, m.N, pb);
        return launch("lora_reduce_kernel", lora_reduce_kernel, a.blocks * a.L + b.blocks * b.L, kThreads, 0, s, tiles, a, b);
    };
    if (pairs == 0) return reduce(nullptr, 1, nullptr, nullptr);
    uint8_t* mem = static_cast<uint8_t*>(ws);
    const BackwardPlan plan = plan_backward(m.L, m.R, m.K, m.N, pairs, m.dtype);
    int st = run_bucket(m.ids, m.L, plan.bucket, ws, s);
    if (st != FTQ_OK) return st;
    const OuterTables tab{reinterpret_cast<const int32_t*>(mem + plan.bucket.off_tiles), reinterpret_cast<const int32_t*>(mem + plan.bucket.off_sorted),
                          reinterpret_cast<const int4*>(mem + plan.bucket.off_tdesc)};
    const TileList rows_of = from_tables(plan.bucket, mem, m.L, table_tile(pairs, m.L) == 64 ? 2 : 1);
    const auto floats = [&](int64_t off) { return reinterpret_cast<float*>(mem + off); };
    const bool want_g = m.d_x || m.d_a, expand_x = m.d_x && m.act_div == 1;   // else rows that several pairs share
    if (want_g) {
        ShrinkArgs shrink{};
        shrink.v = static_cast<const uint8_t*>(m.d_out);
        shrink.ldv = m.ld_d * es;
        shrink.w = static_cast<const uint8_t*>(m.b);
        shrink.ids = m.ids;
        shrink.tiles = rows_of;
        shrink.part = floats(plan.off_part);
        shrink.pairs = pairs;
        shrink.row_bytes = m.N * es;
        shrink.div = 1;
        shrink.L = (int32_t)m.L;
        shrink.R = (int32_t)m.R;
        shrink.splits = (int32_t)plan.splits;
        st = run_shrink<true>(m.dtype, shrink, s);
        if (st != FTQ_OK) return st;
    }
    // the R-vectors of the outer products, and g itself
    const int64_t tiles = plan.bucket.max_tiles;
    const PiecesArgs pg{floats(plan.off_part), m.scale, m.d_x ? floats(plan.off_g) : nullptr, m.d_a ? mem + plan.off_ug : nullptr, pairs, want_g ? tiles : 0, (int32_t)m.L, (int32_t)m.R, (int32_t)plan.splits};
    const PiecesArgs ph{m.h, nullptr, nullptr, mem + plan.off_uh, pairs, m.d_b ? tiles : 0, (int32_t)m.L,
                        (int32_t)m.R, 1};
    st = launch_pieces(m.dtype, rt, tab, pg, ph, s);
    if (st != FTQ_OK) return st;
    if (expand_x) {
        ExpandArgs expand{};
        expand.part = floats(plan.off_g);
        expand.w = static_cast<const uint8_t*>(m.a);
        expand.ids = m.ids;
        expand.tiles = rows_of;
        expand.base = m.base;
        expand.out = m.d_x;
        expand.ld_base = expand.ld_out = expand.C = m.K;
        expand.pairs = pairs;
        expand.L = (int32_t)m.L;
        expand.R = (int32_t)m.R;
        expand.splits = 1;
        st = run_expand<true>(m.dtype, m.dtype, expand, s);
        if (st != FTQ_OK) return st;
    } else if (m.d_x) {
        GatherArgs gather{floats(plan.off_g), static_cast<const uint8_t*>(m.a), m.ids, static_cast<const uint8_t*>(m.base), static_cast<uint8_t*>(m.d_x),
                          m.T, m.K, ceil_div(m.K * es, 1024), ceil_div(m.T, kGatherTokens), (int32_t)m.L, (int32_t)m.R, (int32_t)m.top_k};
        const int64_t grid = ceil_div(gather.slices * gather.groups, kXcds) * kXcds;
        st = by_type(m.dtype, [&](auto dt) {
            return launch_in_turn(grid, kThreads, [&](int64_t first, int64_t n) {
                return launch("lora_gather_kernel", lora_gather_kernel<decltype(dt)::value>, n, kThreads, 0, s, gather, first);
            });
        });
        if (st != FTQ_OK) return st;
    }
    if (!m.d_a && !m.d_b) return FTQ_OK;
    const auto outer = [&](int64_t off_u, const void* v, int64_t ldv, int64_t off_part, float* d, int64_t C, int64_t div, bool by_column, const float* scale) {
        const int64_t col_items = ceil_div(C * es, 512);
        return OuterArgs{mem + off_u, static_cast<const uint8_t*>(v), ldv * es, floats(off_part), d, C, col_items,
                         d ? plan.runs_max * col_items : 0, (int32_t)div, (int32_t)m.L, (int32_t)m.R, by_column, (int32_t)plan.run, scale};
    };
    st = launch_outer(m.dtype, rt, tab, outer(plan.off_ug, m.x, m.ldx, plan.off_pa, m.d_a, m.K, m.act_div, false, nullptr),
                      outer(plan.off_uh, m.d_out, m.ld_d, plan.off_pb, m.d_b, m.N, 1, true, m.scale), s);
    if (st != FTQ_OK) return st;
    return reduce(tab.tiles, plan.run, floats(plan.off_pa), floats(plan.off_pb));
}

}  // namespace ftq
