// Quantisers to 8-bit floating point (OCP e4m3) with one fp32 scale per 128
// values of a row (activations) or per 128 x 128 block (weights):
//
//   scale = max|x| / 448,   code = e4m3(x / scale),   codes 0 when scale is 0.
//
// Both divisions are the IEEE fp32 ones, so codes and scales are unique.  The
// maximum is taken over the bit patterns without their sign as integers, which
// order as the magnitudes do, infinity above the finite values and NaN above
// infinity: a NaN or an infinity in a block reaches its scale.
//
// Both are HBM-streaming kernels: 16-byte loads and stores, every input read once
// (a block's values stay in registers between the maximum and the codes), 16
// values a lane.  What limited them first was arithmetic: the hardware has no
// division, and the IEEE one the compiler writes is about ten instructions a
// value; quotient() makes the same fp32 quotient in six.
#include "ftq_internal.h"

namespace ftq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr int kThreads = 256;
// Workgroups per CU that a launch may have: in effect one pass.  Fewer, that walk
// the blocks, were slower (32768 x 4096 fp32: 130 us with 16 a CU, 118 so).
constexpr int kPerCu = 4096;
constexpr float kMax = 448.0f;
constexpr int kRun = 16;                               // values of a lane
constexpr int kLanes = kFp8Block / kRun;               // lanes of a row of a block

// Sixteen consecutive elements as fp32.  (Cached loads: a lane's 32 or 64 bytes take
// several instructions, each of which touches a part of a line that the next ones
// want; loads past the caches cost 168 instead of 118 us on 32768 x 4096 fp32.)
template <int DT>
__device__ __forceinline__ void load_run(const uint8_t* p, float (&v)[kRun])
{
    if constexpr (DT == FTQ_F32) {
        f32x4 a[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = reinterpret_cast<const f32x4*>(p)[j];
#pragma unroll
        for (int j = 0; j < kRun; ++j) v[j] = a[j / 4][j % 4];
    } else {
        u32x4 a[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) a[j] = reinterpret_cast<const u32x4*>(p)[j];
#pragma unroll
        for (int j = 0; j < kRun / 2; ++j) {
            const uint32_t u = a[j / 4][j % 4];
            const uint16_t lo = (uint16_t)u, hi = (uint16_t)(u >> 16);
            v[2 * j] = DT == FTQ_F16 ? f32_of_f16(lo) : f32_of_bf16(lo);
            v[2 * j + 1] = DT == FTQ_F16 ? f32_of_f16(hi) : f32_of_bf16(hi);
        }
    }
}

__device__ __forceinline__ uint32_t magnitude(const float (&v)[kRun])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) m = max(m, __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);
    return m;
}

// The largest of the eight lanes of a row of a block, in all of them.
__device__ __forceinline__ uint32_t largest8(uint32_t m)
{
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(m, m, 0xB1, 0xF, 0xF, false));    // quad_perm 1 0 3 2
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(m, m, 0x4E, 0xF, 0xF, false));    // quad_perm 2 3 0 1
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(m, m, 0x141, 0xF, 0xF, false));  // row_half_mirror
}

// x / scale rounded to nearest, given inv = 1 / scale rounded to nearest, where
// nothing over- or underflows: the first correction leaves q within a unit in the
// last place, and one more from such a q, with an exact remainder, is the rounded
// quotient (Markstein's theorem on division by fused multiply-adds).
__device__ __forceinline__ float quotient(float x, float scale, float inv)
{
    float q = x * inv;
    q = __builtin_fmaf(__builtin_fmaf(-q, scale, x), inv, q);
    q = __builtin_fmaf(__builtin_fmaf(-q, scale, x), inv, q);
    return __builtin_copysignf(q, x);                  // the remainders of -0 are +0
}

// Four fp32 values to four e4m3 bytes, round to nearest even.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

__device__ __forceinline__ u32x4 codes(const float (&v)[kRun], float scale)
{
    u32x4 r = {0u, 0u, 0u, 0u};
    if (scale > 7.9e-31f && scale < 1.2e30f) {         // 2^-100 .. 2^100: quotients are at most 448 (1 + 2^-23)
        const float inv = 1.0f / scale;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[j] = pack4(quotient(v[4 * j], scale, inv), quotient(v[4 * j + 1], scale, inv),
                         quotient(v[4 * j + 2], scale, inv), quotient(v[4 * j + 3], scale, inv));
        }
    } else if (scale != 0.0f) {                        // tiny (a subnormal scale may be far off), huge, infinite or NaN
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                q[i] = v[4 * j + i] / scale;
                q[i] = q[i] != q[i] ? q[i] : fminf(fmaxf(q[i], -kMax), kMax);
            }
            r[j] = pack4(q[0], q[1], q[2], q[3]);
        }
    }
    return r;
}

// Activations: eight lanes per block of 128.  K % 16 == 0, so a lane's values of a
// row's last block are all inside or all outside.  A group of lanes steps through
// the blocks of all rows; dt and db are the step in rows and blocks.
constexpr int kBlocksPerGroup = kThreads / kLanes;

template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_fp8_kernel(const uint8_t* __restrict__ x, int64_t row_bytes,
                                                                int64_t T, int64_t K, int64_t nb, int64_t dt, int64_t db,
                                                                uint8_t* __restrict__ y, float* __restrict__ scales)
{
    constexpr int kElem = DT == FTQ_F32 ? 4 : 2;
    const int sub = threadIdx.x % kLanes;
    const int64_t i = (int64_t)blockIdx.x * kBlocksPerGroup + threadIdx.x / kLanes;
    int64_t t = i / nb, b = i - t * nb;
    while (t < T) {
        const int64_t k = b * kFp8Block + sub * kRun;
        const bool in = k < K;
        float v[kRun] = {};
        if (in) load_run<DT>(x + t * row_bytes + k * kElem, v);
        const float scale = __builtin_bit_cast(float, largest8(magnitude(v))) / kMax;
        if (in) *reinterpret_cast<u32x4*>(y + t * K + k) = codes(v, scale);
        if (sub == 0) scales[t * nb + b] = scale;
        t += dt;
        b += db;
        if (b >= nb) {
            b -= nb;
            ++t;
        }
    }
}

// Weights: one workgroup per 128 x 128 block, four runs a thread: run j of thread h
// is row j*32 + h/8 of the block, columns (h%8)*16 on.
constexpr int kRuns = kFp8Block * kFp8Block / kRun / kThreads;

template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_fp8_weight_kernel(const uint8_t* __restrict__ w, int64_t E,
                                                                       int64_t N, int64_t K, int64_t nr, int64_t nb,
                                                                       uint8_t* __restrict__ y,
                                                                       float* __restrict__ scales)
{
    constexpr int kElem = DT == FTQ_F32 ? 4 : 2;
    __shared__ uint32_t wave_max[2][kThreads / 64];
    const int r0 = threadIdx.x / kLanes, c0 = threadIdx.x % kLanes * kRun;
    int turn = 0;
    for (int64_t i = blockIdx.x; i < E * nr * nb; i += gridDim.x, turn ^= 1) {
        const int64_t er = i / nb, b = i - er * nb, e = er / nr, r = er - e * nr;
        const int64_t k = b * kFp8Block + c0;
        float v[kRuns][kRun] = {};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < kRuns; ++j) {
            const int64_t n = r * kFp8Block + j * (kThreads / kLanes) + r0;
            if (n < N && k < K) load_run<DT>(w + ((e * N + n) * K + k) * kElem, v[j]);
        }
#pragma unroll
        for (int j = 0; j < kRuns; ++j) m = max(m, magnitude(v[j]));
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
        if (threadIdx.x % 64 == 0) wave_max[turn][threadIdx.x / 64] = m;
        __syncthreads();   // the next block writes the other half of wave_max, so one barrier a block is enough
#pragma unroll
        for (int j = 0; j < kThreads / 64; ++j) m = max(m, wave_max[turn][j]);
        const float scale = __builtin_bit_cast(float, m) / kMax;
#pragma unroll
        for (int j = 0; j < kRuns; ++j) {
            const int64_t n = r * kFp8Block + j * (kThreads / kLanes) + r0;
            if (n < N && k < K) *reinterpret_cast<u32x4*>(y + (e * N + n) * K + k) = codes(v[j], scale);
        }
        if (threadIdx.x == 0) scales[i] = scale;
    }
}

template <int DT>
int launch_rows(const uint8_t* x, int64_t row_bytes, int64_t T, int64_t K, void* y, float* scales,
                const DeviceLimits& lim, hipStream_t s)
{
    const int64_t nb = (K + kFp8Block - 1) / kFp8Block;
    const int64_t groups = (T * nb + kBlocksPerGroup - 1) / kBlocksPerGroup;
    const int64_t grid = stride_grid(groups, lim, kPerCu), step = grid * kBlocksPerGroup;
    return launch("quantize_fp8_kernel", quantize_fp8_kernel<DT>, grid, kThreads, 0, s, x, row_bytes, T, K, nb, step / nb,
                  step % nb, static_cast<uint8_t*>(y), scales);
}

template <int DT>
int launch_weight(const uint8_t* w, int64_t E, int64_t N, int64_t K, void* y, float* scales, const DeviceLimits& lim,
                  hipStream_t s)
{
    const int64_t nr = (N + kFp8Block - 1) / kFp8Block, nb = (K + kFp8Block - 1) / kFp8Block;
    return launch("quantize_fp8_weight_kernel", quantize_fp8_weight_kernel<DT>, stride_grid(E * nr * nb, lim, kPerCu), kThreads,
                  0, s, w, E, N, K, nr, nb, static_cast<uint8_t*>(y), scales);
}

}  // namespace

int run_quantize_fp8(const void* x, int dtype, int64_t ld, int64_t T, int64_t K, void* y, float* scales, hipStream_t s)
{
    DeviceLimits lim;
    int st = device_limits(&lim);
    if (st != FTQ_OK) return st;
    const uint8_t* p = static_cast<const uint8_t*>(x);
    if (dtype == FTQ_F32) return launch_rows<FTQ_F32>(p, ld * 4, T, K, y, scales, lim, s);
    if (dtype == FTQ_F16) return launch_rows<FTQ_F16>(p, ld * 2, T, K, y, scales, lim, s);
    return launch_rows<FTQ_BF16>(p, ld * 2, T, K, y, scales, lim, s);
}

int run_quantize_fp8_weight(const void* w, int dtype, int64_t E, int64_t N, int64_t K, void* y, float* scales,
                            hipStream_t s)
{
    DeviceLimits lim;
    int st = device_limits(&lim);
    if (st != FTQ_OK) return st;
    const uint8_t* p = static_cast<const uint8_t*>(w);
    if (dtype == FTQ_F32) return launch_weight<FTQ_F32>(p, E, N, K, y, scales, lim, s);
    if (dtype == FTQ_F16) return launch_weight<FTQ_F16>(p, E, N, K, y, scales, lim, s);
    return launch_weight<FTQ_BF16>(p, E, N, K, y, scales, lim, s);
}

}  // namespace ftq
