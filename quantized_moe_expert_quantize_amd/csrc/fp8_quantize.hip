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
// Both are HBM-streaming kernels: 16-byte loads, every input read once (a
// block's values stay in registers between the maximum and the codes).
#include "ftq_internal.h"

namespace ftq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr int kThreads = 256;
constexpr float kMax = 448.0f;

// Eight consecutive elements as fp32.
template <int DT>
__device__ __forceinline__ void load8(const uint8_t* p, float (&v)[8])
{
    if constexpr (DT == FTQ_F32) {
        const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
        const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p) + 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
        const u32x4 a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint16_t lo = (uint16_t)a[i], hi = (uint16_t)(a[i] >> 16);
            v[2 * i] = DT == FTQ_F16 ? f32_of_f16(lo) : f32_of_bf16(lo);
            v[2 * i + 1] = DT == FTQ_F16 ? f32_of_f16(hi) : f32_of_bf16(hi);
        }
    }
}

__device__ __forceinline__ uint32_t magnitude8(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);
    return m;
}

// x / scale, saturated; a NaN quotient stays NaN.
__device__ __forceinline__ float code_value(float x, float scale)
{
    const float q = x / scale;
    return q != q ? q : fminf(fmaxf(q, -kMax), kMax);
}

// Four fp32 values to four e4m3 bytes, round to nearest even.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8], float scale)
{
    if (scale == 0.0f) return uint2{0u, 0u};
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = code_value(v[i], scale);
    return uint2{pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7])};
}

// Activations: 16 lanes per block of 128, eight values a lane.  K % 16 == 0, so
// a lane's eight values of a row's last block are all inside or all outside.
constexpr int kLanes = 16;
constexpr int kBlocksPerGroup = kThreads / kLanes;

template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_fp8_kernel(const uint8_t* __restrict__ x, int64_t row_bytes,
                                                                int64_t T, int64_t K, int64_t nb,
                                                                uint8_t* __restrict__ y, float* __restrict__ scales)
{
    constexpr int kElem = DT == FTQ_F32 ? 4 : 2;
    const int sub = threadIdx.x % kLanes;
    const int64_t total = T * nb;
    for (int64_t i = (int64_t)blockIdx.x * kBlocksPerGroup + threadIdx.x / kLanes; i < total;
         i += (int64_t)gridDim.x * kBlocksPerGroup) {
        const int64_t t = i / nb, k = (i - t * nb) * kFp8Block + sub * 8;
        const bool in = k < K;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (in) load8<DT>(x + t * row_bytes + k * kElem, v);
        uint32_t m = magnitude8(v);
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
        const float scale = __builtin_bit_cast(float, m) / kMax;
        if (in) *reinterpret_cast<uint2*>(y + t * K + k) = codes8(v, scale);
        if (sub == 0) scales[i] = scale;
    }
}

// Weights: one workgroup per 128 x 128 block, eight runs of eight values a
// thread: run i of thread h is row i*16 + h/16, columns (h%16)*8 of the block.
constexpr int kRuns = kFp8Block * kFp8Block / 8 / kThreads;

template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_fp8_weight_kernel(const uint8_t* __restrict__ w, int64_t E,
                                                                       int64_t N, int64_t K, int64_t nr, int64_t nb,
                                                                       uint8_t* __restrict__ y,
                                                                       float* __restrict__ scales)
{
    constexpr int kElem = DT == FTQ_F32 ? 4 : 2;
    __shared__ uint32_t wave_max[2][kThreads / 64];
    const int r0 = threadIdx.x / kLanes, c0 = (threadIdx.x % kLanes) * 8;
    int turn = 0;
    for (int64_t i = blockIdx.x; i < E * nr * nb; i += gridDim.x, turn ^= 1) {
        const int64_t e = i / (nr * nb), r = (i / nb) % nr, b = i % nb;
        const int64_t k = b * kFp8Block + c0;
        float v[kRuns][8] = {};
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < kRuns; ++j) {
            const int64_t n = r * kFp8Block + j * (kThreads / kLanes) + r0;
            if (n < N && k < K) load8<DT>(w + ((e * N + n) * K + k) * kElem, v[j]);
        }
#pragma unroll
        for (int j = 0; j < kRuns; ++j) m = max(m, magnitude8(v[j]));
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
            if (n < N && k < K) *reinterpret_cast<uint2*>(y + (e * N + n) * K + k) = codes8(v[j], scale);
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
    return launch("quantize_fp8_kernel", quantize_fp8_kernel<DT>, stride_grid(groups, lim), kThreads, 0, s, x,
                  row_bytes, T, K, nb, static_cast<uint8_t*>(y), scales);
}

template <int DT>
int launch_weight(const uint8_t* w, int64_t E, int64_t N, int64_t K, void* y, float* scales, const DeviceLimits& lim,
                  hipStream_t s)
{
    const int64_t nr = (N + kFp8Block - 1) / kFp8Block, nb = (K + kFp8Block - 1) / kFp8Block;
    return launch("quantize_fp8_weight_kernel", quantize_fp8_weight_kernel<DT>, stride_grid(E * nr * nb, lim), kThreads,
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
