// Top-k weighted combine of the expert outputs of a token's pairs: the step
// after the down projection of an expert FFN (the per-pair activation layout
// of "Current Bug: CuTeDSLMoERunner", Bug 6, and its L2 output).
//
//   out[t][n] = sum_{j < k} gates[t][j] * y[t*k + j][n]
//
// evaluated in fp32 as acc = fma(gates[t][j], y[t*k+j][n], acc) for j = 0, 1,
// ..., k-1 from acc = 0: a fixed order, so the result does not depend on the
// batch or the launch.  Rows of masked pairs hold zeros (the matmul writes
// them) and add nothing.  The kernel streams y once: HBM bound, with four
// consecutive columns per lane (16-byte loads and stores) when N % 4 == 0 and
// the buffers are 16-byte aligned.
#include "ftq_internal.h"

namespace ftq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
constexpr int kThreads = 256;

template <int VEC>
__global__ __launch_bounds__(kThreads) void combine_topk_kernel(const float* __restrict__ y,
                                                                const float* __restrict__ gates,
                                                                float* __restrict__ out, int64_t T, int64_t k,
                                                                int64_t N)
{
    const int64_t nv = N / VEC;                       // column groups per row
    const int64_t total = T * nv;
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += stride) {
        const int64_t t = i / nv, c = (i - t * nv) * VEC;
        if constexpr (VEC == 4) {
            f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int64_t j = 0; j < k; ++j) {
                const float g = gates[t * k + j];
                const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(y + (t * k + j) * N + c));
                acc.x = __builtin_fmaf(g, v.x, acc.x);
                acc.y = __builtin_fmaf(g, v.y, acc.y);
                acc.z = __builtin_fmaf(g, v.z, acc.z);
                acc.w = __builtin_fmaf(g, v.w, acc.w);
            }
            *reinterpret_cast<f32x4*>(out + t * N + c) = acc;
        } else {
            float acc = 0.0f;
            for (int64_t j = 0; j < k; ++j) acc = __builtin_fmaf(gates[t * k + j], y[(t * k + j) * N + c], acc);
            out[t * N + c] = acc;
        }
    }
}

// The gradient: d_y[t*k+j][n] = gates[t][j] * d_out[t][n], and d_gates[t][j] the
// dot product of y[t*k+j] and d_out[t].  One workgroup per pair reads its row of y
// and its token's row of d_out once (the token's pairs follow one another, so that
// d_out comes from the caches after the first) and writes its row of d_y.  A dot
// product is summed by thread, then by a fixed tree.
template <int VEC> struct RunF { float v[VEC]; } __attribute__((packed, aligned(4)));
template <int VEC> struct RunH { uint16_t v[VEC]; } __attribute__((packed, aligned(2)));

template <int VEC, int DT>
__global__ __launch_bounds__(kThreads) void combine_topk_backward_kernel(const float* __restrict__ d_out, const float* __restrict__ y,
                                                                         const float* __restrict__ gates, void* __restrict__ d_y,
                                                                         float* __restrict__ d_gates, int64_t pairs, int64_t k, int64_t N)
{
    __shared__ float part[2][kThreads / 64];
    int turn = 0;
    for (int64_t p = blockIdx.x; p < pairs; p += gridDim.x, turn ^= 1) {
        const float g = d_y ? gates[p] : 0.0f;        // (gates may be null without d_y, y without d_gates)
        const float* dr = d_out + p / k * N;
        const float* yr = y + p * N;
        float dot = 0.0f;
        for (int64_t c = (int64_t)threadIdx.x * VEC; c < N; c += kThreads * VEC) {
            const RunF<VEC> d = *reinterpret_cast<const RunF<VEC>*>(dr + c);
            if (d_gates) {
                const RunF<VEC> v = *reinterpret_cast<const RunF<VEC>*>(yr + c);
#pragma unroll
                for (int i = 0; i < VEC; ++i) dot = __builtin_fmaf(v.v[i], d.v[i], dot);
            }
            if (d_y) {
                if constexpr (DT == FTQ_F32) {
                    RunF<VEC> o;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) o.v[i] = g * d.v[i];
                    *reinterpret_cast<RunF<VEC>*>(static_cast<float*>(d_y) + p * N + c) = o;
                } else {
                    RunH<VEC> o;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) o.v[i] = DT == FTQ_F16 ? f16_of_f32(g * d.v[i]) : bf16_of_f32(g * d.v[i]);
                    *reinterpret_cast<RunH<VEC>*>(static_cast<uint16_t*>(d_y) + p * N + c) = o;
                }
            }
        }
        if (!d_gates) continue;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o);
        if (threadIdx.x % 64 == 0) part[turn][threadIdx.x / 64] = dot;
        __syncthreads();   // the next pair writes the other half of part
        if (threadIdx.x == 0) {
            dot = 0.0f;
#pragma unroll
            for (int w = 0; w < kThreads / 64; ++w) dot += part[turn][w];
            d_gates[p] = dot;
        }
    }
}

}  // namespace

int run_combine_topk_backward(const float* d_out, const float* y, const float* gates, void* d_y, int dtype, float* d_gates,
                              int64_t T, int64_t top_k, int64_t N, hipStream_t s)
{
    const int64_t pairs = T * top_k, grid = std::min<int64_t>(pairs, int64_t(1) << 20);
    const auto go = [&](auto* kernel) {
        return launch("combine_topk_backward_kernel", kernel, grid, kThreads, 0, s, d_out, y, gates, d_y, d_gates, pairs, top_k, N);
    };
    if (N % 4 == 0) {
        if (dtype == FTQ_F32) return go(combine_topk_backward_kernel<4, FTQ_F32>);
        if (dtype == FTQ_F16) return go(combine_topk_backward_kernel<4, FTQ_F16>);
        return go(combine_topk_backward_kernel<4, FTQ_BF16>);
    }
    if (dtype == FTQ_F32) return go(combine_topk_backward_kernel<1, FTQ_F32>);
    if (dtype == FTQ_F16) return go(combine_topk_backward_kernel<1, FTQ_F16>);
    return go(combine_topk_backward_kernel<1, FTQ_BF16>);
}

int run_combine_topk(const float* y, const float* gates, float* out, int64_t T, int64_t top_k, int64_t N,
                     hipStream_t s)
{
    DeviceLimits lim;
    int st = device_limits(&lim);
    if (st != FTQ_OK) return st;
    const bool v4 = N % 4 == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
    const int64_t items = T * (v4 ? N / 4 : N);
    const int64_t grid = stride_grid((items + kThreads - 1) / kThreads, lim);
    if (v4) return launch("combine_topk_kernel<4>", combine_topk_kernel<4>, grid, kThreads, 0, s, y, gates, out, T, top_k, N);
    return launch("combine_topk_kernel<1>", combine_topk_kernel<1>, grid, kThreads, 0, s, y, gates, out, T, top_k, N);
}

}  // namespace ftq
