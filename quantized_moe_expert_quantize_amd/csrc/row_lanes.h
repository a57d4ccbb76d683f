// Reductions over the LPR lanes of a wave that work on one row, in fixed trees and
// without LDS.
#pragma once

#include "ftq_internal.h"

namespace ftq {
namespace {

// Every lane gets the result.

// The value of the lane across one halving step: lanes of a 2^(STEP+1) group hold
// equal values within its halves when STEP is reached, so mirrored lanes do.
template <int STEP>
__device__ __forceinline__ uint32_t across(uint32_t v)
{
    if constexpr (STEP == 0) return __builtin_amdgcn_update_dpp(v, v, 0xB1, 0xF, 0xF, false);    // quad_perm 1 0 3 2
    if constexpr (STEP == 1) return __builtin_amdgcn_update_dpp(v, v, 0x4E, 0xF, 0xF, false);    // quad_perm 2 3 0 1
    if constexpr (STEP == 2) return __builtin_amdgcn_update_dpp(v, v, 0x141, 0xF, 0xF, false);   // row_half_mirror
    return __builtin_amdgcn_update_dpp(v, v, 0x140, 0xF, 0xF, false);                            // row_mirror
}

template <int LPR, typename F>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, F op)
{
    if constexpr (LPR > 1) v = op(v, across<0>(v));
    if constexpr (LPR > 2) v = op(v, across<1>(v));
    if constexpr (LPR > 4) v = op(v, across<2>(v));
    if constexpr (LPR > 8) v = op(v, across<3>(v));
    if constexpr (LPR > 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = op(r[0], r[1]);
    }
    if constexpr (LPR > 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = op(r[0], r[1]);
    }
    return v;
}
__device__ __forceinline__ float as_f(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t as_u(float f) { return __builtin_bit_cast(uint32_t, f); }

template <int LPR> __device__ __forceinline__ uint32_t row_max_u(uint32_t v)
{
    return row_reduce<LPR>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int LPR> __device__ __forceinline__ float row_max(float v)
{
    return as_f(row_reduce<LPR>(as_u(v), [](uint32_t a, uint32_t b) { return as_u(fmaxf(as_f(a), as_f(b))); }));
}
template <int LPR> __device__ __forceinline__ float row_min(float v)
{
    return as_f(row_reduce<LPR>(as_u(v), [](uint32_t a, uint32_t b) { return as_u(fminf(as_f(a), as_f(b))); }));
}
template <int LPR> __device__ __forceinline__ float row_sum(float v)
{
    return as_f(row_reduce<LPR>(as_u(v), [](uint32_t a, uint32_t b) { return as_u(as_f(a) + as_f(b)); }));
}

// The sum over a wave's rows of what the lanes at the same place in them hold, in all of
// them: rotations of 8, 4 and 2 lanes within 16, then the 16s.
template <int LPR> __device__ __forceinline__ float sum_over_rows(float v)
{
    const auto add = [](float a, uint32_t b) { return a + as_f(b); };
    if constexpr (LPR < 16) v = add(v, __builtin_amdgcn_update_dpp(as_u(v), as_u(v), 0x128, 0xF, 0xF, false));
    if constexpr (LPR < 8) v = add(v, __builtin_amdgcn_update_dpp(as_u(v), as_u(v), 0x124, 0xF, 0xF, false));
    if constexpr (LPR < 4) v = add(v, __builtin_amdgcn_update_dpp(as_u(v), as_u(v), 0x122, 0xF, 0xF, false));
    if constexpr (LPR < 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(as_u(v), as_u(v), false, false);
        v = as_f(r[0]) + as_f(r[1]);
    }
    if constexpr (LPR < 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(as_u(v), as_u(v), false, false);
        v = as_f(r[0]) + as_f(r[1]);
    }
    return v;
}

}  // namespace
}  // namespace ftq
