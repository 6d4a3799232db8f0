// kq_step.h -- what the translation units of include/kqstep.h share.
#pragma once

#include "kq_kv.h"
#include "kqstep.h"

namespace kq {
namespace step {

typedef uint64_t u64;

// fp64 across lanes: the two halves go separately.
template <int CTRL> __device__ __forceinline__ double dpp_d(double x) {
    const u64 b = __builtin_bit_cast(u64, x);
    const u32 lo = (u32)__builtin_amdgcn_update_dpp(0, (int)(u32)b, CTRL, 0xF, 0xF, false);
    const u32 hi = (u32)__builtin_amdgcn_update_dpp(0, (int)(u32)(b >> 32), CTRL, 0xF, 0xF, false);
    return __builtin_bit_cast(double, ((u64)hi << 32) | lo);
}
__device__ __forceinline__ double swap16_sum(double x) {
    const u64 b = __builtin_bit_cast(u64, x);
    const auto l = __builtin_amdgcn_permlane16_swap((u32)b, (u32)b, false, false);
    const auto h = __builtin_amdgcn_permlane16_swap((u32)(b >> 32), (u32)(b >> 32), false, false);
    return __builtin_bit_cast(double, ((u64)(u32)h[0] << 32) | (u32)l[0]) +
           __builtin_bit_cast(double, ((u64)(u32)h[1] << 32) | (u32)l[1]);
}
__device__ __forceinline__ double swap32_sum(double x) {
    const u64 b = __builtin_bit_cast(u64, x);
    const auto l = __builtin_amdgcn_permlane32_swap((u32)b, (u32)b, false, false);
    const auto h = __builtin_amdgcn_permlane32_swap((u32)(b >> 32), (u32)(b >> 32), false, false);
    return __builtin_bit_cast(double, ((u64)(u32)h[0] << 32) | (u32)l[0]) +
           __builtin_bit_cast(double, ((u64)(u32)h[1] << 32) | (u32)l[1]);
}

// Sum over groups of LANES (16, 32, 64) neighbouring lanes, in every lane of
// the group; pairs are added in the order of group_sum's tree.
template <int LANES> __device__ __forceinline__ double sum_d(double x) {
    x += dpp_d<0xB1>(x);      // quad_perm 1,0,3,2
    x += dpp_d<0x4E>(x);      // quad_perm 2,3,0,1
    x += dpp_d<0x141>(x);     // row_half_mirror
    x += dpp_d<0x140>(x);     // row_mirror
    if (LANES >= 32) x = swap16_sum(x);
    if (LANES >= 64) x = swap32_sum(x);
    return x;
}

} // namespace step
} // namespace kq
