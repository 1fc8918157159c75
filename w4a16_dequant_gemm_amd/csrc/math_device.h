// math_device.h -- device functions of one number that several sources use.
#pragma once
#include <hip/hip_runtime.h>

namespace {

// exp(x) = 2^n (1 + l) exp2(h) with h + n = x * log2 e rounded and l the natural
// logarithm of what that rounding and the low part of log2 e lost: good to about
// one unit in the last place.
__device__ __forceinline__ float exp_scaled(float x, float n) {
#pragma clang fp contract(off)   // h + n is the rounded h that l belongs to
    constexpr float kLog2e = 0x1.715476p+0f, kLn2 = 0x1.62e43p-1f;
    constexpr float kLowLn2 = 0x1.4ae0cp-26f * kLn2;   // the low part of log2 e, times ln 2
    const float h = x * kLog2e;
    const float l = __builtin_fmaf(__builtin_fmaf(x, kLog2e, -h), kLn2, x * kLowLn2);
    const float e = __builtin_amdgcn_exp2f(h + n);
    return __builtin_fmaf(e, l, e);
}

}  // namespace
