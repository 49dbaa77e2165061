// expert_math.cuh -- SiLU(a) * b, shared by the epilogues of the bf16 and the int8
// expert products.
#pragma once

#include <cuda_runtime.h>

namespace moe {

// 2^x by the special-function unit's approximation, without flushing subnormal
// results to zero (ex2.approx.f32, no .ftz).
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// SiLU(a) * b in float32, with sigma(a) = 1 / (1 + e^-a) formed from
// t = e^-|a| = 2^(-|a| log2 e), which lies in (0, 1]: sigma = 1 / (1 + t) for
// a >= 0 and t / (1 + t) for a < 0.  The divisor 1 + t stays in (1, 2] for
// every a, where the fast division is accurate (to two float32 ulps; with the
// plain form a / (1 + e^-a) the divisor exceeds 2^126 once a < -87.3, where the
// fast division returns 0), and t underflows gradually rather than overflowing.
// Relative error: the rounding of -|a| log2 e moves t by up to |a| 2^-24
// relative, about 2^-17 at |a| = 100, far below the bf16 rounding of h that
// follows.
__device__ __forceinline__ float silu_times(float a, float b) {
    constexpr float kLog2e = 1.4426950408889634f;
    const float t = exp2_approx(-fabsf(a) * kLog2e);
    const float sigma = __fdividef(a >= 0.0f ? 1.0f : t, 1.0f + t);
    return a * sigma * b;
}

}  // namespace moe
