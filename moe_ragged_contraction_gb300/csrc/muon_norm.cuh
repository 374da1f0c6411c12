// Frobenius norm of a matrix from two fp32 sums, for the kernels of
// mxfp8_muon_update.
#pragma once

#include <cuda_runtime.h>

namespace mxw {

constexpr float NORM_UP = 0x1p100f;
constexpr float NORM_LOW = 0x1p-100f;

// sum = sum of u^2, up = sum of (2^100 u)^2, scale a power of two. Returns (pre,
// inv) with scale * u / (||u|| + eps) = (u pre) inv. Squares below 2^-149 are lost
// in `sum`: of up to 2^30 elements they matter less than its rounding while it is
// at least 2^-100. Below that every |u| is under 2^-50, so `up` is finite, and the
// square of the smallest subnormal (2^-149) is 2^-98 in it. NaN where the
// sum is not finite: the whole matrix comes out as NaN.
__device__ __forceinline__ float2 norm_factors(float sum, float up, float eps, float scale) {
    if (!(sum <= 3.4028235e38f)) return make_float2(1.f, __int_as_float(0x7fffffff));
    if (sum >= NORM_LOW) return make_float2(1.f, scale / (sqrtf(sum) + eps));
    return make_float2(NORM_UP, scale / (sqrtf(up) + eps * NORM_UP));
}

}  // namespace mxw
