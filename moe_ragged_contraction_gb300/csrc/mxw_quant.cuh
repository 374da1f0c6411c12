// The MXFP8 scale rule, shared by the quantisers.
#pragma once

#include <stdint.h>

namespace mxw {

// Scale exponent of a 32-element block from the bit pattern of its amax
// (finite): the smallest e with amax <= 448 * 2^e, clamped to [-127, 127].
__device__ __forceinline__ int block_exponent(uint32_t amax_bits) {
    const int eb = static_cast<int>(amax_bits >> 23);
    if (eb == 0) return -127;  // zero or subnormal amax: below 448 * 2^-127
    // amax = 1.m * 2^(eb-127) = f * 2^(eb-126) with f = 1.m / 2 in [0.5, 1);
    // 448 = 0.875 * 2^9, so e = (eb - 126) - 9, plus one when f > 0.875 (1.m > 1.75)
    const int e = eb - 135 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(-127, min(127, e));
}

}  // namespace mxw
