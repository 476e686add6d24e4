// The two roundings of the NVFP4 format: a block's scale up to E4M3, a value to the nearest E2M1 code.
#pragma once

#include <stdint.h>

namespace qerl {

// Smallest non-negative finite E4M3 value >= t, as a byte (saturates at 448).
__device__ __forceinline__ uint32_t e4m3_ceil(float t)
{
    if (!(t > 0.0f)) return 0u;
    if (t > 448.0f) return 0x7Eu;
    const uint32_t u = __float_as_uint(t);
    const int e = (int)(u >> 23) - 127;
    if (e < -6) {
        // Subnormal E4M3 range m * 2^-9 (m = 8 is 2^-6, the first normal, whose
        // byte 0x08 continues the sequence).  t * 512 is exact.
        return (uint32_t)ceilf(t * 512.0f);
    }
    uint32_t m3 = (u >> 20) & 7u, E = (uint32_t)(e + 7);
    if (u & 0xFFFFFu) {  // bits below the 3 kept mantissa bits: round up
        if (++m3 == 8u) {
            m3 = 0u;
            ++E;
        }
    }
    return (E << 3) | m3;
}

// E2M1 code of q: nearest of {0,.5,1,1.5,2,3,4,6} in magnitude, ties to the even
// code (the midpoints .25,1.25,2.5,5 fall down, .75,1.75,3.5 fall up), > 6
// saturates; a zero result is code 0 whatever the sign.
__device__ __forceinline__ uint32_t e2m1_code(float q)
{
    const float a = fabsf(q);
    uint32_t c = (uint32_t)(a > 0.25f) + (uint32_t)(a >= 0.75f) + (uint32_t)(a > 1.25f) + (uint32_t)(a >= 1.75f) +
                 (uint32_t)(a > 2.5f) + (uint32_t)(a >= 3.5f) + (uint32_t)(a > 5.0f);
    return (c != 0u && q < 0.0f) ? (c | 8u) : c;
}

}  // namespace qerl
