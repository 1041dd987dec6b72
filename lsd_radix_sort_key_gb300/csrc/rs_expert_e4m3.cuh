// rs_expert_e4m3.cuh -- blocks of 128 values in 8 bits with a shared scale:
// the scale's choice and the rounding (definitions in rs_expert_block.h).
#pragma once

#include "rs_expert_block.h"
#include "rs_expert_common.cuh"

namespace rsx {

constexpr uint32_t kNotFinite = 0x7F800000u;  // magnitudes from here on are infinite or NaN
constexpr uint32_t kScaleOne = 127;

// The scale byte of a block whose largest finite magnitude has the float bits
// `amax`.  448 = 1.75 * 2^8, so the exponent is that of amax less 8, and one
// more where its significand is above 1.75.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax)
{
    if (amax == 0) return kScaleOne;
    const int e = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e < 1 ? 1u : (uint32_t)e;
}

// 1 / scale, exact (bytes from 1 to 247).
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Two values to e4m3, the first in the low byte; NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d)
{
    return to_e4m3x2(a, b) | to_e4m3x2(c, d) << 16;
}

__device__ __forceinline__ uint32_t magnitude(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// f, or NaN where it is infinite (the conversion above would make 448 of that).
__device__ __forceinline__ float finite_or_nan(float f)
{
    return magnitude(f) == kNotFinite ? __uint_as_float(0x7FC00000u) : f;
}

}  // namespace rsx
