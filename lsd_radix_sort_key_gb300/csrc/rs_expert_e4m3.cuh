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

// ---- values as they are loaded: 32-bit words of one float32 or two 16-bit elements

// The larger of `most` and the magnitudes in a word, in the elements' own bits (which
// are ordered as the magnitudes are); 16-bit ones by halves of the word.
template <typename T>
__device__ __forceinline__ uint32_t larger(uint32_t most, uint32_t word)
{
    if constexpr (sizeof(T) == 4) return max(most, word & 0x7FFFFFFFu);
    else return __vmaxu2(most, word & 0x7FFF7FFFu);
}

// Such a maximum as float bits.
template <typename T>
__device__ __forceinline__ uint32_t largest_bits(uint32_t most)
{
    if constexpr (sizeof(T) == 4) {
        return most;
    } else {
        const uint16_t m = (uint16_t)max(most & 0xFFFFu, most >> 16);
        if constexpr (__is_same(T, __half)) return __float_as_uint(__half2float(__ushort_as_half(m)));
        else return (uint32_t)m << 16;
    }
}

// An element's bits: those from here on are infinite or NaN.
template <typename T>
constexpr uint32_t kNotFiniteBits = sizeof(T) == 4 ? kNotFinite : __is_same(T, __half) ? 0x7C00u : 0x7F80u;

// `larger` over the finite elements alone.
template <typename T>
__device__ __forceinline__ uint32_t larger_finite(uint32_t most, uint32_t word)
{
    if constexpr (sizeof(T) == 4) {
        const uint32_t m = word & 0x7FFFFFFFu;
        return m < kNotFinite ? max(most, m) : most;
    } else {
        const uint32_t lo = word & 0x7FFFu, hi = word >> 16 & 0x7FFFu;
        return __vmaxu2(most, (lo < kNotFiniteBits<T> ? lo : 0u) | (hi < kNotFiniteBits<T> ? hi : 0u) << 16);
    }
}

// The word with NaN in place of infinities.
template <typename T>
__device__ __forceinline__ uint32_t without_infinities(uint32_t word)
{
    if constexpr (sizeof(T) == 4) {
        return __float_as_uint(finite_or_nan(__uint_as_float(word)));
    } else {
        if ((word & 0x7FFFu) == kNotFiniteBits<T>) word |= 1u;
        if ((word >> 16 & 0x7FFFu) == kNotFiniteBits<T>) word |= 0x10000u;
        return word;
    }
}

// Four elements, scaled and rounded.
template <typename T>
__device__ __forceinline__ uint32_t quantize4(const uint32_t* w, float inverse)
{
    if constexpr (sizeof(T) == 4) {
        return to_e4m3x4(__uint_as_float(w[0]) * inverse, __uint_as_float(w[1]) * inverse, __uint_as_float(w[2]) * inverse,
                         __uint_as_float(w[3]) * inverse);
    } else {
        float f[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (__is_same(T, __half)) {
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                f[2 * i] = v.x, f[2 * i + 1] = v.y;
            } else {
                f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
        return to_e4m3x4(f[0] * inverse, f[1] * inverse, f[2] * inverse, f[3] * inverse);
    }
}

}  // namespace rsx
