// rs_expert_groups.cuh -- the ragged side of the experts' products: row
// ranges read from the device and the list of row tiles they cut into, and
// the elementwise parts (activations and their derivatives).
#pragma once

#include "rs_expert_common.cuh"

namespace rsx {

// Row ranges of the experts and, after them, of the unused rows (range number
// `experts`), with the running number of row tiles before each.  `off` has
// experts + 2 entries, `tile` too (its last one is the total).  The given
// offsets are clamped to ascending values in [0, rows] with a first value of
// 0, so every tile lies inside the matrix whatever they hold.
struct Groups {
    uint32_t* off;
    uint32_t* tile;
    uint32_t experts;

    __host__ __device__ static constexpr size_t words(size_t experts) { return 2 * (experts + 2); }

    // All threads of the block call this; `mem` holds words(experts) words.
    // The unused rows get tiles only if `with_tail`.
    __device__ __forceinline__ static Groups make(uint32_t* mem, const int32_t* __restrict__ offsets,
                                                  uint32_t experts, uint32_t rows, uint32_t tile_rows, bool with_tail)
    {
        Groups g{mem, mem + experts + 2, experts};
        if (threadIdx.x < 32) {
            const uint32_t lane = threadIdx.x;
            uint32_t top = 0, tiles = 0;  // largest offset and number of tiles so far
            for (uint32_t e0 = 0; e0 < experts + 2; e0 += 32) {
                const uint32_t e = e0 + lane;  // one past the experts: the end of the unused rows
                uint32_t v = rows;
                if (e <= experts) {
                    const int32_t o = __ldg(offsets + e);
                    v = e == 0 || o < 0 ? 0u : (uint32_t)o < rows ? (uint32_t)o : rows;
                }
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, v, d);
                    if (lane >= d && up > v) v = up;
                }
                if (top > v) v = top;
                uint32_t before = __shfl_up_sync(0xFFFFFFFFu, v, 1);
                if (lane == 0) before = top;
                // tiles of range e - 1 = [before, v): counted into tile[e]
                const bool counted = e >= 1 && (e <= experts || (with_tail && e == experts + 1));
                uint32_t c = counted ? (v - before + tile_rows - 1) / tile_rows : 0u;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, c, d);
                    if (lane >= d) c += up;
                }
                if (e < experts + 2) {
                    g.off[e] = v;
                    g.tile[e] = tiles + c;
                }
                top = __shfl_sync(0xFFFFFFFFu, v, 31);
                tiles += __shfl_sync(0xFFFFFFFFu, c, 31);
            }
        }
        __syncthreads();
        return g;
    }

    __device__ __forceinline__ uint32_t tiles() const { return tile[experts + 1]; }

    // The range that row tile t (< tiles()) belongs to.
    __device__ __forceinline__ uint32_t find(uint32_t t) const
    {
        uint32_t lo = 0, hi = experts + 1;  // tile[lo] <= t < tile[hi]
        while (hi - lo > 1) {
            const uint32_t mid = (lo + hi) / 2;
            if (tile[mid] <= t) lo = mid;
            else hi = mid;
        }
        return lo;
    }
};

// Upper bound of Groups::tiles() for the grid: each range has at most one
// partly filled tile.
inline size_t max_tiles(size_t rows, size_t experts, size_t tile_rows) { return rows / tile_rows + experts + 1; }

// Activations and derivatives in float32.  FAST is for results that are
// rounded to 16 bits: the exponential and the reciprocal are the hardware's
// approximations (a few float32 ulps), and the normal cdf is
//     Phi(-|z|) = t (a1 + t (a2 + t (a3 + t (a4 + t a5)))) exp(-z^2 / 2) / 2,
//     t = 1 / (1 + p |z| / sqrt 2)
// (Abramowitz and Stegun 7.1.26, absolute error of erf at most 1.5e-7; taken on
// the negative side, so that the tail of z Phi(z) keeps its leading digits).
// z Phi(z) is off by at most 2.1e-7, relative to its value 3e-6 at z = -2, 5e-5 at
// -3, 5e-4 at -4 and 4e-3 at -6 (rounding to binary16 costs 5e-4 and more below
// 6e-5, to bfloat16 4e-3; 0.5 z (1 + erf) in float32 is off by 1e-7 there too).
// In the products' epilogue gelu with the library's erfcf took 120 us of a 456
// us product (32768 x 2048 x 4096).
__device__ __forceinline__ float fast_exp2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float fast_reciprocal(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float fast_sigmoid(float z) { return fast_reciprocal(1.0f + fast_exp2(-kLog2e * z)); }

// Phi(z); *density receives exp(-z^2 / 2).
__device__ __forceinline__ float fast_normal_cdf(float z, float* density)
{
    const float t = fast_reciprocal(fmaf(0.3275911f * 0.70710678118654752f, fabsf(z), 1.0f));
    const float e = fast_exp2(z * z * (-0.5f * kLog2e));
    const float poly = fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f), 0.5f * 1.421413741f),
                                    0.5f * -0.284496736f),
                            0.5f * 0.254829592f);
    const float low = t * poly * e;
    *density = e;
    return z < 0.0f ? low : 1.0f - low;
}

template <int ACT, bool FAST>
__device__ __forceinline__ float activate(float z)
{
    if constexpr (ACT == RS_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    if constexpr (ACT == RS_ACT_GELU) {
        float density;
        return FAST ? z * fast_normal_cdf(z, &density) : 0.5f * z * erfcf(-0.70710678118654752f * z);
    }
    if constexpr (ACT == RS_ACT_SILU) return FAST ? z * fast_sigmoid(z) : z / (1.0f + expf(-z));
    return z;
}

template <int ACT, bool FAST>
__device__ __forceinline__ float activate_grad(float z)
{
    if constexpr (ACT == RS_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == RS_ACT_GELU) {
        if constexpr (FAST) {
            float density;
            const float phi = fast_normal_cdf(z, &density);
            return fmaf(z * 0.39894228040143268f, density, phi);
        }
        return 0.5f * erfcf(-0.70710678118654752f * z) + z * (0.39894228040143268f * expf(-0.5f * z * z));
    }
    if constexpr (ACT == RS_ACT_SILU) {
        const float s = FAST ? fast_sigmoid(z) : 1.0f / (1.0f + expf(-z));
        return s * (1.0f + z * (1.0f - s));
    }
    return 1.0f;
}

}  // namespace rsx
