// rs_expert_common.cuh -- what the expert operators share: element types,
// 16-byte vectors, and the host-side checks of their arguments.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "rs_experts.h"

namespace rsx {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v)
{
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (__is_same(T, __half)) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// N adjacent elements moved as one access; N * sizeof(T) is 16 (rows whose
// base and stride are multiples of 16 bytes) or one element.
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T v[N];
};

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T* p)
{
    Vec<T, N> r;
    if constexpr (sizeof(T) * N == 16) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
        r = *reinterpret_cast<const Vec<T, N>*>(&u);
    } else {
        static_assert(N == 1, "one element or 16 bytes");
        r.v[0] = *p;
    }
    return r;
}

template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, N>& r)
{
    if constexpr (sizeof(T) * N == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&r);
    else p[0] = r.v[0];
}

// ---- host side

// A number carried as a type, for generic lambdas.
template <int N>
struct Int {
    static constexpr int value = N;
};

inline bool valid_type(int t) { return t == RS_FLOAT32 || t == RS_FLOAT16 || t == RS_BFLOAT16; }
inline size_t type_bytes(int t) { return t == RS_FLOAT32 ? 4 : 2; }

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline size_t ceil_div(size_t a, size_t b) { return (a + b - 1) / b; }

// Bytes that `rows` rows of `width` elements span at a row stride in elements.
inline size_t span_bytes(size_t rows, size_t width, size_t stride, size_t elem)
{
    return rows == 0 || width == 0 ? 0 : ((rows - 1) * stride + width) * elem;
}

// A matrix of rows: base aligned to its element; strides no longer than 2^40
// elements, so that no byte offset inside it passes 2^63.
inline bool valid_rows(const void* p, size_t elem, size_t width, size_t stride, bool may_broadcast)
{
    if (!p || (uintptr_t)p % elem) return false;
    if (stride > ((size_t)1 << 32)) return false;
    return stride >= width || (may_broadcast && stride == 0);
}

inline bool overlap(const void* a, size_t abytes, const void* b, size_t bbytes)
{
    if (!a || !b || abytes == 0 || bbytes == 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + bbytes && b0 < a0 + abytes;
}

struct Range {
    const void* p;
    size_t bytes;
};

// True if any of the first `outs` ranges overlaps any other range.
inline bool any_alias(const Range* r, int outs, int all)
{
    for (int i = 0; i < outs; ++i)
        for (int j = i + 1; j < all; ++j)
            if (overlap(r[i].p, r[i].bytes, r[j].p, r[j].bytes)) return true;
    return false;
}

inline bool aligned16(const void* p, size_t stride, size_t elem)
{
    return (uintptr_t)p % 16 == 0 && stride * elem % 16 == 0;
}

}  // namespace rsx
