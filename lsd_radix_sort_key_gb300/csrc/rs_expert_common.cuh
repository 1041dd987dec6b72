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

// Programmatic dependent launch, used between the kernels of one call.  A
// kernel launched as the dependent of the one before it may start while that
// one still runs, once all its blocks have called start_next_grid() or ended;
// wait_prior_grid() returns when it has ended and its writes are visible (at
// once after a plain launch).  Every kernel that may be a dependent calls
// wait_prior_grid() before it ends, so that the end of a call's last kernel is
// the end of all.
__device__ __forceinline__ void wait_prior_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void start_next_grid() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// N adjacent elements: 16 bytes.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

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

// r, or zeros.
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> keep_if(bool kept, const Vec<T, N>& r)
{
    static_assert(sizeof(T) * N == 16, "16 bytes");
    uint4 u = *reinterpret_cast<const uint4*>(&r);
    u = make_uint4(kept ? u.x : 0, kept ? u.y : 0, kept ? u.z : 0, kept ? u.w : 0);
    return *reinterpret_cast<const Vec<T, N>*>(&u);
}

template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, N>& r)
{
    if constexpr (sizeof(T) * N == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&r);
    else p[0] = r.v[0];
}

// A vector as floats and back (one rounding each).
template <typename T>
__device__ __forceinline__ void to_floats(float (&f)[kVec<T>], const Vec<T, kVec<T>>& r)
{
    const uint4 u = *reinterpret_cast<const uint4*>(&r);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            f[i] = __uint_as_float(w[i]);
        } else if constexpr (__is_same(T, __half)) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        } else {  // bfloat16 is the high half of a float
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (__is_same(T, __half)) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

template <typename T>
__device__ __forceinline__ Vec<T, kVec<T>> from_floats(const float (&f)[kVec<T>])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
        else w[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
    }
    const uint4 u = make_uint4(w[0], w[1], w[2], w[3]);
    return *reinterpret_cast<const Vec<T, kVec<T>>*>(&u);
}

// Rows that are only element-aligned (an odd width, say) still move 16 bytes
// at a time: the vectors of a written row are cut where its addresses are
// multiples of 16, so element 0 of vector v of a row is v * kVec - lead(row),
// and a row's first and last vectors may be partial.  What is read for such
// a vector starts anywhere: it is taken from the two aligned 16-byte words
// around it (the second is the neighbouring lane's first and comes from L1).
// Those may reach into the rows before and after, so they are read only where
// both lie inside the matrix.
template <typename T>
__device__ __forceinline__ int lead(const T* row)
{
    return (int)((uintptr_t)row % 16 / sizeof(T));
}

// The two words, loaded without a branch so that many can be in flight, and
// then the elements [i, i + kVec) of a row of `width` in a matrix that occupies
// [begin, end); what lies outside the row is unspecified (clear_outside).
template <typename T>
struct Shifted {
    uint4 lo, hi;
    bool inside;
    __device__ __forceinline__ void load(const T* from, const T* begin, const T* end)
    {
        const uintptr_t p = (uintptr_t)from, a = p & ~(uintptr_t)15;
        inside = a >= (uintptr_t)begin && a + (a != p ? 32 : 16) <= (uintptr_t)end;
        lo = hi = make_uint4(0, 0, 0, 0);
        if (inside) lo = __ldg(reinterpret_cast<const uint4*>(a));
        if (inside && a != p) hi = __ldg(reinterpret_cast<const uint4*>(a) + 1);
    }
    __device__ __forceinline__ Vec<T, kVec<T>> get(const T* row, int i, int width) const
    {
        constexpr int N = kVec<T>;
        const uint32_t m = (uint32_t)(uintptr_t)(row + i) & 15;
        // drop the first m bytes: 8 and 4 bytes by selection, 2 by a funnel
        // shift (named values: an array indexed like this goes to memory)
        const bool b8 = m & 8, b4 = m & 4;
        const uint32_t p0 = b8 ? lo.z : lo.x, p1 = b8 ? lo.w : lo.y, p2 = b8 ? hi.x : lo.z, p3 = b8 ? hi.y : lo.w;
        const uint32_t p4 = b8 ? hi.z : hi.x, p5 = b8 ? hi.w : hi.y;
        uint4 u = make_uint4(b4 ? p1 : p0, b4 ? p2 : p1, b4 ? p3 : p2, b4 ? p4 : p3);
        if constexpr (sizeof(T) == 2) {
            const uint32_t last = b4 ? p5 : p4, bits = m & 2 ? 16 : 0;
            u = make_uint4(__funnelshift_r(u.x, u.y, bits), __funnelshift_r(u.y, u.z, bits),
                           __funnelshift_r(u.z, u.w, bits), __funnelshift_r(u.w, last, bits));
        }
        if (!inside) u = ends(row, i, width);
        return *reinterpret_cast<const Vec<T, N>*>(&u);
    }
    // At the matrix's two ends: element by element.
    __device__ __noinline__ static uint4 ends(const T* row, int i, int width)
    {
        constexpr int per = 4 / (int)sizeof(T);  // elements per word
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = 0;
#pragma unroll
            for (int h = 0; h < per; ++h) {
                const int c = i + j * per + h;
                if (c < 0 || c >= width) continue;
                if constexpr (per == 1) w[j] = reinterpret_cast<const uint32_t*>(row)[c];
                else w[j] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[c] << h * 16;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Zeros in place of the elements of vector [i, i + kVec) outside the row.
template <typename T>
__device__ __forceinline__ void clear_outside(float (&f)[kVec<T>], int i, int width)
{
    if (i >= 0 && i + kVec<T> <= width) return;
#pragma unroll
    for (int c = 0; c < kVec<T>; ++c)
        if (i + c < 0 || i + c >= width) f[c] = 0.0f;
}

template <typename T>
__device__ __forceinline__ void store_partial(T* row, int i, int width, const Vec<T, kVec<T>>& r)
{
    const uint4 u = *reinterpret_cast<const uint4*>(&r);
    if (i >= 0 && i + kVec<T> <= width) {
        *reinterpret_cast<uint4*>(row + i) = u;
    } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int c = 0; c < kVec<T>; ++c) {
            if (i + c < 0 || i + c >= width) continue;
            if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(row)[i + c] = w[c];
            else reinterpret_cast<uint16_t*>(row)[i + c] = (uint16_t)(w[c / 2] >> (c & 1) * 16);
        }
    }
}

// ---- host side

constexpr size_t kBlockSmem = 227 * 1024;  // that a block can have

// Lets a kernel be launched with up to `most` bytes of dynamic shared memory.
// The limit belongs to the kernel on the device, not to the calling thread, so
// `most` is what the kernel may ever need and no call lowers it under another
// thread's launch.
template <typename K>
bool allow_smem(K kernel, size_t most)
{
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) == cudaSuccess) return true;
    cudaGetLastError();
    return false;
}

template <typename... P, typename... A>
rs_status launch_kernel(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster,
                        bool dependent, const A&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (dependent) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return RS_ERR_CUDA;
    }
    return RS_OK;
}

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

// A matrix of rows: base aligned to its element; strides no longer than 2^32
// elements, so that with at most 2^30 rows span_bytes stays below 2^64.
inline bool valid_rows(const void* p, size_t elem, size_t width, size_t stride, bool may_broadcast)
{
    if (!p || (uintptr_t)p % elem) return false;
    if (stride > ((size_t)1 << 32)) return false;
    return stride >= width || (may_broadcast && stride == 0);
}

inline bool overlap(const void* a, size_t abytes, const void* b, size_t bbytes)
{
    if (!a || !b || abytes == 0 || bbytes == 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;  // (an end may pass 2^64: differences, not sums)
    return a0 < b0 ? b0 - a0 < abytes : a0 - b0 < bbytes;
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
