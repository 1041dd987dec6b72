// rs_expert_rows.cu -- the row movers of the expert operators: dispatch,
// combine and combine's gradient (formulas in rs_experts.h).
//
// All three go token by token: a token's own row is read (or written) once
// and its K expert rows, which lie anywhere, are each written or read once,
// whole and in order.  So the bytes moved are the least possible,
//   dispatch      (1 + K) rows per token
//   combine       (1 + K)
//   combine grad  (1 + 2K)
// (where rows are only element-aligned, dispatch and combine's gradient load the
// token's own row again for every slot, from the caches after the first),
// with no use of `order`, and the sum over a token's slots is a loop in one
// thread, in slot order: no atomics, the same result every time.
#include <type_traits>

#include "rs_expert_common.cuh"

namespace {

using namespace rsx;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Rows below this belong to experts.
__device__ __forceinline__ uint32_t routed_rows(const int32_t* routed, uint32_t slots_total)
{
    const int32_t r = __ldg(routed);
    return r < 0 ? 0u : (uint32_t)r < slots_total ? (uint32_t)r : slots_total;
}

// A row is cut into vectors of 16 bytes, and these into pieces of 32 * V
// (one warp, V per lane).  SHIFT: rows are only element-aligned, and the
// vectors are cut by the written row's address (lead, Shifted,
// store_partial in rs_expert_common.cuh).
template <typename T, bool SHIFT>
__device__ __forceinline__ uint32_t row_vecs(uint32_t width)
{
    constexpr uint32_t N = kVec<T>;
    return (width + N - 1) / N + (SHIFT ? 1 : 0);  // a lead adds at most one
}

// GL lanes take one token (32, or 16 or 8 where a row has no more vectors, so
// that a warp takes 2 or 4 tokens); its slots are loaded GL at a time, one per
// lane, and handed around by shuffles, in which the whole warp takes part.
template <typename W, int GL>
struct Slots {
    uint32_t row = 0xFFFFFFFFu;
    float weight = 1.0f;
    __device__ __forceinline__ void load(const int32_t* position, const W* weights, size_t first, uint32_t count)
    {
        const uint32_t lane = threadIdx.x % GL;
        row = 0xFFFFFFFFu;
        if (lane < count) {
            row = (uint32_t)__ldg(position + first + lane);
            if (weights) weight = to_float(weights[first + lane]);
        }
    }
    __device__ __forceinline__ uint32_t row_of(uint32_t k) const
    {
        return __shfl_sync(0xFFFFFFFFu, row, k & (GL - 1), GL);
    }
    __device__ __forceinline__ float weight_of(uint32_t k) const
    {
        return __shfl_sync(0xFFFFFFFFu, weight, k & (GL - 1), GL);
    }
};

// One warp moves one piece of a token's row to its K places.  Written bytes
// bound it: 16384 x 8 rows of 4 KB move at 6.5 TB/s with V = 2, 5.4 when each
// slot's position was loaded on its own.
template <typename T, bool SHIFT, int GL, int V>
__global__ void __launch_bounds__(kThreads) k_dispatch(const T* __restrict__ x, size_t x_stride,
                                                       const int32_t* __restrict__ position,
                                                       const int32_t* __restrict__ routed, uint32_t slots_total,
                                                       uint32_t tokens, uint32_t slots, uint32_t width,
                                                       uint32_t pieces, const T* __restrict__ x_begin,
                                                       const T* __restrict__ x_end, T* __restrict__ out,
                                                       size_t out_stride)
{
    constexpr int N = kVec<T>;
    const uint32_t item = blockIdx.x * (kThreads / GL) + threadIdx.x / GL, lane = threadIdx.x % GL;
    uint32_t t = item / pieces;
    const bool live = t < tokens;
    if (GL == 32 && !live) return;
    const uint32_t v0 = (item - t * pieces) * (GL * V) + lane, vecs = live ? row_vecs<T, SHIFT>(width) : 0;
    if (!live) t = 0;  // beside live tokens, for the shuffles
    const uint32_t limit = routed_rows(routed, slots_total);
    const T* row = x + t * x_stride;
    Vec<T, N> r[V];
    if constexpr (!SHIFT) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (v0 + i * GL < vecs) r[i] = load_vec<T, N>(row + (size_t)(v0 + i * GL) * N);
    }
    for (uint32_t k0 = 0; k0 < slots; k0 += GL) {
        const uint32_t here = min(slots - k0, (uint32_t)GL);
        Slots<float, GL> sl;
        sl.load(position, nullptr, (size_t)t * slots + k0, here);
        for (uint32_t k = 0; k < here; ++k) {
            const uint32_t p = sl.row_of(k);
            if (!live || p >= slots_total) continue;
            T* to = out + p * out_stride;
            const bool kept = p < limit;
            if constexpr (SHIFT) {
                const int skip = lead(to);
                Shifted<T> w[V];
#pragma unroll
                for (int i = 0; i < V; ++i) w[i].load(row + ((int)((v0 + i * GL) * N) - skip), x_begin, x_end);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int at = (int)((v0 + i * GL) * N) - skip;
                    if (at < (int)width)
                        store_partial<T>(to, at, (int)width, keep_if(kept, w[i].get(row, at, (int)width)));
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (v0 + i * GL < vecs) store_vec<T, N>(to + (size_t)(v0 + i * GL) * N, keep_if(kept, r[i]));
            }
        }
    }
}

// One warp sums `span` pieces of a token's row over its slots, G slots at a
// time, so G * V row loads per lane are in flight before the first is used.
// Random reads bound it, and the choice of G, V and span is the memory
// system's: measured for 16384 x 8 rows of 4 KB, in TB/s, G x V = 8x1 3.6,
// 4x1 5.2, 4x2 6.6, 2x2 6.5, 2x8 5.7; 65536 x 1 rows of 8 KB: 2x2 4.8 with
// span 1, 6.1 with span 4, 1x4 6.6 with span 4; 8192 x 2 of 16 KB: 2x2 5.6,
// 6.2, 6.4 with span 1, 2, 4.
template <typename T, typename W, bool SHIFT, int G, int V, int GL>
__global__ void __launch_bounds__(kThreads) k_combine(const T* __restrict__ y, size_t y_stride,
                                                      const W* __restrict__ weights,
                                                      const int32_t* __restrict__ position,
                                                      const int32_t* __restrict__ routed, uint32_t slots_total,
                                                      uint32_t tokens, uint32_t slots, uint32_t width, uint32_t parts,
                                                      uint32_t span, const T* __restrict__ y_end, T* __restrict__ out,
                                                      size_t out_stride)
{
    constexpr int N = kVec<T>;
    const uint32_t item = blockIdx.x * (kThreads / GL) + threadIdx.x / GL, lane = threadIdx.x % GL;
    uint32_t t = item / parts;
    const bool live = t < tokens;
    if (GL == 32 && !live) return;
    const uint32_t part = item - t * parts;
    if (!live) t = 0;  // beside live tokens, for the shuffles
    const uint32_t limit = live ? routed_rows(routed, slots_total) : 0, vecs = row_vecs<T, SHIFT>(width);
    T* to = out + t * out_stride;
    const int skip = SHIFT ? lead(to) : 0;
    const uint32_t first = part * span * (GL * V), last = min(vecs, first + span * (GL * V));
    Slots<W, GL> sl;
    sl.load(position, weights, (size_t)t * slots, min(slots, (uint32_t)GL));
    for (uint32_t v0 = first; v0 < last; v0 += GL * V) {
        float acc[V][N] = {};
        for (uint32_t k0 = 0; k0 < slots; k0 += GL) {
            const uint32_t here = min(slots - k0, (uint32_t)GL);
            if (slots > GL) sl.load(position, weights, (size_t)t * slots + k0, here);
            for (uint32_t k = 0; k < here; k += G) {
                using Loaded = std::conditional_t<SHIFT, Shifted<T>, Vec<T, N>>;
                Loaded r[G][V];
                bool kept[G];
                uint32_t p[G];
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    p[j] = sl.row_of(k + j);
                    kept[j] = k + j < here && p[j] < limit;
                    if (!kept[j]) continue;
                    const T* from = y + p[j] * y_stride;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const uint32_t v = v0 + i * GL + lane;
                        if constexpr (SHIFT) r[j][i].load(from + ((int)(v * N) - skip), y, y_end);
                        else if (v < vecs) r[j][i] = load_vec<T, N>(from + (size_t)v * N);
                    }
                }
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const float w = sl.weight_of(k + j);
                    if (!kept[j]) continue;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float f[N];
                        if constexpr (SHIFT)
                            to_floats<T>(f, r[j][i].get(y + p[j] * y_stride, (int)((v0 + i * GL + lane) * N) - skip,
                                                        (int)width));
                        else to_floats<T>(f, r[j][i]);
#pragma unroll
                        for (int c = 0; c < N; ++c) acc[i][c] = fmaf(w, f[c], acc[i][c]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t v = v0 + i * GL + lane;
            if (!live || v >= vecs) continue;
            const Vec<T, N> o = from_floats<T>(acc[i]);
            if constexpr (SHIFT) store_partial<T>(to, (int)(v * N) - skip, (int)width, o);
            else store_vec<T, N>(to + (size_t)v * N, o);
        }
    }
}

// WT warps take one token and walk its row together, V vectors per lane and
// G slots at a time; a slot's dot product is summed over the lanes at the end
// (within the warp by shuffles, over the warps through shared memory), always
// in the same order.  A lane's part is one chain of float32 multiply-adds (width
// / 32 of them): 4096 float32 elements come out 2.1e-7 off in the 2-norm, 1.3e-7
// when summed in pairs.  Up to 8 slots per walk.  G = V = 2 measured best or
// within 3% of it from 1 to 8 slots (16384 x 8 rows of 4 KB 6.6 TB/s; 65536 x 1
// of 8 KB 6.4 against 3.5 with G x V = 8x1); rows of at most 32 vectors leave
// half of V = 2 idle and take 4x1 (131072 x 8 rows of 512 bytes 6.6 against 5.7).
// Unaligned rows: each slot's row has a lead of its own, so dout is read once
// per slot, from L1 after the first.  Rows of 16-bit types read it where it is
// used, which leaves the registers for more rows in flight (16384 x 8 rows of
// 2047 bf16 363 us against 409, 131072 x 8 of 129 408 against 486); 32-bit rows
// along with y's (8191 x 2 of 4095 162 us against 195).
template <typename T, typename W, bool SHIFT, int G, int V, int WT, int GL>
__global__ void __launch_bounds__(kThreads) k_combine_grad(
    const T* __restrict__ dout, size_t dout_stride, const T* __restrict__ y, size_t y_stride,
    const W* __restrict__ weights, const int32_t* __restrict__ position, const int32_t* __restrict__ routed,
    uint32_t slots_total, uint32_t tokens, uint32_t slots, uint32_t width, const T* __restrict__ dout_end,
    const T* __restrict__ y_end, T* __restrict__ dy, size_t dy_stride,
    W* __restrict__ dweights)
{
    constexpr int N = kVec<T>, kSlots = 8;
    constexpr bool early = SHIFT && sizeof(T) == 4;
    __shared__ float part[kWarps][kSlots];
    static_assert(WT == 1 || GL == 32, "several warps or part of one");
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % GL;
    const uint32_t t = WT > 1 ? blockIdx.x * (kWarps / WT) + warp / WT : blockIdx.x * (kThreads / GL) + threadIdx.x / GL;
    const bool live = t < tokens;  // no early return: the block has barriers when WT > 1
    const uint32_t limit = routed_rows(routed, slots_total), vecs = live ? row_vecs<T, SHIFT>(width) : 0;
    const T* grad = dout + (live ? t : 0) * dout_stride;
    for (uint32_t k0 = 0; k0 < slots; k0 += kSlots) {
        const uint32_t here = live ? min(slots - k0, (uint32_t)kSlots) : 0, most = min(slots - k0, (uint32_t)kSlots);
        Slots<W, GL> sl;
        sl.load(position, weights, (size_t)t * slots + k0, here);
        float dot[kSlots] = {};
        for (uint32_t v0 = WT > 1 ? (warp % WT) * (GL * V) : 0; v0 < row_vecs<T, SHIFT>(width); v0 += GL * V * WT) {
            Vec<T, N> d[V];
            if constexpr (!SHIFT) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (v0 + i * GL + lane < vecs) d[i] = load_vec<T, N>(grad + (size_t)(v0 + i * GL + lane) * N);
            }
#pragma unroll
            for (int k = 0; k < kSlots; k += G) {
                if (k >= most) break;
                using Loaded = std::conditional_t<SHIFT, Shifted<T>, Vec<T, N>>;
                Loaded r[G][V], g[early ? G : 1][V];
                uint32_t p[G];
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    p[j] = sl.row_of(k + j);
                    if (k + j >= here) p[j] = 0xFFFFFFFFu;
                    if (p[j] >= limit) continue;
                    const T* from = y + p[j] * y_stride;
                    const int skip = SHIFT ? lead(dy + p[j] * dy_stride) : 0;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const uint32_t v = v0 + i * GL + lane;
                        if constexpr (SHIFT) {
                            r[j][i].load(from + ((int)(v * N) - skip), y, y_end);
                            if constexpr (early) g[j][i].load(grad + ((int)(v * N) - skip), dout, dout_end);
                        } else if (v < vecs) {
                            r[j][i] = load_vec<T, N>(from + (size_t)v * N);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const float w = sl.weight_of(k + j);
                    if (p[j] >= slots_total) continue;
                    T* to = dy + p[j] * dy_stride;
                    const int skip = SHIFT ? lead(to) : 0;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const uint32_t v = v0 + i * GL + lane;
                        if (v >= vecs) continue;
                        Vec<T, N> o{};
                        if (p[j] < limit) {
                            float q[N], f[N], e[N];
                            if constexpr (SHIFT) {
                                const int at = (int)(v * N) - skip;
                                Loaded late;
                                if constexpr (!early) late.load(grad + at, dout, dout_end);
                                to_floats<T>(q, (early ? g[j][i] : late).get(grad, at, (int)width));
                                to_floats<T>(f, r[j][i].get(y + p[j] * y_stride, at, (int)width));
                                clear_outside<T>(q, at, (int)width);
                                clear_outside<T>(f, at, (int)width);
                            } else {
                                to_floats<T>(q, d[i]);
                                to_floats<T>(f, r[j][i]);
                            }
#pragma unroll
                            for (int c = 0; c < N; ++c) {
                                dot[k + j] = fmaf(q[c], f[c], dot[k + j]);
                                e[c] = w * q[c];
                            }
                            o = from_floats<T>(e);
                        }
                        if constexpr (SHIFT) store_partial<T>(to, (int)(v * N) - skip, (int)width, o);
                        else store_vec<T, N>(to + (size_t)v * N, o);
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
#pragma unroll
            for (int d = GL / 2; d; d >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
        float sum = 0.0f;  // lane j: slot j's
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
            if (lane == j) sum = dot[j];
        if constexpr (WT > 1) {
            __syncthreads();
            if (lane < kSlots) part[warp][lane] = sum;
            __syncthreads();
            sum = 0.0f;
            if (warp % WT == 0 && lane < kSlots)
                for (int i = 0; i < WT; ++i) sum += part[warp + i][lane];
        }
        if (warp % WT == 0 && lane < here) dweights[(size_t)t * slots + k0 + lane] = from_float<W>(sum);
    }
}

// Tokens per launch: keeps warp numbers below 2^31.
size_t tokens_per_launch(size_t pieces) { return ((size_t)1 << 30) / pieces; }

struct RowArgs {
    size_t tokens, width;
    int slots;
    const int32_t *position, *routed;
    cudaStream_t stream;
    uint32_t slots_total() const { return (uint32_t)(tokens * (size_t)slots); }
};

rs_status check_rows(const RowArgs& a, int type)
{
    if (!valid_type(type) || a.slots < 1 || a.width > RS_EXPERT_WIDTH_MAX) return RS_ERR_INVALID_ARG;
    if (a.tokens > RS_EXPERT_SLOTS_MAX || a.tokens * (size_t)a.slots > RS_EXPERT_SLOTS_MAX) return RS_ERR_INVALID_ARG;
    if (a.tokens == 0) return RS_OK;
    if (!a.position || !a.routed || (uintptr_t)a.position % 4 || (uintptr_t)a.routed % 4) return RS_ERR_INVALID_ARG;
    return RS_OK;
}

rs_status launched() { return cudaGetLastError() == cudaSuccess ? RS_OK : RS_ERR_CUDA; }

// Lanes per token for rows of so many vectors (97483 x 6 rows of 105 bf16, 15
// vectors: combine 59.6 us with 16, 98 with 32).  17 to 24 vectors take three
// steps of 8 lanes rather than one of 32 (131072 x 8 rows of 129 bf16: dispatch
// 130 us against 200, combine 127 against 160, its gradient 275 against 409; of
// 192 74, 84, 144 against 74, 89, 162; only combine of unaligned 32-bit rows
// loses, 40348 x 8 of 71 60 against 54).
inline int lanes_for(uint32_t vecs)
{
    return vecs <= 8 || (vecs > 16 && vecs <= 24) ? 8 : vecs <= 16 ? 16 : 32;
}

template <typename T, bool SHIFT>
rs_status run_dispatch(const RowArgs& a, const T* x, size_t x_stride, T* out, size_t out_stride)
{
    const uint32_t vecs = (uint32_t)ceil_div(a.width, kVec<T>) + SHIFT;
    auto run = [&](auto kernel, int lanes, int v) {
        const uint32_t pieces = (uint32_t)ceil_div(vecs, lanes * v);
        const size_t step = tokens_per_launch(pieces);
        for (size_t t = 0; t < a.tokens; t += step) {
            const uint32_t here = (uint32_t)(a.tokens - t < step ? a.tokens - t : step);
            kernel<<<(unsigned)ceil_div((size_t)here * pieces, kThreads / lanes), kThreads, 0, a.stream>>>(
                x + t * x_stride, x_stride, a.position + t * a.slots, a.routed, a.slots_total(), here, a.slots,
                (uint32_t)a.width, pieces, x, x + (a.tokens - 1) * x_stride + a.width, out, out_stride);
        }
        return launched();
    };
    switch (lanes_for(vecs)) {
    case 8: return run(k_dispatch<T, SHIFT, 8, 1>, 8, 1);
    case 16: return run(k_dispatch<T, SHIFT, 16, 1>, 16, 1);
    default: return run(k_dispatch<T, SHIFT, 32, 2>, 32, 2);
    }
}

// Warps that keep every SM's memory pipeline full several times over; below
// this the spans of k_combine are cut to spread the work.
constexpr size_t kManyWarps = 16384;

template <typename T, typename W, bool SHIFT, int G, int V, int GL>
rs_status launch_combine(const RowArgs& a, const T* y, size_t y_stride, const W* weights, T* out, size_t out_stride,
                         uint32_t span)
{
    const uint32_t vecs = (uint32_t)ceil_div(a.width, kVec<T>) + SHIFT, pieces = (uint32_t)ceil_div(vecs, GL * V);
    while (span > 1 && a.tokens * ceil_div(pieces, span) < kManyWarps) span /= 2;
    const uint32_t parts = (uint32_t)ceil_div(pieces, span);
    const size_t step = tokens_per_launch(parts);
    for (size_t t = 0; t < a.tokens; t += step) {
        const uint32_t here = (uint32_t)(a.tokens - t < step ? a.tokens - t : step);
        k_combine<T, W, SHIFT, G, V, GL><<<(unsigned)ceil_div((size_t)here * parts, kThreads / GL), kThreads, 0, a.stream>>>(
            y, y_stride, weights ? weights + t * a.slots : nullptr, a.position + t * a.slots, a.routed,
            a.slots_total(), here, a.slots, (uint32_t)a.width, parts, span,
            y + ((size_t)a.slots_total() - 1) * y_stride + a.width, out + t * out_stride, out_stride);
    }
    return launched();
}

template <typename T, typename W, bool SHIFT>
rs_status run_combine(const RowArgs& a, const T* y, size_t y_stride, const W* weights, T* out, size_t out_stride)
{
    const uint32_t vecs = (uint32_t)ceil_div(a.width, kVec<T>) + SHIFT;
    if (lanes_for(vecs) == 8) return launch_combine<T, W, SHIFT, 4, 1, 8>(a, y, y_stride, weights, out, out_stride, 1);
    if (vecs <= 16) return launch_combine<T, W, SHIFT, 4, 1, 16>(a, y, y_stride, weights, out, out_stride, 1);
    if (vecs <= 32) return launch_combine<T, W, SHIFT, 4, 1, 32>(a, y, y_stride, weights, out, out_stride, 1);
    if (a.slots == 1) return launch_combine<T, W, SHIFT, 1, 4, 32>(a, y, y_stride, weights, out, out_stride, 4);
    return launch_combine<T, W, SHIFT, 2, 2, 32>(a, y, y_stride, weights, out, out_stride, 2);
}

template <typename T, typename W, bool SHIFT>
rs_status run_combine_grad(const RowArgs& a, const T* dout, size_t dout_stride, const T* y, size_t y_stride,
                           const W* weights, T* dy, size_t dy_stride, W* dweights)
{
    auto run = [&](auto kernel, int per_block) {
        kernel<<<(unsigned)ceil_div(a.tokens, per_block), kThreads, 0, a.stream>>>(
            dout, dout_stride, y, y_stride, weights, a.position, a.routed, a.slots_total(), (uint32_t)a.tokens,
            (uint32_t)a.slots, (uint32_t)a.width, dout + (a.tokens - 1) * dout_stride + a.width,
            y + ((size_t)a.slots_total() - 1) * y_stride + a.width, dy, dy_stride, dweights);
        return launched();
    };
    const uint32_t vecs = (uint32_t)ceil_div(a.width, kVec<T>) + SHIFT;
    // With few tokens a row's steps are what lasts (1000 x 8 rows of 192 bf16:
    // 5.7 us in one step, 8.1 in three).
    const bool few = a.tokens < 2048;
    if (vecs <= 8 || (!few && lanes_for(vecs) == 8)) return run(k_combine_grad<T, W, SHIFT, 4, 1, 1, 8>, kThreads / 8);
    if (vecs <= 16) return run(k_combine_grad<T, W, SHIFT, 4, 1, 1, 16>, kThreads / 16);
    if (vecs <= 32) return run(k_combine_grad<T, W, SHIFT, 4, 1, 1, 32>, kWarps);
    // Shifted vectors take twice the registers.
    constexpr int G = 2, V = SHIFT ? 1 : 2;
    // Few tokens: a whole block each, so that a row is spread over 256 lanes.
    if (few) return run(k_combine_grad<T, W, SHIFT, G, V, kWarps, 32>, 1);
    return run(k_combine_grad<T, W, SHIFT, G, V, 1, 32>, kWarps);
}

// f(T{}, Int<SHIFT>{}) for the type and alignment at hand.
template <typename F>
rs_status by_type(int type, bool aligned, F f)
{
    switch (type) {
    case RS_FLOAT32: return aligned ? f(float{}, Int<0>{}) : f(float{}, Int<1>{});
    case RS_FLOAT16: return aligned ? f(__half{}, Int<0>{}) : f(__half{}, Int<1>{});
    default:         return aligned ? f(__nv_bfloat16{}, Int<0>{}) : f(__nv_bfloat16{}, Int<1>{});
    }
}

}  // namespace

extern "C" {

rs_status rs_expert_dispatch(rs_float_type type, const void* x, size_t x_stride, const int32_t* position,
                             const int32_t* routed, size_t tokens, int slots, size_t width, void* out,
                             size_t out_stride, void* stream)
{
    const RowArgs a{tokens, width, slots, position, routed, static_cast<cudaStream_t>(stream)};
    const rs_status st = check_rows(a, type);
    if (st != RS_OK || tokens == 0 || width == 0) return st;
    const size_t eb = type_bytes(type);
    if (!valid_rows(x, eb, width, x_stride, true) || !valid_rows(out, eb, width, out_stride, false))
        return RS_ERR_INVALID_ARG;
    const Range r[] = {{out, span_bytes(a.slots_total(), width, out_stride, eb)},
                       {x, span_bytes(tokens, width, x_stride, eb)},
                       {position, (size_t)a.slots_total() * 4},
                       {routed, 4}};
    if (any_alias(r, 1, 4)) return RS_ERR_ALIAS;
    const bool vec = aligned16(x, x_stride, eb) && aligned16(out, out_stride, eb) && width * eb % 16 == 0;
    return by_type(type, vec, [&](auto t, auto n) {
        using T = decltype(t);
        return run_dispatch<T, decltype(n)::value != 0>(a, static_cast<const T*>(x), x_stride, static_cast<T*>(out),
                                                   out_stride);
    });
}

rs_status rs_expert_combine(rs_float_type type, const void* y, size_t y_stride, const void* weights,
                            rs_float_type weight_type, const int32_t* position, const int32_t* routed,
                            size_t tokens, int slots, size_t width, void* out, size_t out_stride, void* stream)
{
    const RowArgs a{tokens, width, slots, position, routed, static_cast<cudaStream_t>(stream)};
    const rs_status st = check_rows(a, type);
    if (st != RS_OK) return st;
    if (weights && ((weight_type != RS_FLOAT32 && weight_type != type) || (uintptr_t)weights % type_bytes(weight_type)))
        return RS_ERR_INVALID_ARG;
    if (tokens == 0 || width == 0) return RS_OK;
    const size_t eb = type_bytes(type);
    if (!valid_rows(y, eb, width, y_stride, true) || !valid_rows(out, eb, width, out_stride, false))
        return RS_ERR_INVALID_ARG;
    const size_t n = a.slots_total();
    const Range r[] = {{out, span_bytes(tokens, width, out_stride, eb)},
                       {y, span_bytes(n, width, y_stride, eb)},
                       {weights, weights ? n * type_bytes(weight_type) : 0},
                       {position, n * 4},
                       {routed, 4}};
    if (any_alias(r, 1, 5)) return RS_ERR_ALIAS;
    const bool vec = aligned16(y, y_stride, eb) && aligned16(out, out_stride, eb) && width * eb % 16 == 0;
    return by_type(type, vec, [&](auto t, auto nn) {
        using T = decltype(t);
        constexpr bool SHIFT = decltype(nn)::value != 0;
        if (!weights || weight_type == RS_FLOAT32)
            return run_combine<T, float, SHIFT>(a, static_cast<const T*>(y), y_stride, static_cast<const float*>(weights),
                                            static_cast<T*>(out), out_stride);
        return run_combine<T, T, SHIFT>(a, static_cast<const T*>(y), y_stride, static_cast<const T*>(weights),
                                    static_cast<T*>(out), out_stride);
    });
}

rs_status rs_expert_combine_grad(rs_float_type type, const void* dout, size_t dout_stride, const void* y,
                                 size_t y_stride, const void* weights, rs_float_type weight_type,
                                 const int32_t* position, const int32_t* routed, size_t tokens, int slots,
                                 size_t width, void* dy, size_t dy_stride, void* dweights, void* stream)
{
    const RowArgs a{tokens, width, slots, position, routed, static_cast<cudaStream_t>(stream)};
    const rs_status st = check_rows(a, type);
    if (st != RS_OK) return st;
    if (weight_type != RS_FLOAT32 && weight_type != type) return RS_ERR_INVALID_ARG;
    if (tokens == 0) return RS_OK;
    const size_t eb = type_bytes(type), wb = type_bytes(weight_type), n = a.slots_total();
    if (!weights || !dweights || (uintptr_t)weights % wb || (uintptr_t)dweights % wb) return RS_ERR_INVALID_ARG;
    if (width == 0)
        return cudaMemsetAsync(dweights, 0, n * wb, a.stream) == cudaSuccess ? RS_OK : RS_ERR_CUDA;
    if (!valid_rows(dout, eb, width, dout_stride, true) || !valid_rows(y, eb, width, y_stride, true) ||
        !valid_rows(dy, eb, width, dy_stride, false))
        return RS_ERR_INVALID_ARG;
    const Range r[] = {{dy, span_bytes(n, width, dy_stride, eb)},
                       {dweights, n * wb},
                       {dout, span_bytes(tokens, width, dout_stride, eb)},
                       {y, span_bytes(n, width, y_stride, eb)},
                       {weights, n * wb},
                       {position, n * 4},
                       {routed, 4}};
    if (any_alias(r, 2, 7)) return RS_ERR_ALIAS;
    const bool vec = aligned16(dout, dout_stride, eb) && aligned16(y, y_stride, eb) &&
                     aligned16(dy, dy_stride, eb) && width * eb % 16 == 0;
    return by_type(type, vec, [&](auto t, auto nn) {
        using T = decltype(t);
        constexpr bool SHIFT = decltype(nn)::value != 0;
        if (weight_type == RS_FLOAT32)
            return run_combine_grad<T, float, SHIFT>(a, static_cast<const T*>(dout), dout_stride,
                                                 static_cast<const T*>(y), y_stride,
                                                 static_cast<const float*>(weights), static_cast<T*>(dy), dy_stride,
                                                 static_cast<float*>(dweights));
        return run_combine_grad<T, T, SHIFT>(a, static_cast<const T*>(dout), dout_stride, static_cast<const T*>(y),
                                         y_stride, static_cast<const T*>(weights), static_cast<T*>(dy), dy_stride,
                                         static_cast<T*>(dweights));
    });
}

}  // extern "C"
