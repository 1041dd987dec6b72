// rs_expert_rows.cu -- the row movers of the expert operators: dispatch,
// combine and combine's gradient (formulas in rs_experts.h).
//
// All three go token by token: a token's own row is read (or written) once
// and its K expert rows, which lie anywhere, are each written or read once,
// whole and in order.  So the bytes moved are the least possible,
//   dispatch      (1 + K) rows per token
//   combine       (1 + K)
//   combine grad  (1 + 2K)
// with no use of `order`, and the sum over a token's slots is a loop in one
// thread, in slot order: no atomics, the same result every time.
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

// One warp moves a piece of kPiece vectors per lane of one token's row to its
// K places.
template <typename T, int N, int PIECE>
__global__ void __launch_bounds__(kThreads) k_dispatch(const T* __restrict__ x, size_t x_stride,
                                                       const int32_t* __restrict__ position,
                                                       const int32_t* __restrict__ routed, uint32_t slots_total,
                                                       uint32_t tokens, uint32_t slots, uint32_t vecs,
                                                       uint32_t pieces, T* __restrict__ out, size_t out_stride)
{
    const uint32_t item = blockIdx.x * kWarps + threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t t = item / pieces;
    if (t >= tokens) return;
    const uint32_t v0 = (item - t * pieces) * (32 * PIECE) + lane;
    const uint32_t limit = routed_rows(routed, slots_total);
    Vec<T, N> r[PIECE];
#pragma unroll
    for (int i = 0; i < PIECE; ++i)
        if (v0 + i * 32 < vecs) r[i] = load_vec<T, N>(x + t * x_stride + (size_t)(v0 + i * 32) * N);
    for (uint32_t k = 0; k < slots; ++k) {
        const uint32_t p = (uint32_t)__ldg(position + (size_t)t * slots + k);
        if (p >= slots_total) continue;
        T* to = out + p * out_stride;
        const Vec<T, N> zero{};
#pragma unroll
        for (int i = 0; i < PIECE; ++i)
            if (v0 + i * 32 < vecs) store_vec<T, N>(to + (size_t)(v0 + i * 32) * N, p < limit ? r[i] : zero);
    }
}

// One warp sums a piece of V vectors per lane over a token's slots, G slots at
// a time: G * V row loads per lane are in flight before the first is used.
// The positions and weights of up to 32 slots are one load each, a slot per
// lane, and handed around by shuffles.
template <typename T, typename W, int N, int G, int V>
__global__ void __launch_bounds__(kThreads) k_combine(const T* __restrict__ y, size_t y_stride,
                                                      const W* __restrict__ weights,
                                                      const int32_t* __restrict__ position,
                                                      const int32_t* __restrict__ routed, uint32_t slots_total,
                                                      uint32_t tokens, uint32_t slots, uint32_t vecs,
                                                      uint32_t pieces, T* __restrict__ out, size_t out_stride)
{
    const uint32_t item = blockIdx.x * kWarps + threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t t = item / pieces;
    if (t >= tokens) return;
    const uint32_t v0 = (item - t * pieces) * (32 * V) + lane;
    const uint32_t limit = routed_rows(routed, slots_total);
    float acc[V][N] = {};
    for (uint32_t k0 = 0; k0 < slots; k0 += 32) {
        const uint32_t here = min(slots - k0, 32u);
        uint32_t my_row = 0xFFFFFFFFu;
        float my_weight = 1.0f;
        if (lane < here) {
            const size_t s = (size_t)t * slots + k0 + lane;
            my_row = (uint32_t)__ldg(position + s);
            if (weights) my_weight = to_float(weights[s]);
        }
        for (uint32_t k = 0; k < here; k += G) {
            Vec<T, N> r[G][V];
            bool kept[G];
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const uint32_t p = __shfl_sync(0xFFFFFFFFu, my_row, (k + j) & 31);
                kept[j] = k + j < here && p < limit;
                if (kept[j]) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (v0 + i * 32 < vecs)
                            r[j][i] = load_vec<T, N>(y + p * y_stride + (size_t)(v0 + i * 32) * N);
                }
            }
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const float w = __shfl_sync(0xFFFFFFFFu, my_weight, (k + j) & 31);
                if (kept[j]) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
#pragma unroll
                        for (int c = 0; c < N; ++c) acc[i][c] = fmaf(w, to_float(r[j][i].v[c]), acc[i][c]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (v0 + i * 32 < vecs) {
            Vec<T, N> o;
#pragma unroll
            for (int c = 0; c < N; ++c) o.v[c] = from_float<T>(acc[i][c]);
            store_vec<T, N>(out + t * out_stride + (size_t)(v0 + i * 32) * N, o);
        }
}

// A group of WT warps takes one token: every lane walks its share of the row,
// for up to kSlots slots at a time, and the lanes' parts of the dot products
// are summed at the end (within the warp by shuffles, over the warps through
// shared memory), always in the same order.
template <typename T, typename W, int N, int WT>
__global__ void __launch_bounds__(kThreads) k_combine_grad(
    const T* __restrict__ dout, size_t dout_stride, const T* __restrict__ y, size_t y_stride,
    const W* __restrict__ weights, const int32_t* __restrict__ position, const int32_t* __restrict__ routed,
    uint32_t slots_total, uint32_t tokens, uint32_t slots, uint32_t vecs, T* __restrict__ dy, size_t dy_stride,
    W* __restrict__ dweights)
{
    constexpr int kSlots = 8;
    __shared__ float part[kWarps][kSlots];
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t t = blockIdx.x * (kWarps / WT) + warp / WT;
    const bool live = t < tokens;  // no early return: the block has barriers when WT > 1
    const uint32_t limit = routed_rows(routed, slots_total);
    for (uint32_t k0 = 0; k0 < slots; k0 += kSlots) {
        uint32_t p[kSlots];
        float w[kSlots], dot[kSlots] = {};
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            p[j] = 0xFFFFFFFFu;
            w[j] = 0.0f;
            if (live && k0 + j < slots) {
                const size_t s = (size_t)t * slots + k0 + j;
                p[j] = (uint32_t)__ldg(position + s);
                if (p[j] < limit) w[j] = to_float(weights[s]);
            }
        }
        for (uint32_t v = (warp % WT) * 32 + lane; live && v < vecs; v += 32 * WT) {
            const Vec<T, N> d = load_vec<T, N>(dout + t * dout_stride + (size_t)v * N);
            Vec<T, N> r[kSlots];
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (p[j] < limit) r[j] = load_vec<T, N>(y + p[j] * y_stride + (size_t)v * N);
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
                if (p[j] >= slots_total) continue;
                Vec<T, N> o{};
                if (p[j] < limit) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float g = to_float(d.v[i]);
                        dot[j] = fmaf(g, to_float(r[j].v[i]), dot[j]);
                        o.v[i] = from_float<T>(w[j] * g);
                    }
                }
                store_vec<T, N>(dy + p[j] * dy_stride + (size_t)v * N, o);
            }
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
            for (int d = 16; d; d >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
        if constexpr (WT > 1) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (lane == 0) part[warp][j] = dot[j];
            __syncthreads();
            if (warp % WT == 0 && lane < kSlots) {
                float sum = 0.0f;
                for (int i = 0; i < WT; ++i) sum += part[warp + i][lane];
                if (live && k0 + lane < slots) dweights[(size_t)t * slots + k0 + lane] = from_float<W>(sum);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (lane == 0 && live && k0 + j < slots)
                    dweights[(size_t)t * slots + k0 + j] = from_float<W>(dot[j]);
        }
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

template <typename T, int N>
rs_status run_dispatch(const RowArgs& a, const T* x, size_t x_stride, T* out, size_t out_stride)
{
    constexpr int kPiece = 4;
    const uint32_t vecs = (uint32_t)(a.width / N), pieces = (uint32_t)ceil_div(vecs, 32 * kPiece);
    const size_t step = tokens_per_launch(pieces);
    for (size_t t = 0; t < a.tokens; t += step) {
        const uint32_t here = (uint32_t)(a.tokens - t < step ? a.tokens - t : step);
        k_dispatch<T, N, kPiece><<<(unsigned)ceil_div((size_t)here * pieces, kWarps), kThreads, 0, a.stream>>>(
            x + t * x_stride, x_stride, a.position + t * a.slots, a.routed, a.slots_total(), here, a.slots, vecs,
            pieces, out, out_stride);
    }
    return launched();
}

template <typename T, typename W, int N, int G, int V>
rs_status launch_combine(const RowArgs& a, const T* y, size_t y_stride, const W* weights, T* out, size_t out_stride)
{
    const uint32_t vecs = (uint32_t)(a.width / N), pieces = (uint32_t)ceil_div(vecs, 32 * V);
    const size_t step = tokens_per_launch(pieces);
    for (size_t t = 0; t < a.tokens; t += step) {
        const uint32_t here = (uint32_t)(a.tokens - t < step ? a.tokens - t : step);
        k_combine<T, W, N, G, V><<<(unsigned)ceil_div((size_t)here * pieces, kWarps), kThreads, 0, a.stream>>>(
            y, y_stride, weights ? weights + t * a.slots : nullptr, a.position + t * a.slots, a.routed,
            a.slots_total(), here, a.slots, vecs, pieces, out + t * out_stride, out_stride);
    }
    return launched();
}

template <typename T, typename W, int N>
rs_status run_combine(const RowArgs& a, const T* y, size_t y_stride, const W* weights, T* out, size_t out_stride)
{
    // eight loads in flight per lane, whatever the number of slots
    if (a.slots > 4) return launch_combine<T, W, N, 8, 1>(a, y, y_stride, weights, out, out_stride);
    if (a.slots > 2) return launch_combine<T, W, N, 4, 2>(a, y, y_stride, weights, out, out_stride);
    return launch_combine<T, W, N, 2, 4>(a, y, y_stride, weights, out, out_stride);
}

template <typename T, typename W, int N>
rs_status run_combine_grad(const RowArgs& a, const T* dout, size_t dout_stride, const T* y, size_t y_stride,
                           const W* weights, T* dy, size_t dy_stride, W* dweights)
{
    const uint32_t vecs = (uint32_t)(a.width / N);
    // Few tokens: a whole block each, so that a row is spread over 256 lanes.
    if (a.tokens < 1024)
        k_combine_grad<T, W, N, kWarps><<<(unsigned)a.tokens, kThreads, 0, a.stream>>>(
            dout, dout_stride, y, y_stride, weights, a.position, a.routed, a.slots_total(), (uint32_t)a.tokens,
            a.slots, vecs, dy, dy_stride, dweights);
    else
        k_combine_grad<T, W, N, 1><<<(unsigned)ceil_div(a.tokens, kWarps), kThreads, 0, a.stream>>>(
            dout, dout_stride, y, y_stride, weights, a.position, a.routed, a.slots_total(), (uint32_t)a.tokens,
            a.slots, vecs, dy, dy_stride, dweights);
    return launched();
}

// f(T{}, Int<N>{}) for the type and alignment at hand.
template <typename F>
rs_status by_type(int type, bool vec, F f)
{
    switch (type) {
    case RS_FLOAT32: return vec ? f(float{}, Int<4>{}) : f(float{}, Int<1>{});
    case RS_FLOAT16: return vec ? f(__half{}, Int<8>{}) : f(__half{}, Int<1>{});
    default:         return vec ? f(__nv_bfloat16{}, Int<8>{}) : f(__nv_bfloat16{}, Int<1>{});
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
        return run_dispatch<T, decltype(n)::value>(a, static_cast<const T*>(x), x_stride, static_cast<T*>(out),
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
        constexpr int N = decltype(nn)::value;
        if (!weights || weight_type == RS_FLOAT32)
            return run_combine<T, float, N>(a, static_cast<const T*>(y), y_stride, static_cast<const float*>(weights),
                                            static_cast<T*>(out), out_stride);
        return run_combine<T, T, N>(a, static_cast<const T*>(y), y_stride, static_cast<const T*>(weights),
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
        constexpr int N = decltype(nn)::value;
        if (weight_type == RS_FLOAT32)
            return run_combine_grad<T, float, N>(a, static_cast<const T*>(dout), dout_stride,
                                                 static_cast<const T*>(y), y_stride,
                                                 static_cast<const float*>(weights), static_cast<T*>(dy), dy_stride,
                                                 static_cast<float*>(dweights));
        return run_combine_grad<T, T, N>(a, static_cast<const T*>(dout), dout_stride, static_cast<const T*>(y),
                                         y_stride, static_cast<const T*>(weights), static_cast<T*>(dy), dy_stride,
                                         static_cast<T*>(dweights));
    });
}

}  // extern "C"
