// rs_expert_quantize.cu -- rows and weights to 8 bits with a scale for each
// block of 128 (definitions in rs_expert_block.h).
//
// Memory bounds all three: a value is read once (2 or 4 bytes) and written
// once (1 byte, for each of its slots where the rows are dispatched), so a
// block is read, its largest magnitude found and its values rounded without
// leaving the registers.
#include "rs_expert_e4m3.cuh"

namespace {

using namespace rsx;

constexpr int kThreads = 256;
constexpr int kLanes = 8;                  // threads to a block of a row, 16 elements each
constexpr int kUnits = kThreads / kLanes;  // blocks of rows that a thread block takes at a time

// 16 adjacent elements of a row, as loaded: 2 or 4 vectors.
template <typename T, bool SHIFT>
struct Sixteen {
    static constexpr int N = kVec<T>, C = 16 / N, W = 16 * (int)sizeof(T) / 4;
    Vec<T, N> v[C];
    // Rows whose vectors are whole and aligned.
    __device__ __forceinline__ void load(const T* row, uint32_t at, uint32_t width, const T*, const T*)
    {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            v[i] = Vec<T, N>{};
            if (at + i * N < width) v[i] = load_vec<T, N>(row + at + i * N);
        }
    }
    __device__ __forceinline__ void get(uint32_t (&w)[W], const T*, uint32_t, uint32_t) const
    {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const uint4 u = *reinterpret_cast<const uint4*>(&v[i]);
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
    }
};

// Rows that are only element-aligned: from the aligned vectors around them.
template <typename T>
struct Sixteen<T, true> {
    static constexpr int N = kVec<T>, C = 16 / N, W = 16 * (int)sizeof(T) / 4;
    Shifted<T> v[C];
    __device__ __forceinline__ void load(const T* row, uint32_t at, uint32_t, const T* begin, const T* end)
    {
#pragma unroll
        for (int i = 0; i < C; ++i) v[i].load(row + at + i * N, begin, end);
    }
    __device__ __forceinline__ void get(uint32_t (&w)[W], const T* row, uint32_t at, uint32_t width) const
    {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const Vec<T, N> r = v[i].get(row, (int)(at + i * N), (int)width);
            const uint4 u = *reinterpret_cast<const uint4*>(&r);
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
        if (at + 16 <= width) return;
#pragma unroll
        for (int i = 0; i < W; ++i) {  // zeros past the row's end
            constexpr uint32_t per = 4 / sizeof(T);
            if (at + i * per >= width) w[i] = 0;
            else if (per == 2 && at + i * per + 1 >= width) w[i] &= 0xFFFFu;
        }
    }
};

// The largest magnitude over a block's lanes.
__device__ __forceinline__ uint32_t max_of_lanes(uint32_t m)
{
#pragma unroll
    for (int d = kLanes / 2; d; d >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    return m;
}

// A block's 16 elements of this lane, rounded; *byte receives the scale.
template <typename T>
__device__ __forceinline__ uint4 quantize16(uint32_t (&w)[16 * sizeof(T) / 4], uint32_t* byte)
{
    constexpr int W = 16 * sizeof(T) / 4;
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) most = larger<T>(most, w[i]);
    most = max_of_lanes(largest_bits<T>(most));
    // (the warp's other blocks come along)
    if (__any_sync(0xFFFFFFFFu, most >= kNotFinite)) {
        most = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            most = larger_finite<T>(most, w[i]);
            w[i] = without_infinities<T>(w[i]);
        }
        most = max_of_lanes(largest_bits<T>(most));
    }
    *byte = scale_byte(most);
    const float inverse = scale_inverse(*byte);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = quantize4<T>(w + i * (W / 4), inverse);
    return make_uint4(q[0], q[1], q[2], q[3]);
}

template <typename T>
struct RowArgs {
    const T* x;
    size_t x_stride;
    const T* x_end;
    uint32_t width, blocks, units;  // blocks of a row, of all rows
    uint8_t* q;
    size_t q_stride;
    uint8_t* scales;
    size_t scales_stride;
    // dispatch only
    const int32_t* position;
    const int32_t* routed;
    uint32_t slots, slots_total;
};

// Eight lanes take a block of a row: V of them, kUnits apart, whose loads are
// all in flight before the first is used.  DISPATCH: the block is written to
// its token's K rows; the eight lanes hold a token's positions, eight at a
// time, and hand them around by shuffles.
template <typename T, bool SHIFT, bool DISPATCH, int V>
__global__ void __launch_bounds__(kThreads) k_quantize_rows(RowArgs<T> p)
{
    const uint32_t lane = threadIdx.x % kLanes;
    const uint32_t first = blockIdx.x * (uint32_t)(kUnits * V) + threadIdx.x / kLanes;
    Sixteen<T, SHIFT> raw[V];
    uint32_t row[V], at[V], place[DISPATCH ? V : 1];
    uint32_t limit = 0;
    if constexpr (DISPATCH) {
        const int32_t r = __ldg(p.routed);
        limit = r < 0 ? 0u : min((uint32_t)r, p.slots_total);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        // a unit past the end repeats the last one and is not written
        const uint32_t u = min(first + v * kUnits, p.units - 1);
        row[v] = u / p.blocks;
        at[v] = (u - row[v] * p.blocks) * RS_QUANT_BLOCK + lane * 16;
        const T* from = p.x + row[v] * p.x_stride;
        raw[v].load(from, at[v], p.width, p.x, p.x_end);
        if constexpr (DISPATCH) {
            place[v] = 0xFFFFFFFFu;
            if (lane < p.slots) place[v] = (uint32_t)__ldg(p.position + (size_t)row[v] * p.slots + lane);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        uint32_t w[16 * sizeof(T) / 4], byte;
        raw[v].get(w, p.x + row[v] * p.x_stride, at[v], p.width);
        const uint4 q = quantize16<T>(w, &byte);
        const bool live = first + v * kUnits < p.units;
        auto write = [&](uint32_t r, const uint4& values, uint32_t scale) {
            if (at[v] < p.width) *reinterpret_cast<uint4*>(p.q + r * p.q_stride + at[v]) = values;
            if (lane == 0) p.scales[r * p.scales_stride + at[v] / RS_QUANT_BLOCK] = (uint8_t)scale;
        };
        if constexpr (!DISPATCH) {
            if (live) write(row[v], q, byte);
        } else {
            for (uint32_t k0 = 0; k0 < p.slots; k0 += kLanes) {
                if (k0) {
                    place[v] = 0xFFFFFFFFu;
                    if (k0 + lane < p.slots)
                        place[v] = (uint32_t)__ldg(p.position + (size_t)row[v] * p.slots + k0 + lane);
                }
                const uint32_t here = min(p.slots - k0, (uint32_t)kLanes);
                for (uint32_t k = 0; k < here; ++k) {
                    const uint32_t r = __shfl_sync(0xFFFFFFFFu, place[v], k, kLanes);
                    if (!live || r >= p.slots_total) continue;
                    if (r < limit) write(r, q, byte);
                    else write(r, make_uint4(0, 0, 0, 0), kScaleOne);
                }
            }
        }
    }
}

template <typename T, bool DISPATCH>
rs_status launch_rows(const RowArgs<T>& p, bool vectors, cudaStream_t s)
{
    auto run = [&](auto kernel, int v) {
        kernel<<<(unsigned)ceil_div(p.units, (size_t)kUnits * v), kThreads, 0, s>>>(p);
        return cudaGetLastError() == cudaSuccess ? RS_OK : RS_ERR_CUDA;
    };
    constexpr int V = sizeof(T) == 4 ? 2 : 4;
    const bool few = p.units < (size_t)kUnits * V * 4 * kSms;  // would leave SMs without work
    if (vectors)
        return few ? run(k_quantize_rows<T, false, DISPATCH, 1>, 1) : run(k_quantize_rows<T, false, DISPATCH, V>, V);
    return few ? run(k_quantize_rows<T, true, DISPATCH, 1>, 1) : run(k_quantize_rows<T, true, DISPATCH, 2>, 2);
}

// ---------------------------------------------------------------- weights

template <typename T>
struct WeightArgs {
    const T* w;
    size_t w_e, w_n, w_k;
    uint32_t outer, inner, down, across;  // blocks of a matrix
    uint8_t* q;
    size_t q_stride;
    uint8_t* scales;
};

constexpr int kWeightThreads = 512;

// One block of 128 x 128 weights per thread block.  A thread holds 4 x 8 of
// them, as the words they were loaded in until they are rounded: widened at once
// they left room for one block per SM, or went to local memory (114 to 140 us for
// 16 x 4096 x 2048 bf16, 64 so).  K adjacent in memory: 4 rows,
// 32 apart, of 8 adjacent elements, which go out as they came in.  N adjacent
// (BY_N): 8 adjacent rows of n in 4 adjacent k, so that what it holds along k for
// one n is 4 bytes of an output row; these pass through shared memory, whose
// words are permuted by n so that neither side has bank conflicts.  VEC: 16-byte
// loads, else single elements.
template <typename T, bool BY_N, bool VEC>
__global__ void __launch_bounds__(kWeightThreads, sizeof(T) == 4 ? 2 : 3) k_quantize_weights(WeightArgs<T> p)
{
    constexpr int N = kVec<T>, WARPS = kWeightThreads / 32;
    __shared__ uint32_t largest[WARPS];
    __shared__ uint64_t turned[BY_N ? 128 * 16 : 1];
    const uint32_t per = p.down * p.across, e = blockIdx.x / per, b = blockIdx.x - e * per;
    const uint32_t n0 = b / p.across * 128, k0 = (b - b / p.across * p.across) * 128;
    const uint32_t hi = threadIdx.x / 16, lo = threadIdx.x % 16;
    const T* w = p.w + e * p.w_e;
    // the 8 elements of step i: (n, k) of the first
    auto n_of = [&](int i) { return n0 + (BY_N ? lo * 8 : hi + 32 * i); };
    auto k_of = [&](int i) { return k0 + (BY_N ? hi * 4 + i : lo * 8); };
    constexpr int W = 8 * sizeof(T) / 4;  // words of 8 elements
    uint32_t raw[4][W];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 8 / N; ++c) {
            Vec<T, N> v{};
            const uint32_t n = n_of(i) + (BY_N ? c * N : 0), k = k_of(i) + (BY_N ? 0 : c * N);
            if constexpr (VEC) {
                if (n < p.outer && k < p.inner) v = load_vec<T, N>(w + n * p.w_n + k * p.w_k);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const uint32_t nn = n + (BY_N ? j : 0), kk = k + (BY_N ? 0 : j);
                    if (nn < p.outer && kk < p.inner) v.v[j] = w[nn * p.w_n + kk * p.w_k];
                }
            }
            const uint4 u = *reinterpret_cast<const uint4*>(&v);
            raw[i][4 * c] = u.x, raw[i][4 * c + 1] = u.y, raw[i][4 * c + 2] = u.z, raw[i][4 * c + 3] = u.w;
        }
    auto of_block = [&](uint32_t most) {
        most = __reduce_max_sync(0xFFFFFFFFu, largest_bits<T>(most));
        __syncthreads();  // (the values of a round before have been read)
        if (threadIdx.x % 32 == 0) largest[threadIdx.x / 32] = most;
        __syncthreads();
        return __reduce_max_sync(0xFFFFFFFFu, largest[threadIdx.x % WARPS]);
    };
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 4 * W; ++i) most = larger<T>(most, raw[i / W][i % W]);
    most = of_block(most);
    if (most >= kNotFinite) {
        most = 0;
#pragma unroll
        for (int i = 0; i < 4 * W; ++i) {
            most = larger_finite<T>(most, raw[i / W][i % W]);
            raw[i / W][i % W] = without_infinities<T>(raw[i / W][i % W]);
        }
        most = of_block(most);
    }
    const uint32_t byte = scale_byte(most);
    if (threadIdx.x == 0) p.scales[blockIdx.x] = (uint8_t)byte;
    const float s = scale_inverse(byte);
    const uint32_t k_end = (p.inner + 15) / 16 * 16;  // rows are written up to a multiple of 16
    uint8_t* q = p.q + (size_t)e * p.outer * p.q_stride;
    if constexpr (BY_N) {
        uint32_t* words = reinterpret_cast<uint32_t*>(turned);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // the four k of this n
            uint32_t v[sizeof(T)];
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = raw[i][j];
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) v[i] = __byte_perm(raw[2 * i][j / 2], raw[2 * i + 1][j / 2], j % 2 ? 0x7632 : 0x5410);
            }
            words[(lo * 8 + j) * 32 + (hi ^ 2 * lo)] = quantize4<T>(v, s);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t n = hi + 32 * i, k = k0 + lo * 8;
            if (n0 + n < p.outer && k < k_end)
                *reinterpret_cast<uint64_t*>(q + (n0 + n) * p.q_stride + k) = turned[n * 16 + (lo ^ (n / 8))];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = quantize4<T>(raw[i], s), c = quantize4<T>(raw[i] + W / 2, s);
            const uint32_t n = n_of(i), k = k_of(i);
            if (n < p.outer && k < k_end)
                *reinterpret_cast<uint64_t*>(q + n * p.q_stride + k) = (uint64_t)c << 32 | a;
        }
    }
}

// ------------------------------------------------------------- host side

// Quantised rows and their scales, which `rows` rows of `width` values need.
struct Quantized {
    void* q;
    size_t q_stride;
    void* scales;
    size_t scales_stride;

    bool valid(size_t width) const
    {
        return q && (uintptr_t)q % 16 == 0 && q_stride % 16 == 0 && q_stride >= width && q_stride <= (size_t)1 << 32 &&
               scales && scales_stride >= ceil_div(width, RS_QUANT_BLOCK) && scales_stride <= (size_t)1 << 32;
    }
    Range values(size_t rows, size_t width) const { return {q, span_bytes(rows, align_up(width, 16), q_stride, 1)}; }
    Range bytes(size_t rows, size_t width) const
    {
        return {scales, span_bytes(rows, ceil_div(width, RS_QUANT_BLOCK), scales_stride, 1)};
    }
};

template <typename T>
RowArgs<T> row_args(const void* x, size_t x_stride, size_t rows, size_t width, const Quantized& out)
{
    RowArgs<T> p{};
    p.x = static_cast<const T*>(x);
    p.x_stride = x_stride;
    p.x_end = p.x + (rows - 1) * x_stride + width;
    p.width = (uint32_t)width;
    p.blocks = (uint32_t)ceil_div(width, RS_QUANT_BLOCK);
    p.units = (uint32_t)(rows * p.blocks);
    p.q = static_cast<uint8_t*>(out.q);
    p.q_stride = out.q_stride;
    p.scales = static_cast<uint8_t*>(out.scales);
    p.scales_stride = out.scales_stride;
    return p;
}

// Whole 16-byte vectors at 16-byte addresses.
bool by_vectors(const void* x, size_t stride, size_t rows, size_t width, size_t elem)
{
    return aligned16(x, rows > 1 ? stride : 0, elem) && width * elem % 16 == 0;
}

bool too_many(size_t rows, size_t width) { return rows * ceil_div(width, RS_QUANT_BLOCK) > 0xFFFFFFFFu; }

}  // namespace

extern "C" {

rs_status rs_expert_quantize(rs_float_type type, const void* x, size_t x_stride, size_t rows, size_t width, void* q,
                             size_t q_stride, void* scales, size_t scales_stride, void* stream)
{
    if (!valid_type(type) || rows > RS_EXPERT_SLOTS_MAX || width > RS_EXPERT_WIDTH_MAX) return RS_ERR_INVALID_ARG;
    if (rows == 0 || width == 0) return RS_OK;
    const size_t eb = type_bytes(type);
    const Quantized out{q, q_stride, scales, scales_stride};
    if (!valid_rows(x, eb, width, x_stride, true) || !out.valid(width) || too_many(rows, width)) return RS_ERR_INVALID_ARG;
    const Range r[] = {out.values(rows, width), out.bytes(rows, width), {x, span_bytes(rows, width, x_stride, eb)}};
    if (any_alias(r, 2, 3)) return RS_ERR_ALIAS;
    return by_type(type, [&](auto t) {
        using T = decltype(t);
        return launch_rows<T, false>(row_args<T>(x, x_stride, rows, width, out), by_vectors(x, x_stride, rows, width, eb),
                                     static_cast<cudaStream_t>(stream));
    });
}

rs_status rs_expert_dispatch_quantized(rs_float_type type, const void* x, size_t x_stride, const int32_t* position,
                                       const int32_t* routed, size_t tokens, int slots, size_t width, void* q,
                                       size_t q_stride, void* scales, size_t scales_stride, void* stream)
{
    if (!valid_type(type) || slots < 1 || tokens > RS_EXPERT_SLOTS_MAX || tokens * slots > RS_EXPERT_SLOTS_MAX ||
        width > RS_EXPERT_WIDTH_MAX)
        return RS_ERR_INVALID_ARG;
    if (tokens == 0 || width == 0) return RS_OK;
    const size_t eb = type_bytes(type), rows = tokens * slots;
    const Quantized out{q, q_stride, scales, scales_stride};
    if (!valid_rows(x, eb, width, x_stride, true) || !out.valid(width) || too_many(tokens, width)) return RS_ERR_INVALID_ARG;
    if (!position || (uintptr_t)position % 4 || !routed || (uintptr_t)routed % 4) return RS_ERR_INVALID_ARG;
    const Range r[] = {out.values(rows, width), out.bytes(rows, width), {x, span_bytes(tokens, width, x_stride, eb)},
                       {position, rows * 4}, {routed, 4}};
    if (any_alias(r, 2, 5)) return RS_ERR_ALIAS;
    return by_type(type, [&](auto t) {
        using T = decltype(t);
        RowArgs<T> p = row_args<T>(x, x_stride, tokens, width, out);
        p.position = position;
        p.routed = routed;
        p.slots = (uint32_t)slots;
        p.slots_total = (uint32_t)rows;
        return launch_rows<T, true>(p, by_vectors(x, x_stride, tokens, width, eb), static_cast<cudaStream_t>(stream));
    });
}

rs_status rs_expert_quantize_weights(rs_float_type type, const void* w, size_t w_expert_stride, size_t w_outer_stride,
                                     size_t w_inner_stride, int num_experts, size_t outer, size_t inner, void* q,
                                     size_t q_stride, void* scales, void* stream)
{
    if (!valid_type(type) || num_experts < 1 || num_experts > RS_EXPERTS_MAX || outer > RS_EXPERT_WIDTH_MAX ||
        inner > RS_EXPERT_WIDTH_MAX)
        return RS_ERR_INVALID_ARG;
    if (outer == 0 || inner == 0) return RS_OK;
    const size_t eb = type_bytes(type), experts = (size_t)num_experts;
    const size_t down = ceil_div(outer, RS_QUANT_BLOCK), across = ceil_div(inner, RS_QUANT_BLOCK);
    if (!w || (uintptr_t)w % eb || down * across * experts > 0x7FFFFFFFu) return RS_ERR_INVALID_ARG;
    // strides of a single expert, row or column are not used; the others are
    // below 2^40 bytes, as the products' are
    size_t se = experts > 1 ? w_expert_stride : 0, sn = outer > 1 ? w_outer_stride : 0, sk = inner > 1 ? w_inner_stride : 0;
    const size_t most = ((size_t)1 << 40) / eb;
    if (se >= most || sn >= most || sk >= most) return RS_ERR_INVALID_ARG;
    if (outer > 1 && inner > 1 && sn != 1 && sk != 1) return RS_ERR_INVALID_ARG;
    const Quantized out{q, q_stride, scales, across};
    if (!out.valid(inner)) return RS_ERR_INVALID_ARG;
    const size_t span = (experts - 1) * se + (outer - 1) * sn + (inner - 1) * sk + 1;
    const Range r[] = {out.values(experts * outer, inner), {scales, experts * down * across}, {w, span * eb}};
    if (any_alias(r, 2, 3)) return RS_ERR_ALIAS;
    const bool by_n = inner > 1 && sk != 1;
    const bool vec = (uintptr_t)w % 16 == 0 && se * eb % 16 == 0 &&
                     (by_n ? sn == 1 && sk * eb % 16 == 0 && outer * eb % 16 == 0
                           : sk == 1 && sn * eb % 16 == 0 && inner * eb % 16 == 0);
    return by_type(type, [&](auto t) {
        using T = decltype(t);
        WeightArgs<T> p{static_cast<const T*>(w), se, sn, sk, (uint32_t)outer, (uint32_t)inner, (uint32_t)down,
                        (uint32_t)across, static_cast<uint8_t*>(q), q_stride, static_cast<uint8_t*>(scales)};
        const unsigned grid = (unsigned)(down * across * experts);
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        if (by_n && vec) k_quantize_weights<T, true, true><<<grid, kWeightThreads, 0, s>>>(p);
        else if (by_n) k_quantize_weights<T, true, false><<<grid, kWeightThreads, 0, s>>>(p);
        else if (vec) k_quantize_weights<T, false, true><<<grid, kWeightThreads, 0, s>>>(p);
        else k_quantize_weights<T, false, false><<<grid, kWeightThreads, 0, s>>>(p);
        return cudaGetLastError() == cudaSuccess ? RS_OK : RS_ERR_CUDA;
    });
}

}  // extern "C"
