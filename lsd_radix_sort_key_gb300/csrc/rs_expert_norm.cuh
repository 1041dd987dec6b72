// rs_expert_norm.cuh -- the norms around an expert block and their gradients
// (definitions in rs_expert_block.h).
//
// With r = 1 / sqrt(mean(v^2) + eps) for a row v of width W,
//     rms(v) = v r,
//     the gradient of rms(v) w for v:  r (g - v r^2 <g, v> / W),  g = d w,
//     and for w:                       the sum over rows of d v r.
// Memory bounds both: each row is read once into registers, which hold it
// across the row's sums, and written once.  The gradient forms r again from
// the row that it has to read anyway (its sum goes with <g, v>), so that no
// statistics are kept between the two calls.  Issue slots are the next bound, so
// the arithmetic is in pairs of elements (16384 x 2048 bf16 with everything: forward 50
// us, 5.4 TB/s, 72% of the issue slots; gradient 74 us, 5.4 TB/s).
#pragma once

#include "rs_expert_block.h"
#include "rs_expert_common.cuh"

namespace rsx {

template <typename T>
struct NormArgs {
    uint32_t rows, width;
    float eps, scale, per_width;  // per_width = 1 / width
    bool wide_params;             // weight, block_weight and gate are float32, else T
    uint32_t gate_rows;           // 0: none
    const T* x;
    size_t x_i;
    const T* block;
    size_t block_i;
    const void* weight;
    const void* block_weight;
    const void* gate;
    T* y;
    size_t y_i;
    T* h;
    size_t h_i;
    const T* dh;
    size_t dh_i;
    const T* dy;
    size_t dy_i;
    T* dx;
    size_t dx_i;
    T* dblock;
    size_t dblock_i;
    void* dweight;
    void* dblock_weight;
    void* dgate;
    float* part;  // gradient: [kind][block][width] column sums
};

// The kinds of column sums.  A gate row whose rows several blocks share has a
// sum from each of them: a block's own first gate row or any later one (there
// is at most one later one that it shares).
enum { kPartWeight, kPartBlockWeight, kPartGateFirst, kPartGateLater, kParts };

// How a row is cut: THREADS threads at most, V accesses each of N elements.
// Adjacent elements are one 16-byte vector; STRIDED ones, for rows that are only
// element-aligned, lie as many elements apart as the block has threads, so that
// neighbouring threads have neighbouring elements.  MODE: where rows wait (Feed).
enum { kRegisters, kOwn };
template <int N_, int V_, int THREADS_, int MODE_, bool STRIDED_>
struct NormShape {
    static constexpr int N = N_, V = V_, THREADS = THREADS_, MODE = MODE_;
    static constexpr bool STRIDED = STRIDED_;
    // The column of element c of access i.
    __device__ __forceinline__ static uint32_t col(int i, int c)
    {
        return STRIDED ? (i * N + c) * blockDim.x + threadIdx.x : (i * blockDim.x + threadIdx.x) * N + c;
    }
    // Whether it exists (a vector's elements all do, or none).
    __device__ __forceinline__ static bool has(int i, int c, uint32_t width) { return col(i, STRIDED ? c : 0) < width; }
};

// N elements as floats and back.
template <typename T, int N>
__device__ __forceinline__ void widen(float (&f)[N], const Vec<T, N>& v)
{
    if constexpr (N == kVec<T>) {
        to_floats<T>(f, v);
    } else {
#pragma unroll
        for (int c = 0; c < N; ++c) f[c] = to_float(v.v[c]);
    }
}

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> narrow(const float (&f)[N])
{
    if constexpr (N == kVec<T>) {
        return from_floats<T>(f);
    } else {
        Vec<T, N> v;
#pragma unroll
        for (int c = 0; c < N; ++c) v.v[c] = from_float<T>(f[c]);
        return v;
    }
}

// A thread's elements of access i of a row, zero where there are none.
template <typename S, typename T>
__device__ __forceinline__ Vec<T, S::N> load_elements(const T* row, int i, uint32_t width)
{
    Vec<T, S::N> v{};
    if constexpr (S::STRIDED) {
#pragma unroll
        for (int c = 0; c < S::N; ++c)
            if (S::has(i, c, width)) v.v[c] = row[S::col(i, c)];
    } else {
        if (S::has(i, 0, width)) v = load_vec<T, S::N>(row + S::col(i, 0));
    }
    return v;
}

template <typename S, typename T>
__device__ __forceinline__ void store_elements(T* row, int i, uint32_t width, const Vec<T, S::N>& v)
{
    if constexpr (S::STRIDED) {
#pragma unroll
        for (int c = 0; c < S::N; ++c)
            if (S::has(i, c, width)) row[S::col(i, c)] = v.v[c];
    } else {
        if (S::has(i, 0, width)) store_vec<T, S::N>(row + S::col(i, 0), v);
    }
}

// A thread's elements of access i of a row of parameters, float32 or T.
template <typename S, typename T>
__device__ __forceinline__ void load_params(float (&f)[S::N], const void* p, size_t row, int i, uint32_t width, bool wide)
{
    if (sizeof(T) == 4 || wide) {
        const float* from = static_cast<const float*>(p) + row;
        if constexpr (S::STRIDED) {
#pragma unroll
            for (int c = 0; c < S::N; ++c) f[c] = S::has(i, c, width) ? __ldg(from + S::col(i, c)) : 0.0f;
        } else if (S::has(i, 0, width)) {
#pragma unroll
            for (int c = 0; c < S::N; c += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(from + S::col(i, c)));
                f[c] = v.x, f[c + 1] = v.y, f[c + 2] = v.z, f[c + 3] = v.w;
            }
        }
    } else {
        widen<T, S::N>(f, load_elements<S, T>(static_cast<const T*>(p) + row, i, width));
    }
}

template <typename S, typename T>
__device__ __forceinline__ void store_params(void* p, size_t row, int i, uint32_t width, const float (&f)[S::N], bool wide)
{
#pragma unroll
    for (int c = 0; c < S::N; ++c) {
        if (!S::has(i, c, width)) continue;
        if (sizeof(T) == 4 || wide) static_cast<float*>(p)[row + S::col(i, c)] = f[c];
        else static_cast<T*>(p)[row + S::col(i, c)] = from_float<T>(f[c]);
    }
}

// Arithmetic on a thread's N elements, two to an instruction: the kernels below issue
// too many to leave all else to memory (a gradient's row of 8 elements per thread
// about 500, 70% of the issue slots).

// d = a b
template <int N>
__device__ __forceinline__ void times(float (&d)[N], const float (&a)[N], const float (&b)[N])
{
#pragma unroll
        for (int c = 0; c < N; c += 2) unpair(mul2(pair_of(a[c], a[c + 1]), pair_of(b[c], b[c + 1])), d[c], d[c + 1]);
}
template <int N>
__device__ __forceinline__ void times(float (&d)[N], const float (&a)[N], float b)
{
#pragma unroll
        for (int c = 0; c < N; c += 2) unpair(mul2(pair_of(a[c], a[c + 1]), pair_of(b, b)), d[c], d[c + 1]);
}

// d = a b + e
template <int N>
__device__ __forceinline__ void times_plus(float (&d)[N], const float (&a)[N], const float (&b)[N], const float (&e)[N])
{
#pragma unroll
        for (int c = 0; c < N; c += 2)
            unpair(fma2(pair_of(a[c], a[c + 1]), pair_of(b[c], b[c + 1]), pair_of(e[c], e[c + 1])), d[c], d[c + 1]);
}
template <int N>
__device__ __forceinline__ void times_plus(float (&d)[N], const float (&a)[N], float b, const float (&e)[N])
{
#pragma unroll
        for (int c = 0; c < N; c += 2)
            unpair(fma2(pair_of(a[c], a[c + 1]), pair_of(b, b), pair_of(e[c], e[c + 1])), d[c], d[c + 1]);
}

// s + <a, b>, by even and odd elements
struct Sum2 {
    uint64_t v = 0;
    template <int N>
    __device__ __forceinline__ void add(const float (&a)[N], const float (&b)[N])
    {
#pragma unroll
            for (int c = 0; c < N; c += 2) v = fma2(pair_of(a[c], a[c + 1]), pair_of(b[c], b[c + 1]), v);
    }
    __device__ __forceinline__ float get() const { return __uint_as_float((uint32_t)v) + __uint_as_float((uint32_t)(v >> 32)); }
};

// Sums over a block's threads.  mem: two halves of [K][32] floats, used in turn
// (`turn` counts the calls), so that one barrier per call is enough: a half is
// written again only after the barrier of the call between.
template <int K>
__device__ __forceinline__ void block_sums(float (&s)[K], float* mem, uint32_t& turn)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], d);
    const uint32_t warps = blockDim.x / 32;
    if (warps == 1) return;
    float* half = mem + (turn++ & 1) * (3 * 32);
    if (threadIdx.x % 32 == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) half[k * 32 + threadIdx.x / 32] = s[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = 0.0f;
    for (uint32_t w = 0; w < warps; w += 4) {  // (the ones past the last warp's are zero)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(half + k * 32 + w);
            s[k] += (v.x + v.y) + (v.z + v.w);
        }
    }
}

__device__ __forceinline__ void clear_sums(float* mem)
{
    for (uint32_t i = threadIdx.x; i < 2 * 3 * 32; i += blockDim.x) mem[i] = 0.0f;
    __syncthreads();
}

// Asynchronous copies of 16 bytes to shared memory, waited for in groups.
__device__ __forceinline__ void copy16(void* to, const void* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LATER>  // all but the last LATER groups have arrived
__device__ __forceinline__ void wait_groups() { asm volatile("cp.async.wait_group %0;" ::"n"(LATER) : "memory"); }

// A matrix whose rows a block walks.
template <typename T>
struct Walked {
    const T* p;  // nullptr: none, its rows read as zero
    size_t stride;
};

// The rows of STREAMS matrices, one after the other, as this thread has them.
//   kOwn        vectors: each thread copies its own 16 bytes to shared memory, for
//               itself, three rows ahead, so no barrier is needed
//   kRegisters  rows too wide for that, and strided elements: one row ahead
// With one row ahead in registers the SMs had too few bytes in flight for vectors
// (16384 x 2048 bf16: forward 63 us, gradient 182).  Strided elements are bound by
// their instructions instead: copied to shared memory by the block they took
// longer (8000 x 2047 bf16, gradient without a block 63 us, 48 through registers).
template <typename T, typename S, int STREAMS>
struct Feed {
    static constexpr int N = S::N, V = S::V, MODE = S::MODE;
    static constexpr uint32_t DEPTH = MODE == kOwn ? 4 : 1;
    static constexpr int HELD = MODE == kRegisters ? STREAMS : 1;
    Vec<T, N> now[HELD][V], next[HELD][V];
    unsigned char* ring;   // [DEPTH][STREAMS][pitch], from this thread's part on
    unsigned char* here;   // the slot of the row at hand
    uint32_t slot, pitch;  // pitch: of a row

    static size_t smem(size_t threads) { return MODE == kOwn ? DEPTH * STREAMS * V * threads * 16 : 0; }

    __device__ __forceinline__ void start(const Walked<T> (&m)[STREAMS], unsigned char* mem, uint32_t first, uint32_t last,
                                          uint32_t width)
    {
        pitch = V * blockDim.x * 16;
        ring = here = mem + threadIdx.x * 16;
        slot = 0;
        if constexpr (MODE == kOwn) {
            for (uint32_t k = 0; k < DEPTH * STREAMS; ++k)  // what is not copied reads as zero
#pragma unroll
                for (int i = 0; i < V; ++i)
                    *reinterpret_cast<uint4*>(ring + k * pitch + i * blockDim.x * 16) = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (uint32_t d = 0; d + 1 < DEPTH; ++d) {
                if (first + d < last) fetch(m, first + d, d, width);
                end_group();
            }
        } else {
#pragma unroll
            for (int k = 0; k < STREAMS; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) next[k][i] = Vec<T, N>{};
            fetch(m, first, 0, width);
        }
    }
    __device__ __forceinline__ void fetch(const Walked<T> (&m)[STREAMS], uint32_t r, uint32_t to, uint32_t width)
    {
#pragma unroll
        for (int k = 0; k < STREAMS; ++k) {
            if (!m[k].p) continue;
            const T* row = m[k].p + r * m[k].stride;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if constexpr (MODE == kRegisters) next[k][i] = load_elements<S, T>(row, i, width);
                else if (S::has(i, 0, width)) copy16(ring + (to * STREAMS + k) * pitch + i * blockDim.x * 16, row + S::col(i, 0));
            }
        }
    }
    // Row r is there afterwards.
    __device__ __forceinline__ void turn_to(const Walked<T> (&m)[STREAMS], uint32_t r, uint32_t first, uint32_t last, uint32_t width)
    {
        if constexpr (MODE == kRegisters) {
#pragma unroll
            for (int k = 0; k < STREAMS; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) now[k][i] = next[k][i];
            if (r + 1 < last) fetch(m, r + 1, 0, width);
        } else {
            if (r != first && ++slot == DEPTH) slot = 0;
            if (r + DEPTH - 1 < last) fetch(m, r + DEPTH - 1, slot == 0 ? DEPTH - 1 : slot - 1, width);
            end_group();
            wait_groups<(int)DEPTH - 1>();
            here = ring + slot * STREAMS * pitch;
        }
    }
    __device__ __forceinline__ void get(float (&f)[N], int stream, int i) const
    {
        if constexpr (MODE == kRegisters) widen<T, N>(f, now[stream][i]);
        else widen<T, N>(f, *reinterpret_cast<const Vec<T, N>*>(here + stream * pitch + i * blockDim.x * 16));
    }
};

// This thread's columns of a row of parameters; `none` where there is none.
template <typename S, typename T>
__device__ __forceinline__ void load_columns(float (&f)[S::V][S::N], const void* p, size_t row, bool wide, float none, uint32_t width)
{
#pragma unroll
    for (int i = 0; i < S::V; ++i) {
#pragma unroll
        for (int c = 0; c < S::N; ++c) f[i][c] = none;
        if (p) load_params<S, T>(f[i], p, row, i, width, wide);
    }
}

// The gate times the block's weight, this thread's columns.
template <typename S, typename T>
__device__ __forceinline__ void load_gate(float (&f)[S::V][S::N], const NormArgs<T>& p, uint32_t gate)
{
    load_columns<S, T>(f, p.gate_rows ? p.gate : nullptr, (size_t)gate * p.width, p.wide_params, 1.0f, p.width);
    if (!p.block_weight) return;
    float w[S::V][S::N];
    load_columns<S, T>(w, p.block_weight, 0, p.wide_params, 1.0f, p.width);
#pragma unroll
    for (int i = 0; i < S::V; ++i) times(f[i], f[i], w[i]);
}

// A block's rows: [first(b), first(b + 1)).
__host__ __device__ inline uint32_t first_row(uint32_t block, uint32_t blocks, uint32_t rows)
{
    return (uint32_t)((uint64_t)block * rows / blocks);
}

constexpr size_t kNormSmem = 128 * 1024;  // the most that a block's rows take: 512 threads, 4 matrices

// 1 / sqrt(mean + eps); the hardware's root is off by two ulps at most.  (Rounded
// correctly it costs the gradient of 16384 x 2048 5 us of 73, for errors 4 to 8% smaller.)
__device__ __forceinline__ float inverse_root(float sum, float per_width, float eps) { return rsqrtf(fmaf(sum, per_width, eps)); }

// Each block walks adjacent rows.  The parameters' columns stay in registers (a
// gate's until it changes): reading them again for every row is 24 KB beside a
// row's 16 (2048 bf16, float32 parameters).
template <typename T, typename S, bool BLOCK>
__global__ void __launch_bounds__(S::THREADS, S::V == 1 ? 1024 / S::THREADS : S::THREADS == 128 ? 6 : 1) k_norm(NormArgs<T> p)
{
    constexpr int N = S::N, V = S::V;
    __shared__ __align__(16) float mem[2 * 3 * 32];
    extern __shared__ __align__(16) unsigned char ring[];
    clear_sums(mem);
    const uint32_t first = first_row(blockIdx.x, gridDim.x, p.rows), last = first_row(blockIdx.x + 1, gridDim.x, p.rows);
    const uint32_t per_gate = p.gate_rows ? p.rows / p.gate_rows : p.rows;
    uint32_t turn = 0, gate = first / per_gate, gate_end = (gate + 1) * per_gate;
    float w[V][N], gw[BLOCK ? V : 1][N];
    constexpr int kStreams = BLOCK ? 2 : 1;
    Walked<T> m[kStreams];
    m[0] = {p.x, p.x_i};
    if constexpr (BLOCK) m[1] = {p.block, p.block_i};
    Feed<T, S, kStreams> feed;
    feed.start(m, ring, first, last, p.width);
    load_columns<S, T>(w, p.weight, 0, p.wide_params, 0.0f, p.width);
    if constexpr (BLOCK) load_gate<S, T>(gw, p, gate);
    for (uint32_t r = first; r < last; ++r) {
        feed.turn_to(m, r, first, last, p.width);
        Vec<T, N> y[V];  // as it is held
        if constexpr (BLOCK) {
            if (r == gate_end) {
                ++gate;
                gate_end += per_gate;
                load_gate<S, T>(gw, p, gate);
            }
            float rb = 1.0f;
            if (p.block_weight) {
                Sum2 sum;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float f[N];
                    feed.get(f, 1, i);
                    sum.add(f, f);
                }
                float s[1] = {sum.get()};
                block_sums(s, mem, turn);
                rb = inverse_root(s[0], p.per_width, p.eps);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f[N], u[N];
                feed.get(u, 1, i);
                times(u, u, rb);
                times(u, u, gw[i]);
                feed.get(f, 0, i);
                times_plus(u, f, p.scale, u);
                y[i] = narrow<T, N>(u);
                store_elements<S, T>(p.y + r * p.y_i, i, p.width, y[i]);
            }
            if (!p.weight) continue;
        }
        auto held = [&](float (&f)[N], int i) {
            if constexpr (BLOCK) widen<T, N>(f, y[i]);
            else feed.get(f, 0, i);
        };
        Sum2 sum;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float f[N];
            held(f, i);
            sum.add(f, f);
        }
        float s[1] = {sum.get()};
        block_sums(s, mem, turn);
        const float rx = inverse_root(s[0], p.per_width, p.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float f[N];
            held(f, i);
            times(f, f, rx);
            times(f, f, w[i]);
            store_elements<S, T>(p.h + r * p.h_i, i, p.width, narrow<T, N>(f));
        }
    }
}

// Each block walks adjacent rows as above and keeps its threads' columns of the
// summed gradients in registers.  Within one gate row, with n = block r,
//     dgate = block_weight S,  dblock_weight += gate S,  S = the sum of d n,
// so one sum serves both until the gate changes.  The gradients of a row are
// multiplied out as r (g - (r <g, v> / W) v r): r^3 alone leaves float32's range for
// rows of magnitude 10^13 or 10^-13.
template <typename T, typename S, bool BLOCK>
__global__ void __launch_bounds__(S::THREADS, S::THREADS > 256 ? 1 : S::STRIDED ? 2 : 3) k_norm_grad(NormArgs<T> p)
{
    constexpr int N = S::N, V = S::V;
    __shared__ __align__(16) float mem[2 * 3 * 32];
    extern __shared__ __align__(16) unsigned char ring[];
    start_next_grid();
    clear_sums(mem);
    const uint32_t first = first_row(blockIdx.x, gridDim.x, p.rows), last = first_row(blockIdx.x + 1, gridDim.x, p.rows);
    const uint32_t per_gate = p.gate_rows ? p.rows / p.gate_rows : p.rows;
    uint32_t turn = 0, gate = first / per_gate, gate_end = (gate + 1) * per_gate;
    constexpr int VB = BLOCK ? V : 1;
    enum { kY, kDh, kDy, kB };
    float w[V][N], gw[VB][N], dw[V][N] = {}, db[VB][N] = {}, sum[VB][N] = {};
    constexpr int kStreams = BLOCK ? 4 : 3;
    Walked<T> m[kStreams];
    m[kY] = {p.dh ? p.x : nullptr, p.x_i};
    m[kDh] = {p.dh, p.dh_i};
    m[kDy] = {p.dy, p.dy_i};
    if constexpr (BLOCK) m[kB] = {p.block, p.block_i};
    Feed<T, S, kStreams> feed;
    feed.start(m, ring, first, last, p.width);
    load_columns<S, T>(w, p.weight, 0, p.wide_params, 0.0f, p.width);
    if constexpr (BLOCK) load_gate<S, T>(gw, p, gate);
    auto store_part = [&](int kind, int i, const float (&f)[N]) {
        float* to = p.part + ((size_t)kind * gridDim.x + blockIdx.x) * p.width;
        if constexpr (S::STRIDED) {
#pragma unroll
            for (int c = 0; c < N; ++c)
                if (S::has(i, c, p.width)) to[S::col(i, c)] = f[c];
        } else if (S::has(i, 0, p.width)) {
#pragma unroll
            for (int c = 0; c < N; c += 4)
                *reinterpret_cast<float4*>(to + S::col(i, c)) = make_float4(f[c], f[c + 1], f[c + 2], f[c + 3]);
        }
    };
    for (uint32_t r = first; r < last; ++r) {
        feed.turn_to(m, r, first, last, p.width);
        Sum2 y_y, g_y, b_b;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float f[N], g[N];
            feed.get(f, kY, i);
            feed.get(g, kDh, i);
            times(g, g, w[i]);
            y_y.add(f, f);
            g_y.add(g, f);
            if constexpr (BLOCK) {
                feed.get(f, kB, i);
                b_b.add(f, f);
            }
        }
        float sums[3] = {y_y.get(), g_y.get(), b_b.get()};
        block_sums(sums, mem, turn);
        const float rx = p.dh ? inverse_root(sums[0], p.per_width, p.eps) : 0.0f;
        const float cx = rx * sums[1] * p.per_width;
        const float rb = BLOCK && p.block_weight ? inverse_root(sums[2], p.per_width, p.eps) : 1.0f;
        Sum2 du_b;
        float du[VB][N];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float f[N], g[N], d[N];
            feed.get(f, kY, i);
            feed.get(g, kDh, i);
            feed.get(d, kDy, i);
            times(f, f, rx);
            times_plus(dw[i], g, f, dw[i]);
            times(g, g, w[i]);
            times_plus(g, f, -cx, g);
            times_plus(d, g, rx, d);
            times(g, d, p.scale);
            if (p.dx) store_elements<S, T>(p.dx + r * p.dx_i, i, p.width, narrow<T, N>(g));
            if constexpr (BLOCK) {
                feed.get(f, kB, i);
                times(g, f, rb);
                times_plus(sum[i], d, g, sum[i]);
                times(du[i], d, gw[i]);
                du_b.add(du[i], f);
            }
        }
        if constexpr (BLOCK) {
            // (a block without a weight has no part in its gradient, whatever it holds)
            if (p.dblock && !p.block_weight) {
#pragma unroll
                for (int i = 0; i < V; ++i) store_elements<S, T>(p.dblock + r * p.dblock_i, i, p.width, narrow<T, N>(du[i]));
            } else if (p.dblock) {
                float dot[1] = {du_b.get()};
                block_sums(dot, mem, turn);
                const float cb = rb * dot[0] * p.per_width * rb;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float f[N];
                    feed.get(f, kB, i);
                    times_plus(f, f, -cb, du[i]);
                    times(f, f, rb);
                    store_elements<S, T>(p.dblock + r * p.dblock_i, i, p.width, narrow<T, N>(f));
                }
            }
            if (r + 1 == last || r + 1 == gate_end) {
                // this block's last row with this gate row: all of its rows, or a part
                const uint32_t begin = gate_end - per_gate;
                const bool whole = begin >= first && gate_end <= last;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float f[N];
                    if (p.dblock_weight) {
#pragma unroll
                        for (int c = 0; c < N; ++c) f[c] = 1.0f;
                        if (p.gate_rows) load_params<S, T>(f, p.gate, (size_t)gate * p.width, i, p.width, p.wide_params);
                        times_plus(db[i], f, sum[i], db[i]);
                    }
                    if (p.dgate) {
#pragma unroll
                        for (int c = 0; c < N; ++c) f[c] = 1.0f;
                        if (p.block_weight) load_params<S, T>(f, p.block_weight, 0, i, p.width, p.wide_params);
                        times(f, f, sum[i]);
                        if (whole) store_params<S, T>(p.dgate, (size_t)gate * p.width, i, p.width, f, p.wide_params);
                        else store_part(begin <= first ? kPartGateFirst : kPartGateLater, i, f);
                    }
#pragma unroll
                    for (int c = 0; c < N; ++c) sum[i][c] = 0.0f;
                }
                if (r + 1 < last) {
                    ++gate;
                    gate_end += per_gate;
                    load_gate<S, T>(gw, p, gate);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (p.dweight) store_part(kPartWeight, i, dw[i]);
        if constexpr (BLOCK)
            if (p.dblock_weight) store_part(kPartBlockWeight, i, db[i]);
    }
}

// The summed gradients from the blocks' parts, in the blocks' order: job 0
// dweight, 1 dblock_weight, 2 + g gate row g (or, with fewer blocks than gate
// rows, the one that block g shares with the next).
constexpr int kFinishThreads = 32, kFinishRows = 32;

// C columns to a thread, 4 where rows of parts begin on 16 bytes.
template <typename T, int C>
__global__ void __launch_bounds__(kFinishThreads* kFinishRows) k_norm_finish(NormArgs<T> p, uint32_t blocks, bool by_gate)
{
    __shared__ float mem[kFinishRows][kFinishThreads * C];
    wait_prior_grid();
    const uint32_t job = blockIdx.y, col = (blockIdx.x * kFinishThreads + threadIdx.x) * C;
    void* to = job == 0 ? p.dweight : job == 1 ? p.dblock_weight : p.dgate;
    if (!to) return;
    uint32_t b0 = 0, b_end = blocks, gate = 0;
    if (job >= 2) {
        auto block_of = [&](uint32_t row) {  // the block whose rows it is among
            uint32_t b = (uint32_t)(((uint64_t)row * blocks + blocks - 1) / p.rows);
            while (b > 0 && first_row(b, blocks, p.rows) > row) --b;
            while (b + 1 < blocks && first_row(b + 1, blocks, p.rows) <= row) ++b;
            return b;
        };
        const uint32_t per_gate = p.rows / p.gate_rows;
        if (by_gate) {
            gate = job - 2;
        } else {
            const uint32_t edge = first_row(job - 1, blocks, p.rows);  // of block job - 2 and the next
            gate = edge / per_gate;
            // shared only if it begins before the edge; summed once, at its first edge
            if (gate * per_gate == edge || first_row(job - 2, blocks, p.rows) > gate * per_gate) return;
        }
        b0 = block_of(gate * per_gate);
        b_end = block_of((gate + 1) * per_gate - 1) + 1;
        if (b_end - b0 == 1) return;  // that block has stored it
    }
    // (of the blocks that share a gate row only the first may have begun with another)
    const uint32_t kind = job < 2 ? job : kPartGateFirst;
    const bool later = job >= 2 && first_row(b0, blocks, p.rows) < gate * (p.rows / p.gate_rows);
    float s[C] = {};
    if (col < p.width) {
        const float* from = p.part + (size_t)kind * blocks * p.width + col;
#pragma unroll 8
        for (uint32_t b = b0 + threadIdx.y; b < b_end; b += kFinishRows) {
            const float* at = from + ((size_t)b + (later && b == b0 ? blocks : 0)) * p.width;
            if constexpr (C == 4) {
                const float4 v = *reinterpret_cast<const float4*>(at);
                s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
            } else {
                s[0] += at[0];
            }
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) mem[threadIdx.y][c * kFinishThreads + threadIdx.x] = s[c];
    __syncthreads();
    if (threadIdx.y < C) {  // row y: column y of each thread
        const uint32_t at = (blockIdx.x * kFinishThreads + threadIdx.x) * C + threadIdx.y;
        if (at >= p.width) return;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kFinishRows; ++i) sum += mem[i][threadIdx.y * kFinishThreads + threadIdx.x];
        const size_t i = (size_t)gate * p.width + at;
        if (sizeof(T) == 4 || p.wide_params) static_cast<float*>(to)[i] = sum;
        else static_cast<T*>(to)[i] = from_float<T>(sum);
    }
}

// Launches, instantiated in rs_expert_norm_<type>.cu.  `vectors`: every matrix
// and parameter allows 16-byte accesses.
template <typename T>
rs_status norm_forward(const NormArgs<T>& p, bool vectors, cudaStream_t s);
template <typename T>
rs_status norm_gradient(const NormArgs<T>& p, bool vectors, uint32_t blocks, cudaStream_t s);

// Blocks of a gradient: the sizes and whether there is a block decide, as the
// order of its sums goes by them.  As many as an SM holds at once by their
// registers: 768 threads' worth where a row takes up to 256 (one per 16 bytes),
// about 576 where its elements are strided (four or eight to a thread), else one.
inline uint32_t norm_grad_blocks(size_t rows, size_t width, size_t elem, bool block)
{
    if (width == 0) return 0;
    const bool strided = width * elem % 16 && width <= 2048;
    const size_t threads = align_up(strided ? ceil_div(width, block ? 4 : 8) : ceil_div(width * elem, 16), 32);
    const size_t per = threads > (strided ? 288 : 256) ? 1 : (strided ? 576 : 768) / threads, blocks = kSms * (per < 8 ? per : 8);
    return (uint32_t)(rows < blocks ? rows : blocks);
}

}  // namespace rsx
