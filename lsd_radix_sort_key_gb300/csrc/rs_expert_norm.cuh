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
// statistics are kept between the two calls.
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

// N adjacent elements as floats and back.
template <typename T, int N>
__device__ __forceinline__ void widen(float (&f)[N], const Vec<T, N>& v)
{
    if constexpr (N == 1) f[0] = to_float(v.v[0]);
    else to_floats<T>(f, v);
}

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> narrow(const float (&f)[N])
{
    if constexpr (N == 1) {
        Vec<T, 1> v;
        v.v[0] = from_float<T>(f[0]);
        return v;
    } else {
        return from_floats<T>(f);
    }
}

// N adjacent parameters, float32 or T.
template <typename T, int N>
__device__ __forceinline__ void load_params(float (&f)[N], const void* p, size_t i, bool wide)
{
    if (sizeof(T) == 4 || wide) {
        const float* from = static_cast<const float*>(p) + i;
        if constexpr (N == 1) {
            f[0] = __ldg(from);
        } else {
#pragma unroll
            for (int c = 0; c < N; c += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(from + c));
                f[c] = v.x, f[c + 1] = v.y, f[c + 2] = v.z, f[c + 3] = v.w;
            }
        }
    } else {
        widen<T, N>(f, load_vec<T, N>(static_cast<const T*>(p) + i));
    }
}

template <typename T, int N>
__device__ __forceinline__ void store_params(void* p, size_t i, const float (&f)[N], bool wide)
{
#pragma unroll
    for (int c = 0; c < N; ++c) {
        if (sizeof(T) == 4 || wide) static_cast<float*>(p)[i + c] = f[c];
        else static_cast<T*>(p)[i + c] = from_float<T>(f[c]);
    }
}

// Arithmetic on a thread's N adjacent elements, two to an instruction: the kernels
// below issue too many to leave all else to memory (a gradient's row of 8 elements per
// thread about 500, 70% of the issue slots).
__device__ __forceinline__ uint64_t pair_of(float a, float b)
{
    return (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b)
{
    a = __uint_as_float((uint32_t)v);
    b = __uint_as_float((uint32_t)(v >> 32));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// d = a b
template <int N>
__device__ __forceinline__ void times(float (&d)[N], const float (&a)[N], const float (&b)[N])
{
    if constexpr (N == 1) d[0] = a[0] * b[0];
    else
#pragma unroll
        for (int c = 0; c < N; c += 2) unpair(mul2(pair_of(a[c], a[c + 1]), pair_of(b[c], b[c + 1])), d[c], d[c + 1]);
}
template <int N>
__device__ __forceinline__ void times(float (&d)[N], const float (&a)[N], float b)
{
    if constexpr (N == 1) d[0] = a[0] * b;
    else
#pragma unroll
        for (int c = 0; c < N; c += 2) unpair(mul2(pair_of(a[c], a[c + 1]), pair_of(b, b)), d[c], d[c + 1]);
}

// d = a b + e
template <int N>
__device__ __forceinline__ void times_plus(float (&d)[N], const float (&a)[N], const float (&b)[N], const float (&e)[N])
{
    if constexpr (N == 1) d[0] = fmaf(a[0], b[0], e[0]);
    else
#pragma unroll
        for (int c = 0; c < N; c += 2)
            unpair(fma2(pair_of(a[c], a[c + 1]), pair_of(b[c], b[c + 1]), pair_of(e[c], e[c + 1])), d[c], d[c + 1]);
}
template <int N>
__device__ __forceinline__ void times_plus(float (&d)[N], const float (&a)[N], float b, const float (&e)[N])
{
    if constexpr (N == 1) d[0] = fmaf(a[0], b, e[0]);
    else
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
        if constexpr (N == 1) v = __float_as_uint(fmaf(a[0], b[0], __uint_as_float((uint32_t)v)));
        else
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

// This thread's columns of the rows that a block walks: STREAMS matrices, V accesses
// of N elements each.  DEPTH > 0: rows are copied to shared memory DEPTH - 1 rows
// ahead, each thread's part by itself and for itself, so no barrier is needed.
// DEPTH 0 (single elements, or rows too wide): one row ahead, in registers.
// With one row ahead the SMs had too few bytes in flight (16384 x 2048 bf16: forward
// 63 us, gradient 182).
template <typename T, int N, int V, int STREAMS, int DEPTH>
struct Feed {
    Vec<T, N> now[DEPTH ? 1 : STREAMS][V], next[DEPTH ? 1 : STREAMS][V];
    unsigned char* ring;  // [DEPTH][STREAMS][V][threads] of 16 bytes, this thread's
    unsigned char* here;  // the slot of the row at hand
    uint32_t slot, pitch;  // pitch: 16 bytes of every thread

    static constexpr size_t smem(size_t threads) { return (size_t)DEPTH * STREAMS * V * threads * 16; }

    __device__ __forceinline__ void* at(uint32_t s, int stream, int i) const
    {
        return ring + ((s * STREAMS + stream) * V + i) * pitch;
    }
    __device__ __forceinline__ void clear(unsigned char* mem)
    {
        pitch = blockDim.x * 16;
        ring = here = mem + threadIdx.x * 16;
        slot = 0;
        if constexpr (DEPTH > 0) {
            for (uint32_t s = 0; s < DEPTH; ++s)
#pragma unroll
                for (int k = 0; k < STREAMS; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) *static_cast<uint4*>(at(s, k, i)) = make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int k = 0; k < STREAMS; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) next[k][i] = Vec<T, N>{};
        }
    }
    // source(k, r): row r of matrix k, or nullptr if there is none (it reads as zero).
    template <typename F>
    __device__ __forceinline__ void fetch(F source, uint32_t r, uint32_t to, uint32_t width)
    {
#pragma unroll
        for (int k = 0; k < STREAMS; ++k) {
            const T* row = source(k, r);
            if (!row) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t c = (i * blockDim.x + threadIdx.x) * N;
                if (c >= width) continue;
                if constexpr (DEPTH > 0) copy16(at(to, k, i), row + c);
                else next[k][i] = load_vec<T, N>(row + c);
            }
        }
    }
    template <typename F>
    __device__ __forceinline__ void start(F source, uint32_t first, uint32_t last, uint32_t width)
    {
        if constexpr (DEPTH > 0) {
#pragma unroll
            for (uint32_t d = 0; d + 1 < DEPTH; ++d) {
                if (first + d < last) fetch(source, first + d, d, width);
                end_group();
            }
        } else {
            fetch(source, first, 0, width);
        }
    }
    // Row r is there afterwards.
    template <typename F>
    __device__ __forceinline__ void turn_to(F source, uint32_t r, uint32_t first, uint32_t last, uint32_t width)
    {
        if constexpr (DEPTH > 0) {
            slot = r == first ? 0 : slot + 1 == DEPTH ? 0 : slot + 1;
            if (r + DEPTH - 1 < last) fetch(source, r + DEPTH - 1, slot == 0 ? DEPTH - 1 : slot - 1, width);
            end_group();
            here = static_cast<unsigned char*>(at(slot, 0, 0));
            wait_groups<DEPTH - 1>();
        } else {
#pragma unroll
            for (int k = 0; k < STREAMS; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) now[k][i] = next[k][i];
            if (r + 1 < last) fetch(source, r + 1, 0, width);
        }
    }
    __device__ __forceinline__ void get(float (&f)[N], int stream, int i) const
    {
        if constexpr (DEPTH > 0) widen<T, N>(f, *reinterpret_cast<const Vec<T, N>*>(here + (stream * V + i) * pitch));
        else widen<T, N>(f, now[stream][i]);
    }
};

// This thread's columns of a row of parameters; `none` where there is none.
template <typename T, int N, int V>
__device__ __forceinline__ void load_columns(float (&f)[V][N], const void* p, size_t at, bool wide, float none, uint32_t width)
{
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
#pragma unroll
        for (int c = 0; c < N; ++c) f[i][c] = none;
        if (p && c0 < width) load_params<T, N>(f[i], p, at + c0, wide);
    }
}

// The gate times the block's weight, this thread's columns.
template <typename T, int N, int V>
__device__ __forceinline__ void load_gate(float (&f)[V][N], const NormArgs<T>& p, uint32_t gate)
{
    load_columns<T, N, V>(f, p.gate_rows ? p.gate : nullptr, (size_t)gate * p.width, p.wide_params, 1.0f, p.width);
    if (!p.block_weight) return;
    float w[V][N];
    load_columns<T, N, V>(w, p.block_weight, 0, p.wide_params, 1.0f, p.width);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int c = 0; c < N; ++c) f[i][c] *= w[i][c];
}

// A block's rows: [first(b), first(b + 1)).
__host__ __device__ inline uint32_t first_row(uint32_t block, uint32_t blocks, uint32_t rows)
{
    return (uint32_t)((uint64_t)block * rows / blocks);
}

// Rows copied ahead by each call.
constexpr int kNormDepth = 4, kGradDepth = 4;
constexpr size_t kNormSmem = 128 * 1024;  // the most that a block's rows take: 512 threads, 4 matrices

// 1 / sqrt(mean + eps); the hardware's root is off by two ulps at most.
__device__ __forceinline__ float inverse_root(float sum, float per_width, float eps) { return rsqrtf(fmaf(sum, per_width, eps)); }

// Each block walks adjacent rows.  The parameters' columns stay in registers (a
// gate's until it changes): reading them again for every row is 24 KB beside a
// row's 16 (2048 bf16, float32 parameters).
template <typename T, int N, int V, int THREADS, bool BLOCK, int DEPTH>
__global__ void __launch_bounds__(THREADS, V == 1 ? 1024 / THREADS : 1) k_norm(NormArgs<T> p)
{
    __shared__ __align__(16) float mem[2 * 3 * 32];
    extern __shared__ __align__(16) unsigned char ring[];
    clear_sums(mem);
    const uint32_t first = first_row(blockIdx.x, gridDim.x, p.rows), last = first_row(blockIdx.x + 1, gridDim.x, p.rows);
    const uint32_t per_gate = p.gate_rows ? p.rows / p.gate_rows : p.rows;
    uint32_t turn = 0, gate = first / per_gate, gate_end = (gate + 1) * per_gate;
    float w[V][N], gw[BLOCK ? V : 1][N];
    Feed<T, N, V, BLOCK ? 2 : 1, DEPTH> feed;
    auto source = [&](int k, uint32_t r) -> const T* { return k == 0 ? p.x + r * p.x_i : p.block + r * p.block_i; };
    feed.clear(ring);
    feed.start(source, first, last, p.width);
    load_columns<T, N, V>(w, p.weight, 0, p.wide_params, 0.0f, p.width);
    if constexpr (BLOCK) load_gate<T, N, V>(gw, p, gate);
    for (uint32_t r = first; r < last; ++r) {
        feed.turn_to(source, r, first, last, p.width);
        Vec<T, N> y[V];  // as it is held
        if constexpr (BLOCK) {
            if (r == gate_end) {
                ++gate;
                gate_end += per_gate;
                load_gate<T, N, V>(gw, p, gate);
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
                const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
                float f[N], u[N];
                feed.get(u, 1, i);
                times(u, u, rb);
                times(u, u, gw[i]);
                feed.get(f, 0, i);
                times_plus(u, f, p.scale, u);
                y[i] = narrow<T, N>(u);
                if (c0 < p.width) store_vec<T, N>(p.y + r * p.y_i + c0, y[i]);
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
            const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
            if (c0 >= p.width) continue;
            float f[N];
            held(f, i);
            times(f, f, rx);
            times(f, f, w[i]);
            store_vec<T, N>(p.h + r * p.h_i + c0, narrow<T, N>(f));
        }
    }
}

// Each block walks adjacent rows as above and keeps its threads' columns of the
// summed gradients in registers.  Within one gate row, with n = block r,
//     dgate = block_weight S,  dblock_weight += gate S,  S = the sum of d n,
// so one sum serves both until the gate changes.
template <typename T, int N, int V, int THREADS, bool BLOCK, int DEPTH>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 3 : 1) k_norm_grad(NormArgs<T> p)
{
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
    Feed<T, N, V, BLOCK ? 4 : 3, DEPTH> feed;
    auto source = [&](int k, uint32_t r) -> const T* {
        switch (k) {
        case kY: return p.dh ? p.x + r * p.x_i : nullptr;
        case kDh: return p.dh ? p.dh + r * p.dh_i : nullptr;
        case kDy: return p.dy ? p.dy + r * p.dy_i : nullptr;
        default: return p.block + r * p.block_i;
        }
    };
    feed.clear(ring);
    feed.start(source, first, last, p.width);
    load_columns<T, N, V>(w, p.weight, 0, p.wide_params, 0.0f, p.width);
    if constexpr (BLOCK) load_gate<T, N, V>(gw, p, gate);
    auto store_part = [&](int kind, int i, const float (&f)[N]) {
        const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
        if (c0 >= p.width) return;
        float* to = p.part + ((size_t)kind * gridDim.x + blockIdx.x) * p.width + c0;
        if constexpr (N == 1) {
            *to = f[0];
        } else {
#pragma unroll
            for (int c = 0; c < N; c += 4) *reinterpret_cast<float4*>(to + c) = make_float4(f[c], f[c + 1], f[c + 2], f[c + 3]);
        }
    };
    for (uint32_t r = first; r < last; ++r) {
        feed.turn_to(source, r, first, last, p.width);
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
        const float kx = rx * rx * rx * p.per_width * sums[1];
        const float rb = BLOCK && p.block_weight ? inverse_root(sums[2], p.per_width, p.eps) : 1.0f;
        Sum2 du_b;
        float du[VB][N];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
            float f[N], g[N], d[N];
            feed.get(f, kY, i);
            feed.get(g, kDh, i);
            feed.get(d, kDy, i);
            times_plus(d, f, -kx, d);
            times(f, f, rx);
            times_plus(dw[i], g, f, dw[i]);
            times(g, g, w[i]);
            times_plus(d, g, rx, d);
            times(g, d, p.scale);
            if (p.dx && c0 < p.width) store_vec<T, N>(p.dx + r * p.dx_i + c0, narrow<T, N>(g));
            if constexpr (BLOCK) {
                feed.get(f, kB, i);
                times(g, f, rb);
                times_plus(sum[i], d, g, sum[i]);
                times(du[i], d, gw[i]);
                du_b.add(du[i], f);
            }
        }
        if constexpr (BLOCK) {
            if (p.dblock) {
                float kb = 0.0f;
                if (p.block_weight) {
                    float dot[1] = {du_b.get()};
                    block_sums(dot, mem, turn);
                    kb = rb * rb * rb * p.per_width * dot[0];
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
                    float f[N];
                    feed.get(f, kB, i);
                    times(f, f, -kb);
                    times_plus(f, du[i], rb, f);
                    if (c0 < p.width) store_vec<T, N>(p.dblock + r * p.dblock_i + c0, narrow<T, N>(f));
                }
            }
            if (r + 1 == last || r + 1 == gate_end) {
                // this block's last row with this gate row: all of its rows, or a part
                const uint32_t begin = gate_end - per_gate;
                const bool whole = begin >= first && gate_end <= last;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
                    if (c0 >= p.width) continue;
                    float f[N];
                    if (p.dblock_weight) {
#pragma unroll
                        for (int c = 0; c < N; ++c) f[c] = 1.0f;
                        if (p.gate_rows) load_params<T, N>(f, p.gate, (size_t)gate * p.width + c0, p.wide_params);
#pragma unroll
                        for (int c = 0; c < N; ++c) db[i][c] = fmaf(f[c], sum[i][c], db[i][c]);
                    }
                    if (p.dgate) {
#pragma unroll
                        for (int c = 0; c < N; ++c) f[c] = 1.0f;
                        if (p.block_weight) load_params<T, N>(f, p.block_weight, c0, p.wide_params);
#pragma unroll
                        for (int c = 0; c < N; ++c) f[c] *= sum[i][c];
                        if (whole) store_params<T, N>(p.dgate, (size_t)gate * p.width + c0, f, p.wide_params);
                        else store_part(begin <= first ? kPartGateFirst : kPartGateLater, i, f);
                    }
#pragma unroll
                    for (int c = 0; c < N; ++c) sum[i][c] = 0.0f;
                }
                if (r + 1 < last) {
                    ++gate;
                    gate_end += per_gate;
                    load_gate<T, N, V>(gw, p, gate);
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
        float sum[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kFinishRows; ++i) sum[0] += mem[i][threadIdx.y * kFinishThreads + threadIdx.x];
        store_params<T, 1>(to, (size_t)gate * p.width + at, sum, p.wide_params);
    }
}

// Launches, instantiated in rs_expert_norm_<type>.cu.  `vectors`: every matrix
// and parameter allows 16-byte accesses.
template <typename T>
rs_status norm_forward(const NormArgs<T>& p, bool vectors, cudaStream_t s);
template <typename T>
rs_status norm_gradient(const NormArgs<T>& p, bool vectors, uint32_t blocks, cudaStream_t s);

// Blocks of a gradient: the sizes alone decide, as the order of its sums goes by
// them.  As many as an SM holds at once, of one thread per 16 bytes of a row (512
// at most): by their registers 768 threads' worth where rows have up to 256
// vectors or are no whole number of vectors, else one block.
inline uint32_t norm_grad_blocks(size_t rows, size_t width, size_t elem)
{
    const size_t threads = align_up(ceil_div(width * elem, 16), 32);
    const bool many = threads <= 256 || (width * elem % 16 && width <= 2048);
    const size_t per = many && threads <= 384 ? 768 / threads : 1, blocks = 152 * (per < 8 ? per : 8);
    return (uint32_t)(rows < blocks ? rows : blocks);
}

}  // namespace rsx
