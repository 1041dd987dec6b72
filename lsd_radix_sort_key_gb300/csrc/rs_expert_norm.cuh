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

// Sums over the threads of a row: blockDim.x of them, 32 or a whole block.
template <int K>
__device__ __forceinline__ void row_sums(float (&s)[K], float* mem)
{
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int d = 16; d; d >>= 1) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], d);
    if (blockDim.x == 32) return;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    __syncthreads();  // (the sums before have been read)
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) mem[k * 32 + warp] = s[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        s[k] = lane < warps ? mem[k * 32 + lane] : 0.0f;
#pragma unroll
        for (int d = 16; d; d >>= 1) s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], d);
    }
}

template <typename T, int N, int V>
struct NormRow {
    Vec<T, N> v[V];
    __device__ __forceinline__ void load(const T* row, uint32_t width)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c = (i * blockDim.x + threadIdx.x) * N;
            v[i] = Vec<T, N>{};
            if (c < width) v[i] = load_vec<T, N>(row + c);
        }
    }
};

// threadIdx.x walks a row, V accesses of N elements per thread; threadIdx.y
// (with 32 threads to a row) takes rows of its own.
template <typename T, int N, int V, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) k_norm(NormArgs<T> p)
{
    __shared__ float mem[32];
    const uint32_t r = blockIdx.x * blockDim.y + threadIdx.y;
    if (r >= p.rows) return;  // (a whole warp, or the block)
    NormRow<T, N, V> x, b;
    x.load(p.x + r * p.x_i, p.width);
    if (p.block) {
        b.load(p.block + r * p.block_i, p.width);
        float rb = 1.0f;
        if (p.block_weight) {
            float s[1] = {};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f[N];
                widen<T, N>(f, b.v[i]);
#pragma unroll
                for (int c = 0; c < N; ++c) s[0] = fmaf(f[c], f[c], s[0]);
            }
            row_sums(s, mem);
            rb = 1.0f / sqrtf(fmaf(s[0], p.per_width, p.eps));
        }
        const size_t gate = p.gate_rows > 1 ? (size_t)(r / (p.rows / p.gate_rows)) * p.width : 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
            if (c0 >= p.width) continue;
            float fx[N], u[N], w[N];
            widen<T, N>(fx, x.v[i]);
            widen<T, N>(u, b.v[i]);
            if (p.block_weight) {
                load_params<T, N>(w, p.block_weight, c0, p.wide_params);
#pragma unroll
                for (int c = 0; c < N; ++c) u[c] *= rb * w[c];
            }
            if (p.gate_rows) {
                load_params<T, N>(w, p.gate, gate + c0, p.wide_params);
#pragma unroll
                for (int c = 0; c < N; ++c) u[c] *= w[c];
            }
#pragma unroll
            for (int c = 0; c < N; ++c) u[c] = fmaf(p.scale, fx[c], u[c]);
            x.v[i] = narrow<T, N>(u);  // y as it is held
            store_vec<T, N>(p.y + r * p.y_i + c0, x.v[i]);
        }
        if (!p.weight) return;
    }
    float s[1] = {};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float f[N];
        widen<T, N>(f, x.v[i]);
#pragma unroll
        for (int c = 0; c < N; ++c) s[0] = fmaf(f[c], f[c], s[0]);
    }
    row_sums(s, mem);
    const float rx = 1.0f / sqrtf(fmaf(s[0], p.per_width, p.eps));
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
        if (c0 >= p.width) continue;
        float f[N], w[N];
        widen<T, N>(f, x.v[i]);
        load_params<T, N>(w, p.weight, c0, p.wide_params);
#pragma unroll
        for (int c = 0; c < N; ++c) f[c] *= rx * w[c];
        store_vec<T, N>(p.h + r * p.h_i + c0, narrow<T, N>(f));
    }
}

// A block's rows: [first(b), first(b + 1)).
__host__ __device__ inline uint32_t first_row(uint32_t block, uint32_t blocks, uint32_t rows)
{
    return (uint32_t)((uint64_t)block * rows / blocks);
}

// Each block walks adjacent rows, the next one's loads in flight while it sums
// over this one, and keeps its threads' columns of the summed gradients in
// registers.
template <typename T, int N, int V, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) k_norm_grad(NormArgs<T> p)
{
    __shared__ float mem[3 * 32];
    start_next_grid();
    const uint32_t first = first_row(blockIdx.x, gridDim.x, p.rows), last = first_row(blockIdx.x + 1, gridDim.x, p.rows);
    const uint32_t per_gate = p.gate_rows ? p.rows / p.gate_rows : p.rows;
    const uint32_t first_gate = first / per_gate;
    float dw[V][N] = {}, db[V][N] = {}, dg[V][N] = {};
    struct {
        NormRow<T, N, V> y, dh, dy, b;
    } next;
    auto fetch = [&](uint32_t r) {
        if (p.dh) {
            next.y.load(p.x + r * p.x_i, p.width);
            next.dh.load(p.dh + r * p.dh_i, p.width);
        }
        if (p.dy) next.dy.load(p.dy + r * p.dy_i, p.width);
        if (p.block) next.b.load(p.block + r * p.block_i, p.width);
    };
    auto store_part = [&](int kind, const float (&f)[V][N]) {
        float* to = p.part + ((size_t)kind * gridDim.x + blockIdx.x) * p.width;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
#pragma unroll
            for (int c = 0; c < N; ++c)
                if (c0 < p.width) to[c0 + c] = f[i][c];
        }
    };
    fetch(first);
    for (uint32_t r = first; r < last; ++r) {
        auto now = next;
        if (r + 1 < last) fetch(r + 1);
        const uint32_t gate = r / per_gate;
        const size_t gate_at = p.gate_rows > 1 ? (size_t)gate * p.width : 0;
        float sums[3] = {};  // y^2, <g, y>, block^2
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
            if (c0 >= p.width) continue;
            float y[N], g[N], w[N];
            if (p.dh) {
                widen<T, N>(y, now.y.v[i]);
                widen<T, N>(g, now.dh.v[i]);
                load_params<T, N>(w, p.weight, c0, p.wide_params);
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    sums[0] = fmaf(y[c], y[c], sums[0]);
                    sums[1] = fmaf(g[c] * w[c], y[c], sums[1]);
                }
            }
            if (p.block_weight) {
                widen<T, N>(y, now.b.v[i]);
#pragma unroll
                for (int c = 0; c < N; ++c) sums[2] = fmaf(y[c], y[c], sums[2]);
            }
        }
        row_sums(sums, mem);
        const float rx = 1.0f / sqrtf(fmaf(sums[0], p.per_width, p.eps)), kx = rx * rx * rx * p.per_width * sums[1];
        const float rb = p.block_weight ? 1.0f / sqrtf(fmaf(sums[2], p.per_width, p.eps)) : 1.0f;
        float dot[1] = {};  // <du, block>
        float du[V][N];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
            if (c0 >= p.width) continue;
            float d[N] = {}, y[N], g[N], w[N];
            if (p.dh) {
                widen<T, N>(y, now.y.v[i]);
                widen<T, N>(g, now.dh.v[i]);
                load_params<T, N>(w, p.weight, c0, p.wide_params);
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    d[c] = fmaf(rx * w[c], g[c], -kx * y[c]);
                    dw[i][c] = fmaf(g[c], y[c] * rx, dw[i][c]);
                }
            }
            if (p.dy) {
                widen<T, N>(g, now.dy.v[i]);
#pragma unroll
                for (int c = 0; c < N; ++c) d[c] += g[c];
            }
            if (p.dx) {
#pragma unroll
                for (int c = 0; c < N; ++c) y[c] = p.scale * d[c];
                store_vec<T, N>(p.dx + r * p.dx_i + c0, narrow<T, N>(y));
            }
            if (!p.block) continue;
            float b[N];
            widen<T, N>(b, now.b.v[i]);
#pragma unroll
            for (int c = 0; c < N; ++c) w[c] = 1.0f;
            if (p.block_weight) load_params<T, N>(w, p.block_weight, c0, p.wide_params);
            if (p.gate_rows) {
                load_params<T, N>(g, p.gate, gate_at + c0, p.wide_params);
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    dg[i][c] = fmaf(d[c], b[c] * rb * w[c], dg[i][c]);
                    d[c] *= g[c];
                }
            }
#pragma unroll
            for (int c = 0; c < N; ++c) {
                if (p.block_weight) db[i][c] = fmaf(d[c], b[c] * rb, db[i][c]);
                du[i][c] = d[c] * w[c];
                dot[0] = fmaf(du[i][c], b[c], dot[0]);
            }
        }
        if (p.dblock) {
            float kb = 0.0f;
            if (p.block_weight) {
                row_sums(dot, mem);
                kb = rb * rb * rb * p.per_width * dot[0];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
                if (c0 >= p.width) continue;
                float b[N];
                widen<T, N>(b, now.b.v[i]);
#pragma unroll
                for (int c = 0; c < N; ++c) b[c] = fmaf(rb, du[i][c], -kb * b[c]);
                store_vec<T, N>(p.dblock + r * p.dblock_i + c0, narrow<T, N>(b));
            }
        }
        if (p.dgate && (r + 1 == last || (r + 1) / per_gate != gate)) {
            // this block's last row with this gate row: whole, or a part of it
            const bool whole = gate * per_gate >= first && (gate + 1) * per_gate <= last;
            if (whole) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t c0 = (i * blockDim.x + threadIdx.x) * N;
                    if (c0 < p.width) store_params<T, N>(p.dgate, gate_at + c0, dg[i], p.wide_params);
                }
            } else {
                store_part(gate == first_gate ? kPartGateFirst : kPartGateLater, dg);
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int c = 0; c < N; ++c) dg[i][c] = 0.0f;
        }
    }
    if (p.dweight) store_part(kPartWeight, dw);
    if (p.dblock_weight) store_part(kPartBlockWeight, db);
}

// The summed gradients from the blocks' parts, in the blocks' order: job 0
// dweight, 1 dblock_weight, 2 + g gate row g (or, with fewer blocks than gate
// rows, the one that block g shares with the next).
constexpr int kFinishCols = 32, kFinishRows = 16;

template <typename T>
__global__ void __launch_bounds__(kFinishCols* kFinishRows) k_norm_finish(NormArgs<T> p, uint32_t blocks, bool by_gate)
{
    __shared__ float mem[kFinishRows][kFinishCols];
    wait_prior_grid();
    const uint32_t job = blockIdx.y, col = blockIdx.x * kFinishCols + threadIdx.x;
    void* to = job == 0 ? p.dweight : job == 1 ? p.dblock_weight : p.dgate;
    if (!to) return;
    uint32_t b0 = 0, b_end = blocks, gate = 0;
    auto block_of = [&](uint32_t row) {  // the block whose rows it is among
        uint32_t b = (uint32_t)(((uint64_t)row * blocks + blocks - 1) / p.rows);
        while (b > 0 && first_row(b, blocks, p.rows) > row) --b;
        while (b + 1 < blocks && first_row(b + 1, blocks, p.rows) <= row) ++b;
        return b;
    };
    const uint32_t per_gate = p.gate_rows ? p.rows / p.gate_rows : p.rows;
    if (job >= 2) {
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
    float s = 0.0f;
    if (col < p.width) {
#pragma unroll 4
        for (uint32_t b = b0 + threadIdx.y; b < b_end; b += kFinishRows) {
            int kind = (int)job;
            if (job >= 2) kind = gate == first_row(b, blocks, p.rows) / per_gate ? kPartGateFirst : kPartGateLater;
            s += p.part[((size_t)kind * blocks + b) * p.width + col];
        }
    }
    mem[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && col < p.width) {
        float sum[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kFinishRows; ++i) sum[0] += mem[i][threadIdx.x];
        store_params<T, 1>(to, (size_t)gate * p.width + col, sum, p.wide_params);
    }
}

// Launches, instantiated in rs_expert_norm_<type>.cu.  `vectors`: every matrix
// and parameter allows 16-byte accesses.
template <typename T>
rs_status norm_forward(const NormArgs<T>& p, bool vectors, cudaStream_t s);
template <typename T>
rs_status norm_gradient(const NormArgs<T>& p, bool vectors, uint32_t blocks, cudaStream_t s);

// Blocks of a gradient: the sizes alone decide, as the order of its sums goes by them.
uint32_t norm_grad_blocks(size_t rows, size_t width, size_t elem);

}  // namespace rsx
