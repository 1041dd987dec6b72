// rs_expert_matmul.cu -- rs_expert_matmul and rs_expert_matmul_grad: the
// experts' products over rows that are laid out by expert.
//
// Three products share one form, D = A B^T summed over the reduction index:
//   forward  D = y [rows, outer],   A = x,    B = w[e],    reduces over inner
//   dx       D = dx [rows, inner],  A = dz,   B = w[e]^T,  reduces over outer
//   dw       D = dw[e] [outer, inner], A = dz^T, B = x^T,  reduces over the expert's rows
// The first two are ragged in D's rows, the third in the reduction.  16-bit
// operands take the tensor cores (rs_expert_tc.cuh), after a copy with aligned
// rows into temp where their rows are not 16-byte aligned or are one row for
// all; float32, and products of nothing, take the multiply-add kernels below.
#include "rs_expert_groups.cuh"
#include "rs_expert_tc.cuh"

// Instantiated in rs_expert_tc_<type>.cu; not here.
namespace rsx {
extern template rs_status tc_ragged_rows<__half>(const TcOperand<__half>&, const TcOperand<__half>&, TcArgs<__half>,
                                                 cudaStream_t);
extern template rs_status tc_ragged_reduce<__half>(const TcOperand<__half>&, const TcOperand<__half>&, TcArgs<__half>,
                                                   cudaStream_t);
extern template rs_status tc_ragged_rows<__nv_bfloat16>(const TcOperand<__nv_bfloat16>&,
                                                        const TcOperand<__nv_bfloat16>&, TcArgs<__nv_bfloat16>,
                                                        cudaStream_t);
extern template rs_status tc_ragged_reduce<__nv_bfloat16>(const TcOperand<__nv_bfloat16>&,
                                                          const TcOperand<__nv_bfloat16>&, TcArgs<__nv_bfloat16>,
                                                          cudaStream_t);
}  // namespace rsx

namespace {

using namespace rsx;

// SMs, for the sizes of tiles below.  Not asked of the device: temp's size and the
// order of dbias's additions go by them, and those are the descriptor's alone.
constexpr size_t kSms = 152;

// -------------------------------------------- products by multiply-adds

// Element (i, k) of A is a[i*a_i + k*a_k]; element (j, k) of B in range e is
// b[e*b_e + j*b_j + k*b_k].
template <typename T>
struct AnyArgs {
    const T* a;
    size_t a_i, a_k;
    const T* b;
    size_t b_e, b_j, b_k;
    T* d;
    size_t d_e, d_i;
    uint32_t cols;       // of D
    uint32_t reduce;     // ragged rows: the reduction's length
    uint32_t out_rows;   // ragged reduction: D's rows
    const int32_t* offsets;
    uint32_t experts, rows;
    const T* bias;
    size_t bias_e;
    const T* residual;
    size_t residual_i;
    T* pre;
    size_t pre_i;
};

constexpr int kAnyThreads = 256;

// One TILE x TILE tile of D per block, float32 multiply-adds.  With TILE = 128 a
// thread has 8 x 8 elements in four 4 x 4 squares 64 apart, so that a step of the
// reduction reads four 16-byte vectors for 64 multiply-adds (32768 x 2048 x 4096
// float32: 36 TFLOP/s, 23 with tiles of 64); the next slab of the reduction is
// fetched into registers meanwhile.  TILE = 64 (4 x 4 per thread, rows 16 apart)
// is for ranges of few rows, where the round trips of the slabs bound it: its
// slabs are four times as deep, and the rows of 16 that a tile does not have
// are not computed.
template <typename T, int ACT, bool RAGGED_K, int TILE>
__global__ void __launch_bounds__(kAnyThreads) k_product_any(AnyArgs<T> p)
{
    constexpr int R = TILE / 16;                      // rows and columns of a thread
    constexpr int kAnyK = TILE == 128 ? 16 : 64;      // depth of a slab
    constexpr int kPer = TILE * kAnyK / kAnyThreads;  // elements of each operand a thread fetches per slab
    constexpr int kPitch = TILE + 4;
    extern __shared__ uint32_t mem[];
    __shared__ __align__(16) float as[kAnyK][kPitch], bs[kAnyK][kPitch];
    const Groups g = Groups::make(mem, p.offsets, p.experts, p.rows, TILE, !RAGGED_K);
    uint32_t e, i0, i_end, k0, k_end;  // rows of D in [i0, i_end), reduction over [k0, k_end)
    if constexpr (RAGGED_K) {
        const uint32_t per = (p.out_rows + TILE - 1) / TILE;
        e = blockIdx.x / per;
        i0 = (blockIdx.x - e * per) * TILE;
        i_end = p.out_rows;
        k0 = g.off[e];
        k_end = g.off[e + 1];
    } else {
        if (blockIdx.x >= g.tiles()) return;
        e = g.find(blockIdx.x);
        i0 = g.off[e] + (blockIdx.x - g.tile[e]) * TILE;
        i_end = g.off[e + 1];
        k0 = 0;
        k_end = e < p.experts ? p.reduce : 0;
    }
    const uint32_t j0 = blockIdx.y * TILE, tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const T* a = p.a;
    const T* b = p.b + (e < p.experts ? e * p.b_e : 0);
    // what this thread fetches: neighbouring threads read neighbouring elements
    const bool a_rows = p.a_k != 1, b_rows = p.b_k != 1;
    auto row_of = [&](bool by_rows, int q) { return by_rows ? (tid + q * kAnyThreads) % TILE : (tid + q * kAnyThreads) / kAnyK; };
    auto k_of = [&](bool by_rows, int q) { return by_rows ? (tid + q * kAnyThreads) / TILE : (tid + q * kAnyThreads) % kAnyK; };
    float fa[kPer], fb[kPer];
    auto fetch = [&](uint32_t k) {
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const uint32_t ai = i0 + row_of(a_rows, q), ak = k + k_of(a_rows, q);
            fa[q] = ai < i_end && ak < k_end ? to_float(a[ai * p.a_i + ak * p.a_k]) : 0.0f;
            const uint32_t bj = j0 + row_of(b_rows, q), bk = k + k_of(b_rows, q);
            fb[q] = bj < p.cols && bk < k_end ? to_float(b[bj * p.b_j + bk * p.b_k]) : 0.0f;
        }
    };
    // row and column of a thread's element r, c
    auto row = [&](int r) { return TILE == 128 ? (r / 4) * 64 + (int)ty * 4 + r % 4 : (int)ty + 16 * r; };
    auto col = [&](int c) { return TILE == 128 ? (c / 4) * 64 + (int)tx * 4 + c % 4 : (int)tx + 16 * c; };
    const int rows = TILE == 128 ? R : (int)min((i_end - i0 + 15) / 16, (uint32_t)R);
    float acc[R][R] = {};
    if (k0 < k_end) fetch(k0);
    for (uint32_t k = k0; k < k_end; k += kAnyK) {
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            as[k_of(a_rows, q)][row_of(a_rows, q)] = fa[q];
            bs[k_of(b_rows, q)][row_of(b_rows, q)] = fb[q];
        }
        __syncthreads();
        if (k + kAnyK < k_end) fetch(k + kAnyK);
#pragma unroll
        for (int kk = 0; kk < kAnyK; ++kk) {
            float av[R], bv[R];
            if constexpr (TILE == 128) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 u = *reinterpret_cast<const float4*>(&as[kk][h * 64 + ty * 4]);
                    const float4 v = *reinterpret_cast<const float4*>(&bs[kk][h * 64 + tx * 4]);
                    av[4 * h] = u.x, av[4 * h + 1] = u.y, av[4 * h + 2] = u.z, av[4 * h + 3] = u.w;
                    bv[4 * h] = v.x, bv[4 * h + 1] = v.y, bv[4 * h + 2] = v.z, bv[4 * h + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    av[q] = as[kk][ty + 16 * q];
                    bv[q] = bs[kk][tx + 16 * q];
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (r < rows) {
#pragma unroll
                    for (int c = 0; c < R; ++c) acc[r][c] = fmaf(av[r], bv[c], acc[r][c]);
                }
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t i = i0 + row(r);
        if (i >= i_end) continue;
#pragma unroll
        for (int c = 0; c < R; ++c) {
            const uint32_t j = j0 + col(c);
            if (j >= p.cols) continue;
            float z = acc[r][c], y = 0.0f;
            if (e < p.experts) {
                if (p.bias) z += to_float(p.bias[e * p.bias_e + j]);
                y = activate<ACT, sizeof(T) == 2>(z);
                if (p.residual) y += to_float(p.residual[i * p.residual_i + j]);
            }
            if (p.pre) p.pre[i * p.pre_i + j] = from_float<T>(z);
            p.d[(RAGGED_K ? e * p.d_e : 0) + i * p.d_i + j] = from_float<T>(y);
        }
    }
}

// Tiles of 128 for ranges of 64 rows or more (on average), if tiles of 64 would
// not fit in two per SM: one of those takes half a tile of 128's time, which
// wins while SMs are idle (64 rows of 1024 x 1024 float32 133 -> 70 us; dw of 2432
// rows and 512 x 1024 292 -> 125) and loses at three per SM (1500 rows, 2 experts
// of 2048 x 1024: 382 us against 268).
bool any_wide(size_t rows, size_t cols, size_t experts)
{
    return rows >= 64 && experts * ceil_div(rows, 64) * ceil_div(cols, 64) > 2 * kSms;
}

template <typename T, int ACT>
rs_status launch_any_rows(const AnyArgs<T>& p, cudaStream_t s)
{
    auto run = [&](auto kernel, size_t tile) {
        const dim3 grid((unsigned)max_tiles(p.rows, p.experts, tile), (unsigned)ceil_div(p.cols, tile));
        kernel<<<grid, kAnyThreads, Groups::words(p.experts) * 4, s>>>(p);
        return cudaGetLastError() == cudaSuccess ? RS_OK : RS_ERR_CUDA;
    };
    if constexpr (sizeof(T) == 4)
        if (any_wide(p.rows / p.experts, p.cols, p.experts) && p.reduce) return run(k_product_any<T, ACT, false, 128>, 128);
    return run(k_product_any<T, ACT, false, 64>, 64);
}

rs_status launch_any_reduce(const AnyArgs<float>& p, cudaStream_t s)
{
    auto run = [&](auto kernel, size_t tile) {
        const dim3 grid((unsigned)(ceil_div(p.out_rows, tile) * p.experts), (unsigned)ceil_div(p.cols, tile));
        kernel<<<grid, kAnyThreads, Groups::words(p.experts) * 4, s>>>(p);
        return cudaGetLastError() == cudaSuccess ? RS_OK : RS_ERR_CUDA;
    };
    if (any_wide(p.out_rows, p.cols, p.experts))
        return run(k_product_any<float, RS_ACT_NONE, true, 128>, 128);
    return run(k_product_any<float, RS_ACT_NONE, true, 64>, 64);
}

// ------------------------------------------------- copies with aligned rows

// `matrices` matrices of `rows` rows of `width` elements, at any strides, to
// rows of `stride` elements (a multiple of 16 bytes, at least width) one after
// the other; one warp per row.  Elements between width and stride may receive
// anything.
template <typename T>
__global__ void __launch_bounds__(256) k_align_rows(const T* __restrict__ from, size_t from_matrix, size_t from_row,
                                                    uint32_t matrices, uint32_t rows, uint32_t width,
                                                    T* __restrict__ to, size_t stride)
{
    const uint64_t n = (uint64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (n >= (uint64_t)matrices * rows) return;
    const uint32_t m = (uint32_t)(n / rows), r = (uint32_t)(n - (uint64_t)m * rows);
    const T* first = from + m * from_matrix;
    const T* last = first + (rows - 1) * from_row + width;
    const T* src = first + r * from_row;
    T* dst = to + n * stride;
    for (uint32_t v = threadIdx.x % 32; v * kVec<T> < width; v += 32) {
        Shifted<T> w;
        w.load(src + v * kVec<T>, first, last);
        store_vec<T, kVec<T>>(dst + v * kVec<T>, w.get(src, (int)(v * kVec<T>), (int)width));
    }
}

// A matrix of 16-bit rows as the tensor-core kernels take it, and where its
// aligned copy goes if it has to be copied.
struct Operand {
    const void* p;
    size_t row_stride, matrix_stride;
    size_t matrices, rows, width;
    bool copy;
    size_t at, bytes;  // in temp

    size_t copy_stride() const { return align_up(width, 8); }
};

Operand operand(const void* p, size_t row_stride, size_t matrix_stride, size_t matrices, size_t rows, size_t width)
{
    Operand o{p, row_stride, matrix_stride, matrix_stride ? matrices : 1, rows, width, false, 0, 0};
    if (rows <= 1) o.row_stride = o.copy_stride();  // a single row's stride is not used
    if (o.matrices <= 1) o.matrix_stride = 0;
    o.copy = (uintptr_t)p % 16 || o.row_stride * 2 % 16 || o.row_stride < width || o.matrix_stride * 2 % 16;
    if (o.copy) o.bytes = align_up(o.matrices * rows * o.copy_stride() * 2, 256);
    return o;
}

// Makes the copy if there is to be one; p and the strides are then the copy's.
template <typename T>
rs_status settle(Operand* o, void* temp, cudaStream_t s)
{
    if (!o->copy) return RS_OK;
    T* to = reinterpret_cast<T*>(static_cast<char*>(temp) + o->at);
    k_align_rows<T><<<(unsigned)ceil_div(o->matrices * o->rows, 8), 256, 0, s>>>(
        static_cast<const T*>(o->p), o->matrix_stride, o->row_stride, (uint32_t)o->matrices, (uint32_t)o->rows,
        (uint32_t)o->width, to, o->copy_stride());
    o->p = to;
    o->row_stride = o->copy_stride();
    o->matrix_stride = o->matrices > 1 ? o->rows * o->copy_stride() : 0;
    return cudaGetLastError() == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

// ------------------------------------------- dz = dy * act'(pre), and dbias

constexpr int kDzThreads = 256, kDzWarps = kDzThreads / 32;

// Vectors of a row that a lane takes: whole rows should pass through memory at
// once, so a block spans DZV * 32 vectors and neighbouring blocks neighbouring
// columns (16384 x 2048 bf16 with dbias: 37.6 us so, 39.4 with one vector and
// neighbouring blocks a row tile apart).
template <int N>
constexpr int kDzVecs = N > 1 ? 2 : 1;

// Rows of a tile: 128, fewer while those would not make kDzBlocks blocks: a
// warp's rows one after the other are what lasts then (gradients of silu in
// bf16, always 128 rows -> so: 3001 rows, 8 experts of 1000 x 1160 55.6 -> 39.4 us,
// 2048, 16 of 1024 x 2048 67.7 -> 49.3, 4096, 8 of 2048 x 2048 87.7 -> 72.7).
// Two per SM; four cost dbias longer sums and gain nothing (16384 x 2048 bf16,
// silu, sums only: 36.9 us with 304, 38.4 with 608, 42.6 with 1216).
constexpr size_t kDzBlocks = 2 * kSms;

size_t dz_tile_rows(size_t rows, size_t cols, size_t elem_bytes)
{
    const size_t across = ceil_div(cols * elem_bytes, 1024);
    size_t tile = 128;
    while (tile > 16 && ceil_div(rows, tile) * across < kDzBlocks) tile /= 2;
    return tile;
}

// One block takes a tile of at most tile_rows rows of one expert and kDzVecs *
// 32 vectors of columns; each warp every eighth row.  part (if given) receives
// the tile's column sums, [row tile][cols], of the values before rounding.  dz
// itself is rounded to T, the type the tensor cores take: that costs dx and dw a
// factor of about sqrt 2 in error (bf16 2.3e-3 against 1.7e-3), and in binary16
// a |dy act'| up to 2^-25 becomes 0 and one of 65520 or more infinite, as in any
// dz that is stored between two calls.
template <typename T, int ACT, int N>
__global__ void __launch_bounds__(kDzThreads) k_act_grad(const T* __restrict__ dy, size_t dy_i,
                                                         const T* __restrict__ pre, size_t pre_i, T* __restrict__ dz,
                                                         size_t dz_i, float* __restrict__ part,
                                                         const int32_t* __restrict__ offsets, uint32_t experts,
                                                         uint32_t rows, uint32_t cols, uint32_t tile_rows)
{
    constexpr int V = kDzVecs<N>, kCols = 32 * V * N;
    extern __shared__ uint32_t mem[];
    __shared__ float sums[kDzWarps][kCols];
    start_next_grid();
    const Groups g = Groups::make(mem, offsets, experts, rows, tile_rows, false);
    const uint32_t across = (cols + kCols - 1) / kCols, tile = blockIdx.x / across;
    if (tile >= g.tiles()) return;
    const uint32_t e = g.find(tile), warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t r0 = g.off[e] + (tile - g.tile[e]) * tile_rows;
    const uint32_t r_end = min(r0 + tile_rows, g.off[e + 1]);
    const uint32_t c0 = (blockIdx.x - tile * across) * kCols + lane * N;
    float sum[V][N] = {};
#pragma unroll 2
    for (uint32_t r = r0 + warp; r < r_end; r += kDzWarps) {
        Vec<T, N> d[V], z[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t c = c0 + v * 32 * N;
            d[v] = z[v] = Vec<T, N>{};
            if (c < cols) {
                d[v] = load_vec<T, N>(dy + r * dy_i + c);
                if constexpr (ACT != RS_ACT_NONE) z[v] = load_vec<T, N>(pre + r * pre_i + c);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t c = c0 + v * 32 * N;
            Vec<T, N> o;
            float g[N], y[N];
            if constexpr (N > 1) {
                to_floats<T>(g, d[v]);
                to_floats<T>(y, z[v]);
            } else {
                g[0] = to_float(d[v].v[0]);
                y[0] = to_float(z[v].v[0]);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                g[i] *= activate_grad<ACT, sizeof(T) == 2>(y[i]);
                sum[v][i] += g[i];
            }
            if constexpr (N > 1) o = from_floats<T>(g);
            else o.v[0] = from_float<T>(g[0]);
            if (dz && c < cols) store_vec<T, N>(dz + r * dz_i + c, o);
        }
    }
    if (!part) return;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) sums[warp][(v * 32 + lane) * N + i] = sum[v][i];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < kCols; i += kDzThreads) {
        const uint32_t col = (blockIdx.x - tile * across) * kCols + i;
        if (col >= cols) break;
        float s = 0.0f;
        for (int w = 0; w < kDzWarps; ++w) s += sums[w][i];
        part[(size_t)tile * cols + col] = s;
    }
}

// dbias[e] = the sum of its row tiles' sums, in order.  Blocks of 128 threads and
// 32 registers fit beside a block of the tensor-core kernels, and with
// wait_first off (k_act_grad is known to have ended) run there unnoticed.
constexpr int kBiasThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kBiasThreads, 16) k_bias_grad(const float* __restrict__ part, T* __restrict__ dbias,
                                                                const int32_t* __restrict__ offsets, uint32_t experts,
                                                                uint32_t rows, uint32_t cols, uint32_t tile_rows,
                                                                bool wait_first)
{
    extern __shared__ uint32_t mem[];
    if (wait_first) wait_prior_grid();
    const Groups g = Groups::make(mem, offsets, experts, rows, tile_rows, false);
    const uint32_t e = blockIdx.x, c = blockIdx.y * kBiasThreads + threadIdx.x;
    if (c < cols) {
        float s = 0.0f;
#pragma unroll 8
        for (uint32_t t = g.tile[e]; t < g.tile[e + 1]; ++t) s += part[(size_t)t * cols + c];
        dbias[(size_t)e * cols + c] = from_float<T>(s);
    }
    wait_prior_grid();
}

// ------------------------------------------------------------- host side

// temp starts with the status words of the tensor-core kernels.
constexpr size_t kStatusBytes = kStatusWords * 4;

Operand rows_operand(const void* p, size_t stride, size_t rows, size_t width)
{
    return operand(p, stride, 0, 1, rows, width);
}

// Which side of an expert's matrix is adjacent in memory: inner or outer.  The
// inner stride of a single column says nothing, so a column whose outer stride
// is not 1 either is rows of one element.  (A single row with an inner stride
// is the same by its outer side.)
bool inner_adjacent(const rs_expert_matmul_desc* d)
{
    return d->w_inner_stride == 1 || (d->inner == 1 && d->w_outer_stride != 1);
}

Operand weights_operand(const rs_expert_matmul_desc* d)
{
    const bool by_inner = inner_adjacent(d);
    return operand(d->w, by_inner ? d->w_outer_stride : d->w_inner_stride, d->w_expert_stride, d->num_experts,
                   by_inner ? d->outer : d->inner, by_inner ? d->inner : d->outer);
}

// What temp holds after the status words; offsets in bytes.
struct Layout {
    size_t dz, dz_stride, part;
    Operand x, w, g;  // g: dy itself, where it is the products' operand
    size_t total;
};

Layout layout(const rs_expert_matmul_desc* d, bool grad)
{
    const size_t eb = type_bytes(d->type);
    const bool dx = grad && d->dx && d->rows && d->inner && d->outer;
    const bool dw = grad && d->dw && d->rows && d->inner && d->outer;
    Layout l{};
    size_t at = kStatusBytes;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align_up(bytes, 256);
        return here;
    };
    if (grad && d->activation != RS_ACT_NONE && (d->dx || d->dw)) {
        l.dz_stride = align_up(d->outer, 16 / eb);
        l.dz = take(d->rows * l.dz_stride * eb);
    }
    if (grad && d->dbias) l.part = take(max_tiles(d->rows, d->num_experts, dz_tile_rows(d->rows, d->outer, eb)) * d->outer * 4);
    if (eb == 2) {
        if (dw || (!grad && d->rows && d->inner && d->outer)) l.x = rows_operand(d->x, d->x_stride, d->rows, d->inner);
        if (dx || (!grad && d->rows && d->inner && d->outer)) l.w = weights_operand(d);
        if ((dx || dw) && d->activation == RS_ACT_NONE) l.g = rows_operand(d->y, d->y_stride, d->rows, d->outer);
        for (Operand* o : {&l.x, &l.w, &l.g})
            if (o->copy) o->at = take(o->bytes);
    }
    l.total = at;
    return l;
}

rs_status check_common(const rs_expert_matmul_desc* d)
{
    if (!d || !valid_type(d->type)) return RS_ERR_INVALID_ARG;
    if (d->activation < RS_ACT_NONE || d->activation > RS_ACT_SILU) return RS_ERR_INVALID_ARG;
    if (d->num_experts < 1 || d->num_experts > RS_EXPERTS_MAX || d->stall_tile < 0) return RS_ERR_INVALID_ARG;
    if (d->rows > RS_EXPERT_SLOTS_MAX || d->inner > RS_EXPERT_WIDTH_MAX || d->outer > RS_EXPERT_WIDTH_MAX)
        return RS_ERR_INVALID_ARG;
    return RS_OK;
}

// The last weight's element offset plus one (below 2^61 bytes by check_weights).
size_t weight_span(const rs_expert_matmul_desc* d)
{
    return (size_t)(d->num_experts - 1) * d->w_expert_stride + (d->outer - 1) * d->w_outer_stride +
           (d->inner - 1) * d->w_inner_stride + 1;
}

rs_status check_weights(const rs_expert_matmul_desc* d)
{
    const size_t eb = type_bytes(d->type);
    if (!d->w || (uintptr_t)d->w % eb) return RS_ERR_INVALID_ARG;
    // strides that are used: below 2^40 bytes, what a tensor map can hold
    auto fits = [&](size_t count, size_t stride) { return count <= 1 || stride < ((size_t)1 << 40) / eb; };
    if (!fits((size_t)d->num_experts, d->w_expert_stride) || !fits(d->outer, d->w_outer_stride) ||
        !fits(d->inner, d->w_inner_stride))
        return RS_ERR_INVALID_ARG;
    if (d->w_inner_stride != 1 && d->w_outer_stride != 1 && d->inner != 1 && d->outer != 1) return RS_ERR_INVALID_ARG;
    return RS_OK;
}

template <typename F>
rs_status by_act(int act, F f)
{
    switch (act) {
    case RS_ACT_NONE: return f(Int<RS_ACT_NONE>{});
    case RS_ACT_RELU: return f(Int<RS_ACT_RELU>{});
    case RS_ACT_GELU: return f(Int<RS_ACT_GELU>{});
    default:          return f(Int<RS_ACT_SILU>{});
    }
}

template <typename T>
TcArgs<T> tc_args(const rs_expert_matmul_desc* d, size_t first_word, size_t words)
{
    TcArgs<T> p{};
    p.offsets = d->offsets;
    p.experts = (uint32_t)d->num_experts;
    p.rows = (uint32_t)d->rows;
    p.status = static_cast<uint32_t*>(d->temp) + first_word;
    p.status_words = (uint32_t)words;
    p.stall = (uint32_t)d->stall_tile;
    return p;
}

// The weights as B of a product whose columns run over outer (forward) or inner (dx).
template <typename T>
TcOperand<T> weight_tc(const rs_expert_matmul_desc* d, const Operand& w, bool cols_are_outer)
{
    return TcOperand<T>{static_cast<const T*>(w.p), w.row_stride, w.matrix_stride, inner_adjacent(d) != cols_are_outer};
}

template <typename T>
AnyArgs<T> any_args(const rs_expert_matmul_desc* d)
{
    AnyArgs<T> p{};
    p.offsets = d->offsets;
    p.experts = (uint32_t)d->num_experts;
    p.rows = (uint32_t)d->rows;
    return p;
}

template <typename T>
rs_status forward(const rs_expert_matmul_desc* d)
{
    cudaStream_t s = static_cast<cudaStream_t>(d->stream);
    if constexpr (sizeof(T) == 2) {
        if (d->inner) {
            Layout l = layout(d, false);
            rs_status st = settle<T>(&l.x, d->temp, s);
            if (st == RS_OK) st = settle<T>(&l.w, d->temp, s);
            if (st != RS_OK) return st;
            TcArgs<T> p = tc_args<T>(d, 0, kStatusWords);
            p.cols = (uint32_t)d->outer;
            p.reduce = (uint32_t)d->inner;
            p.act = d->activation;
            p.d = static_cast<T*>(d->y);
            p.d_i = d->y_stride;
            p.bias = static_cast<const T*>(d->bias);
            p.bias_e = d->bias_stride;
            p.residual = static_cast<const T*>(d->residual);
            p.residual_i = d->residual_stride;
            p.pre = static_cast<T*>(d->pre);
            p.pre_i = d->pre_stride;
            return tc_ragged_rows<T>({static_cast<const T*>(l.x.p), l.x.row_stride, 0, false},
                                     weight_tc<T>(d, l.w, true), p, s);
        }
    }
    if (cudaMemsetAsync(d->temp, 0, kStatusBytes, s) != cudaSuccess) return RS_ERR_CUDA;
    AnyArgs<T> p = any_args<T>(d);
    p.a = static_cast<const T*>(d->x);
    p.a_i = d->x_stride;
    p.a_k = 1;
    p.b = static_cast<const T*>(d->w);
    p.b_e = d->w_expert_stride;
    p.b_j = d->w_outer_stride;
    p.b_k = d->w_inner_stride;
    p.d = static_cast<T*>(d->y);
    p.d_i = d->y_stride;
    p.cols = (uint32_t)d->outer;
    p.reduce = (uint32_t)d->inner;
    p.bias = static_cast<const T*>(d->bias);
    p.bias_e = d->bias_stride;
    p.residual = static_cast<const T*>(d->residual);
    p.residual_i = d->residual_stride;
    p.pre = static_cast<T*>(d->pre);
    p.pre_i = d->pre_stride;
    return by_act(d->activation, [&](auto act) {
        return launch_any_rows<T, decltype(act)::value>(p, s);
    });
}

template <typename T>
rs_status gradient(const rs_expert_matmul_desc* d)
{
    cudaStream_t s = static_cast<cudaStream_t>(d->stream);
    const size_t eb = sizeof(T), groups = Groups::words(d->num_experts) * 4;
    const uint32_t experts = (uint32_t)d->num_experts, rows = (uint32_t)d->rows, cols = (uint32_t)d->outer;
    Layout l = layout(d, true);
    char* temp = static_cast<char*>(d->temp);
    const bool act = d->activation != RS_ACT_NONE;
    const T* dy = static_cast<const T*>(d->y);
    const T* pre = static_cast<const T*>(d->pre);
    T* dz = act && (d->dx || d->dw) ? reinterpret_cast<T*>(temp + l.dz) : nullptr;
    float* part = d->dbias ? reinterpret_cast<float*>(temp + l.part) : nullptr;
    if constexpr (sizeof(T) == 2)
        for (Operand* o : {&l.x, &l.w, &l.g}) {
            const rs_status st = settle<T>(o, temp, s);
            if (st != RS_OK) return st;
        }
    // the products' operand: dz, or dy where there is no activation
    const T* g = act ? dz : sizeof(T) == 2 ? static_cast<const T*>(l.g.p) : dy;
    const size_t g_stride = act ? l.dz_stride : sizeof(T) == 2 ? l.g.row_stride : d->y_stride;
    const uint32_t tile_rows = (uint32_t)dz_tile_rows(rows, cols, eb);
    if ((dz || part) && cols) {
        constexpr int kVec = 16 / sizeof(T);
        const bool vec = aligned16(dy, d->y_stride, eb) && (!act || aligned16(pre, d->pre_stride, eb)) &&
                         d->outer % kVec == 0;
        const rs_status st = by_act(d->activation, [&](auto a) {
            constexpr int ACT = decltype(a)::value;
            const size_t tiles = max_tiles(rows, experts, tile_rows);
            if (vec)
                k_act_grad<T, ACT, kVec><<<(unsigned)(tiles * ceil_div(cols, 32 * kDzVecs<kVec> * kVec)), kDzThreads,
                                           groups, s>>>(dy, d->y_stride, pre, d->pre_stride, dz, l.dz_stride, part,
                                                        d->offsets, experts, rows, cols, tile_rows);
            else
                k_act_grad<T, ACT, 1><<<(unsigned)(tiles * ceil_div(cols, 32)), kDzThreads, groups, s>>>(
                    dy, d->y_stride, pre, d->pre_stride, dz, l.dz_stride, part, d->offsets, experts, rows, cols,
                    tile_rows);
            return cudaGetLastError() == cudaSuccess ? RS_OK : RS_ERR_CUDA;
        });
        if (st != RS_OK) return st;
    }
    // dx and dw share the status words; what takes none of them leaves them clear.
    const bool want_dx = d->dx && rows && d->inner, want_dw = d->dw && d->inner && cols;
    const bool formed = (dz || part) && cols;  // k_act_grad was launched
    bool tc_dx = false, tc_dw = false;
    if constexpr (sizeof(T) == 2) {
        if (want_dx && cols) {
            TcArgs<T> p = tc_args<T>(d, 0, want_dw ? kStatusWords / 2 : kStatusWords);
            p.cols = (uint32_t)d->inner;
            p.reduce = cols;
            p.d = static_cast<T*>(d->dx);
            p.d_i = d->dx_stride;
            p.dependent = p.wait_first = formed;
            const rs_status st = tc_ragged_rows<T>({g, g_stride, 0, false}, weight_tc<T>(d, l.w, false), p, s);
            if (st != RS_OK) return st;
            tc_dx = true;
        }
        if (want_dw && rows) {
            TcArgs<T> p = tc_args<T>(d, want_dx ? kStatusWords / 2 : 0, want_dx ? kStatusWords / 2 : kStatusWords);
            p.cols = (uint32_t)d->inner;
            p.out_rows = cols;
            p.d = static_cast<T*>(d->dw);
            p.d_e = d->outer * d->inner;
            p.d_i = d->inner;
            // beside dx's kernel it need not wait for that one: dz is complete
            // before any block of it starts
            p.dependent = formed || tc_dx;
            p.wait_first = !tc_dx;
            const rs_status st = tc_ragged_reduce<T>(
                {g, g_stride, 0, true}, {static_cast<const T*>(l.x.p), l.x.row_stride, 0, true}, p, s);
            if (st != RS_OK) return st;
            tc_dw = true;
        }
    }
    if (part && cols) {
        const rs_status st = launch_kernel(k_bias_grad<T>, dim3(experts, (unsigned)ceil_div(cols, kBiasThreads)), kBiasThreads,
                                           groups, s, 1, true, (const float*)part, static_cast<T*>(d->dbias), d->offsets,
                                           experts, rows, cols, tile_rows, !tc_dx && !tc_dw);
        if (st != RS_OK) return st;
    }
    if (!tc_dx && (!want_dw || want_dx)) {
        const size_t bytes = want_dx && want_dw ? kStatusBytes / 2 : kStatusBytes;
        if (cudaMemsetAsync(temp, 0, bytes, s) != cudaSuccess) return RS_ERR_CUDA;
    }
    if (!tc_dw && want_dw) {
        const size_t skip = want_dx ? kStatusBytes / 2 : 0;
        if (cudaMemsetAsync(temp + skip, 0, kStatusBytes - skip, s) != cudaSuccess) return RS_ERR_CUDA;
    }
    if (want_dx && !tc_dx) {
        AnyArgs<T> p = any_args<T>(d);
        p.a = g;
        p.a_i = g_stride;
        p.a_k = 1;
        p.b = static_cast<const T*>(d->w);
        p.b_e = d->w_expert_stride;
        p.b_j = d->w_inner_stride;
        p.b_k = d->w_outer_stride;
        p.d = static_cast<T*>(d->dx);
        p.d_i = d->dx_stride;
        p.cols = (uint32_t)d->inner;
        p.reduce = cols;
        const rs_status st = launch_any_rows<T, RS_ACT_NONE>(p, s);
        if (st != RS_OK) return st;
    }
    if (want_dw && !tc_dw) {
        if (rows == 0)
            return cudaMemsetAsync(d->dw, 0, d->outer * d->inner * experts * eb, s) == cudaSuccess ? RS_OK : RS_ERR_CUDA;
        if constexpr (sizeof(T) == 4) {
            AnyArgs<T> p = any_args<T>(d);
            p.a = g;
            p.a_i = 1;
            p.a_k = g_stride;
            p.b = static_cast<const T*>(d->x);
            p.b_j = 1;
            p.b_k = d->x_stride;
            p.d = static_cast<T*>(d->dw);
            p.d_e = d->outer * d->inner;
            p.d_i = d->inner;
            p.cols = (uint32_t)d->inner;
            p.out_rows = cols;
            return launch_any_reduce(p, s);
        }
    }
    return RS_OK;
}

template <typename F>
rs_status by_type(int type, F f)
{
    switch (type) {
    case RS_FLOAT32: return f(float{});
    case RS_FLOAT16: return f(__half{});
    default:         return f(__nv_bfloat16{});
    }
}

}  // namespace

extern "C" {

size_t rs_expert_matmul_temp_bytes(const rs_expert_matmul_desc* d)
{
    return check_common(d) == RS_OK ? layout(d, false).total : (size_t)-1;
}

rs_status rs_expert_matmul(const rs_expert_matmul_desc* d)
{
    rs_status st = check_common(d);
    if (st != RS_OK) return st;
    if (d->rows == 0 || d->outer == 0) return RS_OK;
    const size_t eb = type_bytes(d->type), xw = d->inner, yw = d->outer, n = d->rows;
    if (!d->offsets || (uintptr_t)d->offsets % 4) return RS_ERR_INVALID_ARG;
    if (!valid_rows(d->y, eb, yw, d->y_stride, false)) return RS_ERR_INVALID_ARG;
    if (d->pre && !valid_rows(d->pre, eb, yw, d->pre_stride, false)) return RS_ERR_INVALID_ARG;
    if (d->bias && !valid_rows(d->bias, eb, yw, d->bias_stride, true)) return RS_ERR_INVALID_ARG;
    if (d->residual && !valid_rows(d->residual, eb, yw, d->residual_stride, true)) return RS_ERR_INVALID_ARG;
    if (xw) {
        if (!valid_rows(d->x, eb, xw, d->x_stride, true)) return RS_ERR_INVALID_ARG;
        if ((st = check_weights(d)) != RS_OK) return st;
    }
    const size_t need = layout(d, false).total;
    if (!d->temp || (uintptr_t)d->temp % 256) return RS_ERR_INVALID_ARG;
    if (d->temp_bytes < need) return RS_ERR_TEMP_TOO_SMALL;
    const Range r[] = {{d->y, span_bytes(n, yw, d->y_stride, eb)},
                       {d->pre, d->pre ? span_bytes(n, yw, d->pre_stride, eb) : 0},
                       {d->temp, need},
                       {d->x, span_bytes(n, xw, d->x_stride, eb)},
                       {d->w, xw ? weight_span(d) * eb : 0},
                       {d->bias, d->bias ? span_bytes(d->num_experts, yw, d->bias_stride, eb) : 0},
                       {d->residual, d->residual ? span_bytes(n, yw, d->residual_stride, eb) : 0},
                       {d->offsets, ((size_t)d->num_experts + 1) * 4}};
    if (any_alias(r, 3, 8)) return RS_ERR_ALIAS;
    return by_type(d->type, [&](auto t) { return forward<decltype(t)>(d); });
}

size_t rs_expert_matmul_grad_temp_bytes(const rs_expert_matmul_desc* d)
{
    return check_common(d) == RS_OK ? layout(d, true).total : (size_t)-1;
}

rs_status rs_expert_matmul_grad(const rs_expert_matmul_desc* d)
{
    rs_status st = check_common(d);
    if (st != RS_OK) return st;
    if (!d->dx && !d->dw && !d->dbias) return RS_OK;
    const size_t eb = type_bytes(d->type), xw = d->inner, yw = d->outer, n = d->rows;
    const bool act = d->activation != RS_ACT_NONE;
    if (!d->offsets || (uintptr_t)d->offsets % 4) return RS_ERR_INVALID_ARG;
    if ((uintptr_t)d->dw % eb || (uintptr_t)d->dbias % eb) return RS_ERR_INVALID_ARG;
    if (n && yw) {
        if (!valid_rows(d->y, eb, yw, d->y_stride, true)) return RS_ERR_INVALID_ARG;
        if (act && !valid_rows(d->pre, eb, yw, d->pre_stride, true)) return RS_ERR_INVALID_ARG;
    }
    if (d->dw && n && xw && !valid_rows(d->x, eb, xw, d->x_stride, true)) return RS_ERR_INVALID_ARG;
    if (d->dx && n && xw) {
        if (!valid_rows(d->dx, eb, xw, d->dx_stride, false)) return RS_ERR_INVALID_ARG;
        if (yw && (st = check_weights(d)) != RS_OK) return st;
    }
    const size_t need = layout(d, true).total;
    if (!d->temp || (uintptr_t)d->temp % 256) return RS_ERR_INVALID_ARG;
    if (d->temp_bytes < need) return RS_ERR_TEMP_TOO_SMALL;
    const Range r[] = {{d->dx, d->dx ? span_bytes(n, xw, d->dx_stride, eb) : 0},
                       {d->dw, d->dw ? (size_t)d->num_experts * xw * yw * eb : 0},
                       {d->dbias, d->dbias ? (size_t)d->num_experts * yw * eb : 0},
                       {d->temp, need},
                       {d->y, span_bytes(n, yw, d->y_stride, eb)},
                       {act ? d->pre : nullptr, span_bytes(n, yw, d->pre_stride, eb)},
                       {d->dw ? d->x : nullptr, span_bytes(n, xw, d->x_stride, eb)},
                       {d->dx ? d->w : nullptr, xw && yw ? weight_span(d) * eb : 0},
                       {d->offsets, ((size_t)d->num_experts + 1) * 4}};
    if (any_alias(r, 4, 9)) return RS_ERR_ALIAS;
    return by_type(d->type, [&](auto t) { return gradient<decltype(t)>(d); });
}

rs_status rs_expert_matmul_status(const void* temp, void* stream)
{
    if (!temp) return RS_ERR_INVALID_ARG;
    uint32_t words[kStatusWords];
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(words, temp, sizeof words, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return RS_ERR_CUDA;
    for (uint32_t w : words)
        if (w) return RS_ERR_DEVICE_TIMEOUT;
    return RS_OK;
}

}  // extern "C"
