// rs_expert_tc.cuh -- the experts' products on the tensor cores: 16-bit
// operands whose rows are 16-byte aligned.
//
// D = A B^T, a 128 x BN tile of D per step of a persistent block.  Warp 0's
// first lane copies 64-deep slices of A and B into a ring of shared-memory
// stages (TMA, 128-byte swizzle); warp 1's first lane feeds them to
// tcgen05.mma, which accumulates in float32 in tensor memory; warps 4-11 read
// finished accumulators, apply the epilogue and store, while the next tile
// accumulates in the other half of tensor memory.
//   Ragged rows (forward, dx): a tile starts at its expert's rows and may run
//     past them; the surplus rows of D are computed and not stored.
//   Ragged reduction (dw): the reduction runs over an expert's rows; the last
//     slice's rows past the expert's end, which belong to the next expert, are
//     overwritten with zeros in shared memory before they are used.
// Either operand may have its reduction index or its row index adjacent in
// memory (K-major / MN-major): both copy with rows of 128 bytes and both feed
// the instruction directly, so nothing is transposed.
#pragma once

#include "rs_expert_groups.cuh"
#include "rs_tc.cuh"

namespace rsx {

constexpr int kTcRows = 128;    // tile rows
constexpr int kTcDepth = 64;    // reduction elements per stage: one swizzled row of 128 bytes
constexpr int kTcThreads = 384;
constexpr int kTcFirstEpilogueWarp = 4, kTcEpilogueWarps = 8;
constexpr int kTcMaxBlocks = 256;
constexpr uint32_t kStatusWords = 2 * kTcMaxBlocks;  // at the start of temp

template <typename T>
struct TcArgs {
    const int32_t* offsets;
    uint32_t experts, rows;
    uint32_t cols;      // of D
    uint32_t reduce;    // ragged rows: the reduction's length
    uint32_t out_rows;  // ragged reduction: D's rows
    int act;            // rs_activation
    uint32_t b_expert;  // ragged rows: 1, or 0 if every expert has the same B
    T* d;
    size_t d_e, d_i;
    const T* bias;
    size_t bias_e;
    const T* residual;
    size_t residual_i;
    T* pre;
    size_t pre_i;
    uint32_t* status;  // one word per block: 0, or 1 if a wait ran out; the rest of the area is cleared
    uint32_t status_words;
    uint32_t stall;    // testing hook: tile stall - 1 is never copied
};

template <int BN>
struct TcShape {
    static constexpr uint32_t kA = kTcRows * kTcDepth * 2, kB = BN * kTcDepth * 2, kStage = kA + kB;
    static constexpr int kStages = BN == 256 ? 4 : 6;
    static constexpr uint32_t kStaging = 32 * 64;  // bytes per epilogue warp: 32 rows of 32 elements
    static constexpr size_t smem(size_t experts)
    {
        return 1024 + (size_t)kStages * kStage + kTcEpilogueWarps * kStaging + (2 * kStages + 4) * 8 + 16 +
               Groups::words(experts) * 4;
    }
};

// Where a tile is: rows [i0, i_end) and columns from j0 of D, expert e, and
// the reduction [k0, k_end).
struct TcTile {
    uint32_t e, i0, i_end, j0, k0, k_end;
};

template <int BN, bool RAGGED_K, typename T>
__device__ __forceinline__ TcTile tc_tile(const TcArgs<T>& p, const Groups& g, uint32_t tile)
{
    const uint32_t across = (p.cols + BN - 1) / BN;
    const uint32_t down = tile / across;
    TcTile t;
    t.j0 = (tile - down * across) * BN;
    if constexpr (RAGGED_K) {
        const uint32_t per = (p.out_rows + kTcRows - 1) / kTcRows;
        t.e = down / per;
        t.i0 = (down - t.e * per) * kTcRows;
        t.i_end = p.out_rows;
        t.k0 = g.off[t.e];
        t.k_end = g.off[t.e + 1];
    } else {
        t.e = g.find(down);
        t.i0 = g.off[t.e] + (down - g.tile[t.e]) * kTcRows;
        t.i_end = g.off[t.e + 1];
        t.k0 = 0;
        t.k_end = t.e < p.experts ? p.reduce : 0;
    }
    return t;
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u)
{
    if constexpr (__is_same(T, __half)) return __half22float2(*reinterpret_cast<const __half2*>(&u));
    else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}

// One warp's 32 x 32 piece of D goes through shared memory, so that the lane
// that holds a row in tensor memory need not store it: `mine` is this lane's
// row as 4 vectors of 8 elements, and memory sees 4 lanes per row.  The
// vectors are permuted by the row so that neither side has bank conflicts.
__device__ __forceinline__ uint32_t stage_slot(uint32_t row, uint32_t vec) { return row * 4 + (vec ^ ((row >> 1) & 3)); }

template <typename T>
__device__ __forceinline__ void store_piece(uint4* stage, const uint32_t (&mine)[16], T* d, size_t d_i, uint32_t i0,
                                            uint32_t i_end, uint32_t j0, uint32_t cols, bool vec)
{
    const uint32_t lane = threadIdx.x % 32;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        stage[stage_slot(lane, q)] = make_uint4(mine[4 * q], mine[4 * q + 1], mine[4 * q + 2], mine[4 * q + 3]);
    __syncwarp();
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const uint32_t row = n * 8 + lane / 4, q = lane % 4, i = i0 + row, j = j0 + q * 8;
        if (i < i_end && j < cols) {
            const uint4 v = stage[stage_slot(row, q)];
            T* to = d + i * d_i + j;
            if (vec && j + 8 <= cols) *reinterpret_cast<uint4*>(to) = v;
            else {
                const T* s = reinterpret_cast<const T*>(&v);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (j + c < cols) to[c] = s[c];
            }
        }
    }
    __syncwarp();
}

// The reverse: this lane's row of a 32 x 32 piece (zeros outside).
template <typename T>
__device__ __forceinline__ void load_piece(uint4* stage, uint32_t (&mine)[16], const T* d, size_t d_i, uint32_t i0,
                                           uint32_t i_end, uint32_t j0, uint32_t cols, bool vec)
{
    const uint32_t lane = threadIdx.x % 32;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const uint32_t row = n * 8 + lane / 4, q = lane % 4, i = i0 + row, j = j0 + q * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (i < i_end && j < cols) {
            const T* from = d + i * d_i + j;
            if (vec && j + 8 <= cols) v = __ldg(reinterpret_cast<const uint4*>(from));
            else {
                T* s = reinterpret_cast<T*>(&v);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (j + c < cols) s[c] = from[c];
            }
        }
        stage[stage_slot(row, q)] = v;
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 v = stage[stage_slot(lane, q)];
        mine[4 * q] = v.x;
        mine[4 * q + 1] = v.y;
        mine[4 * q + 2] = v.z;
        mine[4 * q + 3] = v.w;
    }
    __syncwarp();
}

template <typename T>
__device__ __forceinline__ bool rows_aligned(const T* p, size_t stride)
{
    return ((uintptr_t)p | (stride * sizeof(T))) % 16 == 0;
}

// out = act(z) + residual, rounded.
template <typename T, int ACT>
__device__ __forceinline__ void finish(uint32_t (&out)[16], const uint32_t (&z)[32], const uint32_t (&res)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 r = unpack2<T>(res[i]);
        out[i] = pack2<T>(activate<ACT, true>(__uint_as_float(z[2 * i])) + r.x,
                          activate<ACT, true>(__uint_as_float(z[2 * i + 1])) + r.y);
    }
}

// A_MN / B_MN: the operand's row index, not its reduction index, is adjacent
// in memory.  Ragged rows: A is K-major rows of map_a (2-d), B is per expert
// (map_b 3-d).  Ragged reduction: both are MN-major columns of 2-d maps.
template <typename T, int BN, bool RAGGED_K, bool B_MN>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_product_tc(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, TcArgs<T> p)
{
    using namespace rstc;
    using S = TcShape<BN>;
    constexpr bool A_MN = RAGGED_K;
    static_assert(!RAGGED_K || B_MN, "both operands of a ragged reduction are MN-major");
    extern __shared__ unsigned char raw[];
    unsigned char* ring = raw + (1024 - smem_addr(raw) % 1024) % 1024;  // stages are 1024-byte aligned
    unsigned char* staging = ring + S::kStages * S::kStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + kTcEpilogueWarps * S::kStaging);
    uint64_t* empty = full + S::kStages;
    uint64_t* acc_full = empty + S::kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    uint32_t* failed = slot + 1;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 32) {
        tma_prefetch(&map_a);
        tma_prefetch(&map_b);
        for (int s = 0; s < S::kStages; ++s) {
            bar_init(full + s, 1);
            bar_init(empty + s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(acc_full + s, 1);
            bar_init(acc_empty + s, kTcEpilogueWarps);
        }
        bar_init_fence();
        *failed = 0;
    }
    if (warp == 2) tmem_alloc(slot, 512);
    tc_fence_before();
    // (the barrier inside make() orders all of the above)
    const Groups g = Groups::make(slot + 4, p.offsets, p.experts, p.rows, kTcRows, !RAGGED_K);
    tc_fence_after();
    const uint32_t tmem = *slot;
    const uint32_t across = (p.cols + BN - 1) / BN;
    const uint32_t tiles = (RAGGED_K ? (p.out_rows + kTcRows - 1) / kTcRows * p.experts : g.tiles()) * across;

    uint32_t issued = 0;  // stages filled so far (the copying thread)
    if (warp == 0 && lane == 0) {
        bool ok = true;
        for (uint32_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
            const TcTile t = tc_tile<BN, RAGGED_K>(p, g, tile);
            if (tile + 1 == p.stall) break;
            for (uint32_t k = t.k0; k < t.k_end; k += kTcDepth, ++issued) {
                const uint32_t s = issued % S::kStages, round = issued / S::kStages;
                if (!bar_wait(empty + s, (round & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                unsigned char* a = ring + s * S::kStage;
                unsigned char* b = a + S::kA;
                bar_expect(full + s, S::kStage);
                if constexpr (RAGGED_K) {
#pragma unroll
                    for (int i = 0; i < kTcRows / 64; ++i)
                        tma_load_2d(a + i * 8192, &map_a, (int)(t.i0 + i * 64), (int)k, full + s);
#pragma unroll
                    for (int i = 0; i < BN / 64; ++i)
                        tma_load_2d(b + i * 8192, &map_b, (int)(t.j0 + i * 64), (int)k, full + s);
                } else {
                    const int e = (int)(t.e * p.b_expert);
                    tma_load_2d(a, &map_a, (int)k, (int)t.i0, full + s);
                    if constexpr (B_MN) {
#pragma unroll
                        for (int i = 0; i < BN / 64; ++i)
                            tma_load_3d(b + i * 8192, &map_b, (int)(t.j0 + i * 64), (int)k, e, full + s);
                    } else {
                        tma_load_3d(b, &map_b, (int)k, (int)t.j0, e, full + s);
                    }
                }
            }
        }
        if (!ok) *failed = 1;
    } else if (warp == 1) {
        constexpr uint32_t kDesc = mma_desc(!__is_same(T, __half), A_MN, B_MN, kTcRows, BN);
        constexpr uint32_t kAStep = A_MN ? 2048 : 32, kBStep = B_MN ? 2048 : 32;
        uint32_t used = 0, n = 0;
        bool ok = true;
        for (uint32_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
            const TcTile t = tc_tile<BN, RAGGED_K>(p, g, tile);
            if (t.k0 >= t.k_end) continue;
            const uint32_t h = n & 1, acc = tmem + h * 256;
            ok = bar_wait_warp(acc_empty + h, ((n >> 1) & 1) ^ 1);
            if (!ok) break;
            tc_fence_after();
            ++n;
            for (uint32_t k = t.k0; k < t.k_end; k += kTcDepth, ++used) {
                const uint32_t s = used % S::kStages;
                ok = bar_wait_warp(full + s, (used / S::kStages) & 1);
                if (!ok) break;
                unsigned char* a = ring + s * S::kStage;
                uint32_t steps = kTcDepth / 16;
                if constexpr (RAGGED_K) {
                    const uint32_t left = t.k_end - k;
                    if (left < kTcDepth) {  // rows [left, 16 * steps) are another expert's
                        steps = (left + 15) / 16;
                        const uint32_t vecs = (steps * 16 - left) * 8;  // 16-byte vectors per box of 64 columns
                        for (uint32_t v = lane; v < vecs; v += 32)
#pragma unroll
                            for (int i = 0; i < (kTcRows + BN) / 64; ++i)
                                reinterpret_cast<uint4*>(a + i * 8192 + left * 128)[v] = make_uint4(0, 0, 0, 0);
                        fence_async_smem();
                        __syncwarp();
                    }
                }
                if (lane == 0) {
                    tc_fence_after();
                    const uint32_t sa = smem_addr(a);
                    const uint64_t da = smem_desc(sa, A_MN ? 8192 : 16), db = smem_desc(sa + S::kA, B_MN ? 8192 : 16);
                    for (uint32_t i = 0; i < steps; ++i)
                        mma_f16(acc, da + i * (kAStep >> 4), db + i * (kBStep >> 4), kDesc, k > t.k0 || i > 0);
                    mma_commit(empty + s);
                }
                __syncwarp();
            }
            if (lane == 0) mma_commit(acc_full + h);
        }
        if (!ok) *failed = 1;
    } else if (warp >= kTcFirstEpilogueWarp) {
        const uint32_t w = warp - kTcFirstEpilogueWarp;
        const uint32_t quarter = warp % 4;            // the 32 tensor-memory lanes this warp can read
        const uint32_t c0 = (w / 4) * (BN / 2);       // and its half of the columns
        uint4* stage = reinterpret_cast<uint4*>(staging + w * S::kStaging);
        const bool vec_d = rows_aligned(p.d, p.d_i | (RAGGED_K ? p.d_e : 0)), vec_pre = rows_aligned(p.pre, p.pre_i);
        const bool vec_res = rows_aligned(p.residual, p.residual_i), vec_bias = rows_aligned(p.bias, p.bias_e);
        uint32_t n = 0;
        for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const TcTile t = tc_tile<BN, RAGGED_K>(p, g, tile);
            const bool some = t.k0 < t.k_end;
            const uint32_t h = n & 1;
            if (some) {
                if (!bar_wait_warp(acc_full + h, (n >> 1) & 1)) {
                    *failed = 1;
                    break;
                }
                tc_fence_after();
                ++n;
            }
            const uint32_t i0 = t.i0 + quarter * 32;
            T* d = p.d + (RAGGED_K ? t.e * p.d_e : 0);
            for (uint32_t c = c0; c < c0 + BN / 2; c += 32) {
                const uint32_t j = t.j0 + c;
                if (j >= p.cols) break;
                uint32_t z[32], out[16] = {};
                if (some) {
                    tmem_load32(z, tmem + h * 256 + c + (quarter << 21));  // lane 32 * quarter in the high half
                    tmem_load_wait();
                    if (p.bias) {
                        const T* bias = p.bias + t.e * p.bias_e + j;
                        if (vec_bias && j + 32 <= p.cols) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const uint4 b = __ldg(reinterpret_cast<const uint4*>(bias) + q);
                                const uint32_t u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float2 f = unpack2<T>(u[i]);
                                    z[8 * q + 2 * i] = __float_as_uint(__uint_as_float(z[8 * q + 2 * i]) + f.x);
                                    z[8 * q + 2 * i + 1] = __float_as_uint(__uint_as_float(z[8 * q + 2 * i + 1]) + f.y);
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (j + i < p.cols)
                                    z[i] = __float_as_uint(__uint_as_float(z[i]) + to_float(bias[i]));
                        }
                    }
                    if (p.pre) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            out[i] = pack2<T>(__uint_as_float(z[2 * i]), __uint_as_float(z[2 * i + 1]));
                        store_piece<T>(stage, out, p.pre, p.pre_i, i0, t.i_end, j, p.cols, vec_pre);
                    }
                    uint32_t res[16] = {};
                    if (p.residual)
                        load_piece<T>(stage, res, p.residual, p.residual_i, i0, t.i_end, j, p.cols, vec_res);
                    switch (p.act) {
                    case RS_ACT_NONE: finish<T, RS_ACT_NONE>(out, z, res); break;
                    case RS_ACT_RELU: finish<T, RS_ACT_RELU>(out, z, res); break;
                    case RS_ACT_GELU: finish<T, RS_ACT_GELU>(out, z, res); break;
                    default: finish<T, RS_ACT_SILU>(out, z, res); break;
                    }
                } else if (p.pre) {
                    store_piece<T>(stage, out, p.pre, p.pre_i, i0, t.i_end, j, p.cols, vec_pre);
                }
                store_piece<T>(stage, out, d, p.d_i, i0, t.i_end, j, p.cols, vec_d);
            }
            if (some) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(acc_empty + h);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0) {
        if (*failed)  // a copy must not land in shared memory that this block no longer owns
            for (uint32_t s = 0; s < S::kStages && s < issued; ++s) {
                const uint32_t last = (issued - 1 - s) / S::kStages;
                bar_wait(full + s, last & 1);
            }
        p.status[blockIdx.x] = *failed;
    }
    if (blockIdx.x == 0)
        for (uint32_t i = gridDim.x + threadIdx.x; i < p.status_words; i += kTcThreads) p.status[i] = 0;
    __syncthreads();
    if (warp == 2) tmem_free(tmem, 512);
}

// Launches one product; RS_ERR_UNSUPPORTED if the operands cannot be copied
// this way (alignment, strides), so that the caller takes the general kernel.
// Instantiated in rs_expert_tc_<type>.cu.
template <typename T>
struct TcOperand {
    const T* p;
    size_t row_stride;     // elements between rows of the adjacent dimension
    size_t expert_stride;  // B of a ragged-rows product; 0: shared by all
    bool mn;               // the row index is adjacent, not the reduction
};
template <typename T>
rs_status tc_ragged_rows(const TcOperand<T>& a, const TcOperand<T>& b, TcArgs<T> args, cudaStream_t stream);
template <typename T>
rs_status tc_ragged_reduce(const TcOperand<T>& a, const TcOperand<T>& b, TcArgs<T> args, cudaStream_t stream);

}  // namespace rsx
