// rs_expert_tc.cuh -- the experts' products on the tensor cores: 16-bit
// operands whose rows are 16-byte aligned.
//
// D = A B^T, one tile of D per step of a persistent block (BN columns, 128
// rows) or pair of blocks (PAIR: 256 rows, a cluster of two on neighbouring
// SMs).  Warp 0's first lane copies 64-deep slices of A and B into a ring of
// shared-memory stages (TMA, 128-byte swizzle); warp 1's first lane feeds them
// to tcgen05.mma, which accumulates in float32 in tensor memory; 16 epilogue
// warps read finished accumulators, apply the epilogue and store, while the
// next tile accumulates in the other half of tensor memory.
//   Ragged rows (forward, dx): a tile starts at its expert's rows and may run
//     past them; the surplus rows of D are computed and not stored.
//   Ragged reduction (dw): the reduction runs over an expert's rows; the last
//     slice's rows past the expert's end, which belong to the next expert, are
//     overwritten with zeros in shared memory by warp 3 before the slice is
//     handed on (the copy reports to warp 3, and warp 3 to the multiplying
//     warp).
// Either operand may have its reduction index or its row index adjacent in
// memory (K-major / MN-major): both copy with rows of 128 bytes and both feed
// the instruction directly, so nothing is transposed.
//
// Why pairs: a block's 128 x 256 tile reads 12 KB of shared memory per K = 16
// step (128 cycles of the tensor pipe) while TMA writes as much, which held the
// pipe at 75% (ncu); a pair reads each half of B once for both blocks, 8 KB and
// 8 KB.
#pragma once

#include "rs_expert_groups.cuh"
#include "rs_tc.cuh"

namespace rsx {

constexpr int kTcRows = 128;   // tile rows of a block
constexpr int kTcDepth = 64;   // reduction elements per stage: one swizzled row of 128 bytes
constexpr int kTcFirstEpilogueWarp = 4, kTcEpilogueWarps = 16;
constexpr int kTcThreads = 32 * (kTcFirstEpilogueWarp + kTcEpilogueWarps);
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
    uint32_t dependent;   // launched as the dependent of the kernel before it
    uint32_t wait_first;  // and needs what that one writes
    uint32_t stall;    // testing hook: tile stall - 1 is never copied
};

template <int BN, bool PAIR>
struct TcShape {
    static constexpr int kCols = PAIR ? BN / 2 : BN;  // B rows that a block holds
    static constexpr uint32_t kA = kTcRows * kTcDepth * 2, kB = kCols * kTcDepth * 2, kStage = kA + kB;
    static constexpr int kStages = kCols == 256 ? 4 : 6;
    static constexpr uint32_t kStaging = 32 * 32;  // bytes per epilogue warp: 32 rows of 16 elements
    static constexpr uint32_t kTileRows = PAIR ? 2 * kTcRows : kTcRows;
    static constexpr size_t smem(size_t experts)
    {
        return 1024 + (size_t)kStages * kStage + kTcEpilogueWarps * kStaging + (3 * kStages + 4) * 8 + 16 +
               Groups::words(experts) * 4;
    }
};

// Where a tile is: rows [i0, i_end) and columns from j0 of D, expert e, and
// the reduction [k0, k_end).
struct TcTile {
    uint32_t e, i0, i_end, j0, k0, k_end;
    __device__ __forceinline__ uint32_t slices() const { return (k_end - k0 + kTcDepth - 1) / kTcDepth; }
};

template <int BN, uint32_t ROWS, bool RAGGED_K, typename T>
__device__ __forceinline__ TcTile tc_tile(const TcArgs<T>& p, const Groups& g, uint32_t tile)
{
    const uint32_t across = (p.cols + BN - 1) / BN;
    const uint32_t down = tile / across;
    TcTile t;
    t.j0 = (tile - down * across) * BN;
    if constexpr (RAGGED_K) {
        const uint32_t per = (p.out_rows + ROWS - 1) / ROWS;
        t.e = down / per;
        t.i0 = (down - t.e * per) * ROWS;
        t.i_end = p.out_rows;
        t.k0 = g.off[t.e];
        t.k_end = g.off[t.e + 1];
    } else {
        t.e = g.find(down);
        t.i0 = g.off[t.e] + (down - g.tile[t.e]) * ROWS;
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

// How a warp's 32 x 16 piece of a matrix meets memory.  A lane holds a row of
// it as 16 elements: one whole 32-byte sector, which it loads or stores itself
// where the rows are 32-byte aligned and the piece is whole (`direct`).
// Otherwise the piece goes through shared memory, 2 lanes per row, so that
// memory sees 16-byte vectors where the rows allow those, and elements where
// not; the vectors are permuted by the row so that neither side has bank
// conflicts.
template <typename T>
struct Rows {
    T* p;
    size_t stride;
    bool direct, vec;
    __device__ __forceinline__ Rows(T* p, size_t stride, size_t expert_stride) : p(p), stride(stride)
    {
        const uintptr_t bits = (uintptr_t)p | stride * sizeof(T) | expert_stride * sizeof(T);
        direct = bits % 32 == 0;
        vec = bits % 16 == 0;
    }
};

__device__ __forceinline__ uint32_t stage_slot(uint32_t row, uint32_t vec) { return row * 2 + (vec ^ ((row >> 2) & 1)); }

template <typename T>
__device__ __forceinline__ void store_piece(uint4* stage, const uint32_t (&mine)[8], const Rows<T>& d, uint32_t i0,
                                            uint32_t i_end, uint32_t j0, uint32_t cols)
{
    const uint32_t lane = threadIdx.x % 32;
    if (d.direct && j0 + 16 <= cols) {
        if (i0 + lane < i_end) rstc::store_sector(d.p + (i0 + lane) * d.stride + j0, mine);
        return;
    }
    stage[stage_slot(lane, 0)] = make_uint4(mine[0], mine[1], mine[2], mine[3]);
    stage[stage_slot(lane, 1)] = make_uint4(mine[4], mine[5], mine[6], mine[7]);
    __syncwarp();
    if (d.vec && j0 + 16 <= cols) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const uint32_t row = n * 16 + lane / 2, q = lane % 2, i = i0 + row;
            if (i < i_end) *reinterpret_cast<uint4*>(d.p + i * d.stride + j0 + q * 8) = stage[stage_slot(row, q)];
        }
    } else {  // element by element, 16 lanes to a row
#pragma unroll 1
        for (int n = 0; n < 16; ++n) {
            const uint32_t row = n * 2 + lane / 16, c = lane % 16, i = i0 + row;
            const uint16_t v = reinterpret_cast<const uint16_t*>(stage)[stage_slot(row, c / 8) * 8 + c % 8];
            if (i < i_end && j0 + c < cols) reinterpret_cast<uint16_t*>(d.p)[i * d.stride + j0 + c] = v;
        }
    }
    __syncwarp();
}

// The reverse, in two steps: the piece as the accesses bring it (zeros
// outside), fetched ahead of its use, and then this lane's row of it.
template <typename T>
__device__ __forceinline__ void fetch_piece(uint32_t (&v)[8], const Rows<const T>& d, uint32_t i0, uint32_t i_end,
                                            uint32_t j0, uint32_t cols)
{
    const uint32_t lane = threadIdx.x % 32;
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = 0;
    if (d.direct && j0 + 16 <= cols) {
        if (i0 + lane < i_end) rstc::load_sector(v, d.p + (i0 + lane) * d.stride + j0);
        return;
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const uint32_t row = n * 16 + lane / 2, q = lane % 2, i = i0 + row, j = j0 + q * 8;
        if (i < i_end && j < cols) {
            const T* from = d.p + i * d.stride + j;
            if (d.vec && j + 8 <= cols) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(from));
                v[4 * n] = u.x, v[4 * n + 1] = u.y, v[4 * n + 2] = u.z, v[4 * n + 3] = u.w;
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (j + c < cols)
                        v[4 * n + c / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(from)[c] << (c & 1) * 16;
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void spread_piece(uint4* stage, uint32_t (&v)[8], const Rows<const T>& d, uint32_t j0,
                                             uint32_t cols)
{
    if (d.direct && j0 + 16 <= cols) return;
    const uint32_t lane = threadIdx.x % 32;
#pragma unroll
    for (int n = 0; n < 2; ++n)
        stage[stage_slot(n * 16 + lane / 2, lane % 2)] = make_uint4(v[4 * n], v[4 * n + 1], v[4 * n + 2], v[4 * n + 3]);
    __syncwarp();
    const uint4 lo = stage[stage_slot(lane, 0)], hi = stage[stage_slot(lane, 1)];
    v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
    v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
    __syncwarp();
}

// z = act(z)
template <int ACT>
__device__ __forceinline__ void activate_all(uint32_t (&z)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = __float_as_uint(activate<ACT, true>(__uint_as_float(z[i])));
}

// z += v (16 elements)
template <typename T>
__device__ __forceinline__ void add_all(uint32_t (&z)[16], const uint32_t (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = unpack2<T>(v[i]);
        z[2 * i] = __float_as_uint(__uint_as_float(z[2 * i]) + f.x);
        z[2 * i + 1] = __float_as_uint(__uint_as_float(z[2 * i + 1]) + f.y);
    }
}

template <typename T>
__device__ __forceinline__ void round_all(uint32_t (&out)[8], const uint32_t (&z)[16])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = pack2<T>(__uint_as_float(z[2 * i]), __uint_as_float(z[2 * i + 1]));
}

template <typename T>
__device__ __forceinline__ void add_bias(uint32_t (&z)[16], const T* bias, uint32_t left, bool vec)
{
    uint32_t w[8] = {};
    if (vec && left >= 16) {
        const uint4 lo = __ldg(reinterpret_cast<const uint4*>(bias)), hi = __ldg(reinterpret_cast<const uint4*>(bias) + 1);
        w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
        w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < left) w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(bias)[i] << (i & 1) * 16;
    }
    add_all<T>(z, w);
}

// A pair's tile of at most 128 rows is multiplied as one of 128 rows, 64 to a
// block, in half the time (an expert's last tile, every second time).
template <bool PAIR, bool RAGGED_K>
__device__ __forceinline__ bool half_tile(const TcTile& t)
{
    return PAIR && !RAGGED_K && t.i_end - t.i0 <= kTcRows;
}

// Zeros over rows [left, next multiple of 16) of every box of 64 columns in a
// stage (the steps of 16 after that are not multiplied); a whole warp.
template <uint32_t STAGE>
__device__ __forceinline__ void mend_slice(unsigned char* stage, uint32_t left)
{
    const uint32_t vecs = ((left + 15) / 16 * 16 - left) * 8;
    for (uint32_t v = threadIdx.x % 32; v < vecs; v += 32)
#pragma unroll
        for (uint32_t i = 0; i < STAGE / 8192; ++i)
            reinterpret_cast<uint4*>(stage + i * 8192 + left * 128)[v] = make_uint4(0, 0, 0, 0);
    rstc::fence_async();
    __syncwarp();
}

// Ragged rows: A is K-major rows of map_a (2-d), B is per expert (map_b, 3-d),
// its row index adjacent in memory (B_MN) or its reduction index.  Ragged
// reduction: both are MN-major columns of 2-d maps.  With 128
// columns the tiles of ragged rows are often far from full, and A is copied in
// boxes of 16 rows, as many as the tile has rows for.
template <typename T, int BN, bool RAGGED_K, bool B_MN, bool PAIR>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_product_tc(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, TcArgs<T> p)
{
    using namespace rstc;
    using S = TcShape<BN, PAIR>;
    constexpr bool A_MN = RAGGED_K, FEW = BN == 128 && !RAGGED_K;
    static_assert(!RAGGED_K || B_MN, "both operands of a ragged reduction are MN-major");
    extern __shared__ unsigned char raw[];
    unsigned char* ring = raw + (1024 - smem_addr(raw) % 1024) % 1024;  // stages are 1024-byte aligned
    unsigned char* staging = ring + S::kStages * S::kStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + kTcEpilogueWarps * S::kStaging);
    uint64_t* empty = full + S::kStages;
    uint64_t* tail = empty + S::kStages;  // of slices that warp 3 mends
    uint64_t* acc_full = tail + S::kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    uint32_t* failed = slot + 1;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = PAIR ? cluster_rank() : 0, blocks = PAIR ? 2 : 1;
    const uint32_t first_tile = blockIdx.x / blocks, tile_step = gridDim.x / blocks;

    if (threadIdx.x == 32) {
        tma_prefetch(&map_a);
        tma_prefetch(&map_b);
        for (int s = 0; s < S::kStages; ++s) {
            // the leader's: one arrival with the bytes of both blocks, or (ragged
            // reduction) one of each block, from its copying or mending warp
            bar_init(full + s, RAGGED_K ? blocks : 1);
            bar_init(empty + s, 1);  // each block's own
            bar_init(tail + s, 1);   // each block's own
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(acc_full + s, 1);                            // each block's own
            bar_init(acc_empty + s, kTcEpilogueWarps * blocks);   // the leader's
        }
        bar_init_fence();
        *failed = 0;
    }
    if (warp == 2) tmem_alloc<PAIR>(slot, 512);
    tc_fence_before();
    // (the barrier inside make() orders all of the above)
    const Groups g = Groups::make(slot + 4, p.offsets, p.experts, p.rows, S::kTileRows, !RAGGED_K);
    if (p.wait_first) wait_prior_grid();
    start_next_grid();
    if constexpr (PAIR) cluster_sync();  // the other block's barriers are ready too
    tc_fence_after();
    const uint32_t tmem = *slot;
    const uint32_t across = (p.cols + BN - 1) / BN;
    const uint32_t tiles =
        (RAGGED_K ? (p.out_rows + S::kTileRows - 1) / S::kTileRows * p.experts : g.tiles()) * across;

    uint32_t issued = 0;  // stages filled so far (the copying warp)
    if (warp == 0) {
        uint32_t s = 0, round = 0;
        bool ok = true;
        for (uint32_t tile = first_tile; ok && tile < tiles; tile += tile_step) {
            const TcTile t = tc_tile<BN, S::kTileRows, RAGGED_K>(p, g, tile);
            if (tile + 1 == p.stall) break;
            const bool half = half_tile<PAIR, RAGGED_K>(t);
            const uint32_t own = half ? kTcRows / 2 : kTcRows;  // rows of a block
            const int i0 = (int)(t.i0 + rank * own), j0 = (int)(t.j0 + rank * S::kCols);
            // Rows past the expert's end are not stored, so whole boxes of them are
            // not copied: what the stage held before stands in for them.
            const uint32_t rows = RAGGED_K ? 0 : t.i_end - t.i0;  // of the tile, and more
            const uint32_t a_boxes = FEW ? min((rows + 15) / 16, kTcRows / 16u) : 1;
            const bool second = PAIR && !RAGGED_K && rows > own;  // the pair's second block has rows
            const uint32_t tile_bytes = RAGGED_K ? S::kStage
                                        : PAIR   ? 2 * S::kB + (second ? 2 : 1) * S::kA
                                        : FEW    ? S::kB + a_boxes * 2048
                                                 : S::kStage;
            for (uint32_t k = t.k0; k < t.k_end; k += kTcDepth, ++issued) {
                ok = bar_wait_warp(empty + s, (round & 1) ^ 1);
                if (!ok) break;
                unsigned char* a = ring + s * S::kStage;
                unsigned char* b = a + S::kA;
                if (elect_one()) {
                    uint32_t bar = PAIR ? cluster_addr(full + s, 0) : smem_addr(full + s);
                    if constexpr (RAGGED_K) {
                        if (t.k_end - k < kTcDepth) {
                            bar = PAIR ? cluster_addr(tail + s, rank) : smem_addr(tail + s);
                            bar_expect(tail + s, S::kStage);
                        } else if (rank != 0) {
                            bar_expect_cluster(bar, S::kStage);
                        } else {
                            bar_expect(full + s, S::kStage);
                        }
                    } else if (rank == 0) {
                        bar_expect(full + s, tile_bytes);
                    }
                    if constexpr (RAGGED_K) {
#pragma unroll
                        for (int i = 0; i < kTcRows / 64; ++i)
                            tma_load_2d<PAIR>(a + i * 8192, &map_a, i0 + i * 64, (int)k, bar);
#pragma unroll
                        for (int i = 0; i < S::kCols / 64; ++i)
                            tma_load_2d<PAIR>(b + i * 8192, &map_b, j0 + i * 64, (int)k, bar);
                    } else {
                        const int e = (int)(t.e * p.b_expert);
                        if constexpr (FEW) {
                            for (uint32_t i = 0; i < a_boxes; ++i)
                                tma_load_2d<PAIR>(a + i * 2048, &map_a, (int)k, i0 + (int)i * 16, bar);
                        } else if (!PAIR || rank == 0 || second) {
                            tma_load_2d<PAIR>(a, &map_a, (int)k, i0, bar);
                        }
                        if constexpr (B_MN) {
#pragma unroll
                            for (int i = 0; i < S::kCols / 64; ++i)
                                tma_load_3d<PAIR>(b + i * 8192, &map_b, j0 + i * 64, (int)k, e, bar);
                        } else {
                            tma_load_3d<PAIR>(b, &map_b, (int)k, j0, e, bar);
                        }
                    }
                }
                __syncwarp();
                if (++s == S::kStages) s = 0, ++round;
            }
        }
        if (!ok) *failed = 1;
    } else if (warp == 1 && rank == 0) {
        constexpr uint32_t kWhole = mma_desc(!__is_same(T, __half), A_MN, B_MN, S::kTileRows, BN);
        constexpr uint32_t kHalf = mma_desc(!__is_same(T, __half), A_MN, B_MN, S::kTileRows / 2, BN);
        constexpr uint32_t kAStep = A_MN ? 2048 : 32, kBStep = B_MN ? 2048 : 32;
        const uint64_t desc_a = smem_desc(smem_addr(ring), A_MN ? 8192 : 16);
        const uint64_t desc_b = smem_desc(smem_addr(ring) + S::kA, B_MN ? 8192 : 16);
        uint32_t s = 0, round = 0, n = 0;
        bool ok = true;
        for (uint32_t tile = first_tile; ok && tile < tiles; tile += tile_step) {
            const TcTile t = tc_tile<BN, S::kTileRows, RAGGED_K>(p, g, tile);
            if (t.k0 >= t.k_end) continue;
            const uint32_t h = n & 1, acc = tmem + h * 256, free = ((n >> 1) & 1) ^ 1;
            ok = PAIR ? bar_wait_cluster_warp(acc_empty + h, free) : bar_wait_warp(acc_empty + h, free);
            if (!ok) break;
            tc_fence_after();
            ++n;
            const uint32_t desc = half_tile<PAIR, RAGGED_K>(t) ? kHalf : kWhole;
            uint32_t more = 0;  // nothing accumulated yet
            for (uint32_t k = t.k0; k < t.k_end; k += kTcDepth) {
                ok = PAIR && RAGGED_K ? bar_wait_cluster_warp(full + s, round & 1) : bar_wait_warp(full + s, round & 1);
                if (!ok) break;
                const uint32_t steps = RAGGED_K ? min((t.k_end - k + 15) / 16, kTcDepth / 16u) : kTcDepth / 16;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t da = desc_a + s * (S::kStage >> 4), db = desc_b + s * (S::kStage >> 4);
                    if (steps == kTcDepth / 16) {
#pragma unroll
                        for (uint32_t i = 0; i < kTcDepth / 16; ++i)
                            mma_f16<PAIR>(acc, da + i * (kAStep >> 4), db + i * (kBStep >> 4), desc, more | i);
                    } else {
                        for (uint32_t i = 0; i < steps; ++i)
                            mma_f16<PAIR>(acc, da + i * (kAStep >> 4), db + i * (kBStep >> 4), desc, more | i);
                    }
                    mma_commit<PAIR>(empty + s);
                }
                __syncwarp();
                more = 1;
                if (++s == S::kStages) s = 0, ++round;
            }
            if (ok && elect_one()) mma_commit<PAIR>(acc_full + h);
            __syncwarp();
        }
        // What was issued is done before anything it uses is given up, also when
        // the epilogue's wait for it has run out.
        if (s || round) ok &= bar_wait_warp(empty + (s ? s : S::kStages) - 1, (s ? round : round - 1) & 1);
        if (!ok) *failed = 1;
    } else if (RAGGED_K && warp == 3) {
        uint32_t used = 0, phases = 0;  // slices so far; bit s: the next phase of tail[s]
        uint32_t skipped = 0;           // of `used`, those since the last wait
        for (uint32_t tile = first_tile; tile < tiles; tile += tile_step) {
            const TcTile t = tc_tile<BN, S::kTileRows, RAGGED_K>(p, g, tile);
            used += t.slices();
            skipped += t.slices();
            const uint32_t left = (t.k_end - t.k0) % kTcDepth;
            if (left == 0) continue;
            const uint32_t s = (used - 1) % S::kStages;
            if (!bar_wait_warp(tail + s, phases >> s & 1, skipped)) {
                *failed = 1;
                break;
            }
            skipped = 0;
            phases ^= 1u << s;
            mend_slice<S::kStage>(ring + s * S::kStage, left);
            if (elect_one()) {
                if constexpr (PAIR) bar_arrive_cluster<true>(cluster_addr(full + s, 0));
                else bar_arrive(full + s);
            }
            __syncwarp();
        }
    } else if (warp >= kTcFirstEpilogueWarp) {
        constexpr uint32_t kPer = BN / (kTcEpilogueWarps / 4);  // columns per warp
        const uint32_t w = warp - kTcFirstEpilogueWarp;
        const uint32_t quarter = warp % 4;  // the 32 tensor-memory lanes this warp can read
        uint4* stage = reinterpret_cast<uint4*>(staging + w * S::kStaging);
        Rows<T> d(p.d, p.d_i, RAGGED_K ? p.d_e : 0);
        const Rows<T> pre(p.pre, p.pre_i, 0);
        const Rows<const T> residual(p.residual, p.residual_i, 0);
        const bool vec_bias = ((uintptr_t)p.bias | p.bias_e * sizeof(T)) % 16 == 0;
        uint32_t n = 0;
        // A first tile that takes a while is gone through twice.  The rehearsal,
        // while it is being multiplied, waits for nothing, frees nothing and stores
        // no row; it brings this code and the bias into the caches (uncached a piece
        // takes 2300 cycles, then 1500: 1000 rows of 4 experts of 2048 x 2048
        // 15.9 us without, 15.0 with; 64 rows with reduce = 128 would lose 1 us).
        bool rehearsal = (RAGGED_K ? p.rows / p.experts : p.reduce) >= 512;
        for (uint32_t tile = first_tile; tile < tiles; tile += rehearsal ? 0 : tile_step, rehearsal = false) {
            TcTile t = tc_tile<BN, S::kTileRows, RAGGED_K>(p, g, tile);
            const bool some = t.k0 < t.k_end;
            const uint32_t h = n & 1;
            // A half tile's rows are 64 to a block: tensor memory holds columns 0..127
            // of D in lanes 0..63 and columns 128..255 in lanes 64..127.
            const bool half = half_tile<PAIR, RAGGED_K>(t);
            const uint32_t per = half ? kPer / 2 : kPer, c0 = w / 4 * per;  // this warp's columns in tensor memory
            const uint32_t i0 = t.i0 + rank * (half ? 64 : kTcRows) + (half ? quarter % 2 : quarter) * 32;
            const uint32_t j_first = t.j0 + (half ? quarter / 2 * (BN / 2) : 0);  // D's column of column 0 there
            if constexpr (RAGGED_K) d.p = p.d + t.e * p.d_e;
            // a piece with no rows or columns to store is not read either
            const uint32_t c_end = i0 >= t.i_end || j_first + c0 >= p.cols ? c0 : min(c0 + per, p.cols - j_first);
            if (rehearsal) t.i_end = 0;  // (once the columns are known)
            // One piece ahead: the next piece's accumulators and residual are on
            // their way while this one is finished (a load from tensor memory takes
            // about 1000 cycles beside a busy tensor pipe), the first piece's
            // residual while the tile is still being multiplied.
            uint32_t z[2][16], add[2][8];
            auto fetch_residual = [&](uint32_t c, uint32_t (&r)[8]) {
                if (p.residual && c < c_end) fetch_piece<T>(r, residual, i0, t.i_end, j_first + c, p.cols);
            };
            auto fetch_acc = [&](uint32_t c, uint32_t (&zz)[16]) {
                if (c < c_end) tmem_load16(zz, tmem + h * 256 + c + (quarter << 21));  // lane 32 * quarter on top
            };
            // this warp's part of the accumulator has been read: it may be multiplied into again
            auto release = [&] {
                if (rehearsal) return;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) bar_arrive_cluster<false>(cluster_addr(acc_empty + h, 0));
                    else bar_arrive(acc_empty + h);
                }
            };
            if (some) {
                fetch_residual(c0, add[0]);
                if (!rehearsal) {
                    if (!bar_wait_warp(acc_full + h, (n >> 1) & 1, t.slices())) {
                        *failed = 1;
                        break;
                    }
                    tc_fence_after();
                    ++n;
                }
                if (c0 >= c_end) release();
                fetch_acc(c0, z[0]);
#pragma unroll 1
                for (uint32_t c2 = c0; c2 < c_end; c2 += 32)
#pragma unroll
                for (uint32_t q = 0; q < 2; ++q) {
                    const uint32_t c = c2 + q * 16, j = j_first + c;
                    if (c >= c_end) break;
                    uint32_t(&zz)[16] = z[q & 1];
                    tmem_load_wait(zz);
                    if (c + 16 >= c_end) release();
                    fetch_acc(c + 16, z[(q & 1) ^ 1]);
                    fetch_residual(c + 16, add[(q & 1) ^ 1]);
                    uint32_t out[8];
                    if (p.bias) add_bias<T>(zz, p.bias + t.e * p.bias_e + j, p.cols - j, vec_bias);
                    if (p.pre) {
                        round_all<T>(out, zz);
                        store_piece<T>(stage, out, pre, i0, t.i_end, j, p.cols);
                    }
                    if (p.act == RS_ACT_RELU) activate_all<RS_ACT_RELU>(zz);
                    else if (p.act == RS_ACT_GELU) activate_all<RS_ACT_GELU>(zz);
                    else if (p.act == RS_ACT_SILU) activate_all<RS_ACT_SILU>(zz);
                    if (p.residual) {
                        spread_piece<T>(stage, add[q & 1], residual, j, p.cols);
                        add_all<T>(zz, add[q & 1]);
                    }
                    round_all<T>(out, zz);
                    store_piece<T>(stage, out, d, i0, t.i_end, j, p.cols);
                }
            } else {  // unused rows, or an expert without rows
                const uint32_t out[8] = {};
                for (uint32_t c = c0; c < c_end; c += 16) {
                    if (p.pre) store_piece<T>(stage, out, pre, i0, t.i_end, j_first + c, p.cols);
                    store_piece<T>(stage, out, d, i0, t.i_end, j_first + c, p.cols);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // neither block's memory goes while the other's work may reach it
    tc_fence_after();
    if (threadIdx.x == 0) {
        if (*failed && rank == 0)  // a copy must not land in shared memory that its block no longer owns
            for (uint32_t s = 0; s < S::kStages && s < issued; ++s) {
                const uint32_t last = (issued - 1 - s) / S::kStages;
                bar_wait(full + s, last & 1);
            }
        p.status[blockIdx.x] = *failed;
    }
    if (blockIdx.x == 0)
        for (uint32_t i = gridDim.x + threadIdx.x; i < p.status_words; i += kTcThreads) p.status[i] = 0;
    __syncthreads();
    if constexpr (PAIR) cluster_sync();
    if (warp == 2) tmem_free<PAIR>(tmem, 512);
    wait_prior_grid();
}

// Launches one product.  Bases and strides are multiples of 16 bytes, strides
// below 2^40 bytes (the caller's checks and copies see to it); RS_ERR_CUDA if
// the driver makes no tensor map.  Instantiated in rs_expert_tc_<type>.cu.
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
