// rs_expert_split.cuh -- an expert product with fewer tiles than SMs: the
// reduction of each 128 x 128 tile is cut over a cluster of blocks.
//
// Block r of C multiplies its share of the 64-deep slices into its own tensor
// memory, as in rs_expert_tc.cuh, and lays the float32 partial tile in its
// shared memory.  Once all C have (an mbarrier in every block that all warps of
// the cluster arrive on), block r finishes the rows i = r mod C: it reads the
// C partial values of an element over the cluster's network, adds them in block
// order, applies the epilogue and stores.  Nothing goes through global memory
// and the order of the additions is fixed.
//
// What bounds it: a block alone takes 0.22 us per slice, the round trip of its
// copies over the depth of its ring, so a single tile of 64 slices took 17.9 us
// and 64 rows of one expert of 4096 x 4096 (32 tiles) 20.4; figures with the
// reduction cut are at the rule, in rs_expert_tc_launch.cuh.
#pragma once

#include "rs_expert_tc.cuh"

namespace rsx {

struct SplitShape {
    static constexpr int kBN = 128, kStages = 4;
    static constexpr uint32_t kA = kTcRows * kTcDepth * 2, kB = kBN * kTcDepth * 2, kStage = kA + kB;
    static constexpr uint32_t kPitch = kBN + 4;  // floats per row of the partial tile: no bank conflicts
    static constexpr uint32_t kPart = kTcRows * kPitch * 4;
    static constexpr size_t smem(size_t experts)
    {
        return 1024 + kStages * kStage + kPart + (3 * kStages + 4) * 8 + 16 + Groups::words(experts) * 4;
    }
};

__device__ __forceinline__ float4 load_cluster4(uint32_t cluster_addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

// Four elements of a row from column j on.
template <typename T>
__device__ __forceinline__ void store4(const Rows<T>& d, uint32_t i, uint32_t j, uint32_t cols, const float (&v)[4])
{
    T* to = d.p + i * d.stride + j;
    if (d.vec && j + 4 <= cols) {
        *reinterpret_cast<uint2*>(to) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (j + c < cols) to[c] = from_float<T>(v[c]);
    }
}

// A block's share [begin, end) of a tile's reduction, in whole slices.
struct Share {
    uint32_t begin, end;
    __device__ __forceinline__ Share(const TcTile& t, uint32_t rank, uint32_t blocks)
    {
        const uint32_t slices = t.slices();
        begin = t.k0 + (uint32_t)((uint64_t)slices * rank / blocks) * kTcDepth;
        end = min(t.k0 + (uint32_t)((uint64_t)slices * (rank + 1) / blocks) * kTcDepth, t.k_end);
    }
    __device__ __forceinline__ uint32_t slices() const { return (end - begin + kTcDepth - 1) / kTcDepth; }
};

// RAGGED_K and B_MN as in k_product_tc.
template <typename T, bool RAGGED_K, bool B_MN>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_product_split(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, TcArgs<T> p)
{
    using namespace rstc;
    using S = SplitShape;
    extern __shared__ unsigned char raw[];
    unsigned char* ring = raw + (1024 - smem_addr(raw) % 1024) % 1024;  // stages are 1024-byte aligned
    float* part = reinterpret_cast<float*>(ring + S::kStages * S::kStage);
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + S::kStages * S::kStage + S::kPart);
    uint64_t* empty = full + S::kStages;
    uint64_t* tail = empty + S::kStages;  // of slices that warp 3 mends
    uint64_t* acc_full = tail + S::kStages;
    uint64_t* acc_empty = acc_full + 1;
    uint64_t* part_full = acc_full + 2;   // every block's partial tile is written
    uint64_t* part_empty = acc_full + 3;  // this block's has been read by every block
    uint32_t* slot = reinterpret_cast<uint32_t*>(acc_full + 4);
    uint32_t* failed = slot + 1;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank(), blocks = cluster_size();
    const uint32_t first_tile = blockIdx.x / blocks, tile_step = gridDim.x / blocks;

    if (threadIdx.x == 32) {
        tma_prefetch(&map_a);
        tma_prefetch(&map_b);
        for (int s = 0; s < S::kStages; ++s) {
            bar_init(full + s, 1);
            bar_init(empty + s, 1);
            bar_init(tail + s, 1);
        }
        bar_init(acc_full, 1);
        bar_init(acc_empty, kTcEpilogueWarps);
        bar_init(part_full, kTcEpilogueWarps * blocks);
        bar_init(part_empty, kTcEpilogueWarps * blocks);
        bar_init_fence();
        *failed = 0;
    }
    if (warp == 2) tmem_alloc<false>(slot, S::kBN);
    tc_fence_before();
    // (the barrier inside make() orders all of the above)
    const Groups g = Groups::make(slot + 4, p.offsets, p.experts, p.rows, kTcRows, !RAGGED_K);
    if (p.wait_first) wait_prior_grid();
    start_next_grid();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *slot;
    const uint32_t tiles =
        (RAGGED_K ? (p.out_rows + kTcRows - 1) / kTcRows * p.experts : g.tiles()) * ((p.cols + S::kBN - 1) / S::kBN);

    uint32_t issued = 0;
    if (warp == 0) {
        uint32_t s = 0, round = 0;
        bool ok = true;
        for (uint32_t tile = first_tile; ok && tile < tiles; tile += tile_step) {
            const TcTile t = tc_tile<S::kBN, kTcRows, RAGGED_K>(p, g, tile);
            if (t.k0 >= t.k_end) continue;
            if (tile + 1 == p.stall) break;
            const Share share(t, rank, blocks);
            const uint32_t boxes = min((t.i_end - t.i0 + 15) / 16, kTcRows / 16u);
            const int e = (int)(t.e * p.b_expert);
            for (uint32_t k = share.begin; k < share.end; k += kTcDepth, ++issued) {
                ok = bar_wait_warp(empty + s, (round & 1) ^ 1);
                if (!ok) break;
                unsigned char* a = ring + s * S::kStage;
                unsigned char* b = a + S::kA;
                if (elect_one()) {
                    uint64_t* ready = RAGGED_K && t.k_end - k < kTcDepth ? tail + s : full + s;
                    const uint32_t bar = smem_addr(ready);
                    bar_expect(ready, RAGGED_K ? S::kStage : S::kB + boxes * 2048);
                    if constexpr (RAGGED_K) {
#pragma unroll
                        for (int i = 0; i < kTcRows / 64; ++i)
                            tma_load_2d<false>(a + i * 8192, &map_a, (int)(t.i0 + i * 64), (int)k, bar);
#pragma unroll
                        for (int i = 0; i < S::kBN / 64; ++i)
                            tma_load_2d<false>(b + i * 8192, &map_b, (int)(t.j0 + i * 64), (int)k, bar);
                    } else {
                        for (uint32_t i = 0; i < boxes; ++i)
                            tma_load_2d<false>(a + i * 2048, &map_a, (int)k, (int)(t.i0 + i * 16), bar);
                    }
                    if constexpr (RAGGED_K) {
                    } else if constexpr (B_MN) {
#pragma unroll
                        for (int i = 0; i < S::kBN / 64; ++i)
                            tma_load_3d<false>(b + i * 8192, &map_b, (int)(t.j0 + i * 64), (int)k, e, bar);
                    } else {
                        tma_load_3d<false>(b, &map_b, (int)k, (int)t.j0, e, bar);
                    }
                }
                __syncwarp();
                if (++s == S::kStages) s = 0, ++round;
            }
        }
        if (!ok) *failed = 1;
    } else if (warp == 1) {
        constexpr uint32_t kDesc = mma_desc(!__is_same(T, __half), RAGGED_K, B_MN, kTcRows, S::kBN);
        constexpr uint32_t kAStep = RAGGED_K ? 2048 : 32, kBStep = B_MN ? 2048 : 32;
        const uint64_t desc_a = smem_desc(smem_addr(ring), RAGGED_K ? 8192 : 16);
        const uint64_t desc_b = smem_desc(smem_addr(ring) + S::kA, B_MN ? 8192 : 16);
        uint32_t s = 0, round = 0, n = 0;
        bool ok = true;
        for (uint32_t tile = first_tile; ok && tile < tiles; tile += tile_step) {
            const TcTile t = tc_tile<S::kBN, kTcRows, RAGGED_K>(p, g, tile);
            if (t.k0 >= t.k_end) continue;
            const Share share(t, rank, blocks);
            ok = bar_wait_warp(acc_empty, (n & 1) ^ 1);
            if (!ok) break;
            tc_fence_after();
            ++n;
            uint32_t more = 0;
            for (uint32_t k = share.begin; k < share.end; k += kTcDepth) {
                ok = bar_wait_warp(full + s, round & 1);
                if (!ok) break;
                const uint32_t steps = RAGGED_K ? min((t.k_end - k + 15) / 16, kTcDepth / 16u) : kTcDepth / 16;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t da = desc_a + s * (S::kStage >> 4), db = desc_b + s * (S::kStage >> 4);
                    if (steps == kTcDepth / 16) {
#pragma unroll
                        for (uint32_t i = 0; i < kTcDepth / 16; ++i)
                            mma_f16<false>(tmem, da + i * (kAStep >> 4), db + i * (kBStep >> 4), kDesc, more | i);
                    } else {
                        for (uint32_t i = 0; i < steps; ++i)
                            mma_f16<false>(tmem, da + i * (kAStep >> 4), db + i * (kBStep >> 4), kDesc, more | i);
                    }
                    mma_commit<false>(empty + s);
                }
                __syncwarp();
                more = 1;
                if (++s == S::kStages) s = 0, ++round;
            }
            if (ok && elect_one()) mma_commit<false>(acc_full);
            __syncwarp();
        }
        // as in k_product_tc: what was issued is done before anything it uses is given up
        if (s || round) ok &= bar_wait_warp(empty + (s ? s : S::kStages) - 1, (s ? round : round - 1) & 1);
        if (!ok) *failed = 1;
    } else if (RAGGED_K && warp == 3) {
        uint32_t used = 0, phases = 0;  // slices so far; bit s: the next phase of tail[s]
        uint32_t skipped = 0;           // of `used`, those since the last wait
        for (uint32_t tile = first_tile; tile < tiles; tile += tile_step) {
            const TcTile t = tc_tile<S::kBN, kTcRows, RAGGED_K>(p, g, tile);
            if (t.k0 >= t.k_end) continue;
            const Share share(t, rank, blocks);
            if (share.begin >= share.end) continue;
            used += share.slices();
            skipped += share.slices();
            const uint32_t left = (share.end - share.begin) % kTcDepth;
            if (left == 0) continue;
            const uint32_t s = (used - 1) % S::kStages;
            if (!bar_wait_warp(tail + s, phases >> s & 1, skipped)) {
                *failed = 1;
                break;
            }
            skipped = 0;
            phases ^= 1u << s;
            mend_slice<S::kStage>(ring + s * S::kStage, left);
            if (elect_one()) bar_arrive(full + s);
            __syncwarp();
        }
    } else if (warp >= kTcFirstEpilogueWarp) {
        const uint32_t w = warp - kTcFirstEpilogueWarp, quarter = warp % 4, c0 = w / 4 * 32;
        Rows<T> d(p.d, p.d_i, RAGGED_K ? p.d_e : 0);
        const Rows<T> pre(p.pre, p.pre_i, 0);
        const uint32_t peer = cluster_addr(part, lane < blocks ? lane : 0);  // lane r: block r's partial tile
        const uint32_t told_full = cluster_addr(part_full, lane < blocks ? lane : 0);
        const uint32_t told_empty = cluster_addr(part_empty, lane < blocks ? lane : 0);
        uint32_t n = 0;
        for (uint32_t tile = first_tile; tile < tiles; tile += tile_step) {
            const TcTile t = tc_tile<S::kBN, kTcRows, RAGGED_K>(p, g, tile);
            const uint32_t rows = min(t.i_end - t.i0, (uint32_t)kTcRows), j = t.j0 + lane * 4;
            const float nothing[4] = {};
            if constexpr (RAGGED_K) d.p = p.d + t.e * p.d_e;
            if (t.k0 >= t.k_end) {  // unused rows, or an expert without rows
                for (uint32_t i = rank + blocks * w; i < rows && j < p.cols; i += blocks * kTcEpilogueWarps) {
                    if (p.pre) store4<T>(pre, t.i0 + i, j, p.cols, nothing);
                    store4<T>(d, t.i0 + i, j, p.cols, nothing);
                }
                continue;
            }
            const Share share(t, rank, blocks);
            if (!bar_wait_warp(acc_full, n & 1, share.slices()) || !bar_wait_cluster_warp(part_empty, (n & 1) ^ 1)) {
                *failed = 1;
                break;
            }
            tc_fence_after();
            if (quarter * 32 < rows) {
                const uint32_t row = quarter * 32 + lane;
#pragma unroll
                for (uint32_t c = c0; c < c0 + 32; c += 16) {
                    uint32_t z[16];
                    tmem_load16(z, tmem + c + (quarter << 21));
                    tmem_load_wait(z);
                    if (share.begin >= share.end) {  // nothing was multiplied
#pragma unroll
                        for (int q = 0; q < 16; ++q) z[q] = 0;
                    }
                    if (row < rows) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *reinterpret_cast<uint4*>(part + row * S::kPitch + c + 4 * q) =
                                make_uint4(z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(acc_empty);
            if (lane < blocks) bar_arrive_cluster<true>(told_full);
            if (!bar_wait_cluster_warp(part_full, n & 1, share.slices())) {
                *failed = 1;
                break;
            }
            ++n;
            for (uint32_t i = rank + blocks * w; i < rows; i += blocks * kTcEpilogueWarps) {
                float z[4] = {};
                for (uint32_t r = 0; r < blocks; ++r) {
                    const uint32_t from = __shfl_sync(0xFFFFFFFFu, peer, r);
                    const float4 v = load_cluster4(from + (i * S::kPitch + lane * 4) * 4);
                    z[0] += v.x, z[1] += v.y, z[2] += v.z, z[3] += v.w;
                }
                if (j >= p.cols) continue;
                if (p.bias) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (j + c < p.cols) z[c] += to_float(p.bias[t.e * p.bias_e + j + c]);
                }
                if (p.pre) store4<T>(pre, t.i0 + i, j, p.cols, z);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (p.act == RS_ACT_RELU) z[c] = activate<RS_ACT_RELU, true>(z[c]);
                    else if (p.act == RS_ACT_GELU) z[c] = activate<RS_ACT_GELU, true>(z[c]);
                    else if (p.act == RS_ACT_SILU) z[c] = activate<RS_ACT_SILU, true>(z[c]);
                    if (p.residual && j + c < p.cols)
                        z[c] += to_float(p.residual[(t.i0 + i) * p.residual_i + j + c]);
                }
                store4<T>(d, t.i0 + i, j, p.cols, z);
            }
            __syncwarp();
            // what was read is in registers by now
            if (lane < blocks) bar_arrive_cluster<false>(told_empty);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no block's shared memory goes while another may read it
    tc_fence_after();
    if (threadIdx.x == 0) {
        if (*failed)  // a copy must not land in shared memory that this block no longer owns
            for (uint32_t s = 0; s < S::kStages && s < issued; ++s)
                bar_wait(full + s, (issued - 1 - s) / S::kStages & 1);
        p.status[blockIdx.x] = *failed;
    }
    if (blockIdx.x == 0)
        for (uint32_t i = gridDim.x + threadIdx.x; i < p.status_words; i += kTcThreads) p.status[i] = 0;
    __syncthreads();
    if (warp == 2) tmem_free<false>(tmem, S::kBN);
    wait_prior_grid();
}

}  // namespace rsx
