// rs_expert_sort.cu -- rs_expert_sort: the slots of a mixture-of-experts layer
// in stable order of their expert, the inverse of that order, and the
// experts' row ranges.
//
// This is one counting-sort pass on a digit of up to 1025 values (the experts
// and one more for dropped slots):
//     position(s) = base(e) + #{s' < s : expert(s') = e},  e = expert(s),
// base the exclusive scan of the experts' counts.  Slots are cut into one
// chunk of consecutive slots per block, a chunk into tiles of at most
// kTileSlots, a tile into one run of consecutive slots per warp.  Then
// #{s' < s, same expert} = slots of e in earlier chunks + in earlier tiles +
// in earlier warps of this tile + in earlier slots of this warp; the last two
// come from one counter per (warp, expert) in shared memory and from the lanes
// of equal expert: every lane sets its bit in its expert's mask (one word per
// (warp, expert), atomicOr) and reads it back.  An SM takes 70 cycles for
// __match_any_sync, 9 of the 23 us that 2^20 slots of 256 experts took with it,
// and 4.6 for each of the ballots that would do; ballots are left to the sorts
// of more than 511 experts, whose masks would not fit.  The whole sort is ONE kernel: up to
// kOneBlockSlots one block; up to kClusterSlots a cluster of 8, whose blocks
// read each other's counts over the cluster's network; above that a
// cooperative launch of at most one block per SM: every block publishes its
// counts, one warp per expert scans them over the blocks, and every block reads
// back its own.  (Every block
// summing all counts before its own needs one meeting of the grid less, 1.3 us,
// but reads blocks * experts words: 6.7 us.)  A block of such a grid puts a
// tile's slots in expert order in shared memory first, so that `order` is
// written in runs and not in single words (4.6 us).
//
// The bytes are few (12 or 16 per slot), so the time is launches and
// dependent round trips.  On the device alone (captured graph, int64 numbers):
// 512 slots of 128 experts 3.1 us, 30018 of 160 8.1, 65536 of 64 9.0, 2^20 of
// 256 17.7, of which 3.6 are the numbers' way from device memory (14.1 when the
// same input is sorted again).
#include <cooperative_groups.h>

#include "rs_expert_common.cuh"

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kItems = 8;  // slots per thread of a tile
constexpr uint32_t kTileSlots = kMaxThreads * kItems;
constexpr uint32_t kOneBlockSlots = 2048;
constexpr uint32_t kClusterBlocks = 8;
constexpr uint32_t kClusterSlots = kClusterBlocks * 4096;  // 30018 slots: 8.7 us, in a grid 9.4; 65536: 11.6, 9.1
constexpr uint32_t kChunkSlots = 2048;  // least slots per block of a cooperative launch
constexpr uint32_t kMaxBlocks = 256;
constexpr size_t kMaskBins = 512;  // masks for so many experts and the dropped slots

struct SortParams {
    const void* ids;
    int id_bytes;
    uint32_t n;
    uint32_t experts;
    uint32_t chunk;  // slots per block
    int32_t* order;
    int32_t* position;
    int32_t* offsets;
    bool cluster;      // the blocks are one cluster
    uint32_t* counts;  // [blocks][experts + 1], then [experts + 1] totals; unused by a single block
};

// The slot's expert, or `experts` for a dropped slot.
__device__ __forceinline__ uint32_t load_expert(const SortParams& p, uint32_t s)
{
    if (p.id_bytes == 8) {
        const unsigned long long v = __ldg(static_cast<const unsigned long long*>(p.ids) + s);
        return v < p.experts ? (uint32_t)v : p.experts;
    }
    const uint32_t v = __ldg(static_cast<const uint32_t*>(p.ids) + s);
    return v < p.experts ? v : p.experts;
}

// A block's shared memory: per expert the first row of its next slots (base),
// the tile's count (total) and the sum of the tile's counts of lower experts
// (local); per (warp, expert) a counter; and in a grid the tile's slots in
// expert order.  masks: and per (warp, expert) a mask of lanes, zero between uses.
struct Shared {
    uint32_t *base, *total, *local, *sorted, *mask;
    uint16_t* counter;
    uint32_t bins;
    __device__ __forceinline__ Shared(uint32_t* mem, uint32_t bins, bool grid, bool masks)
        : base(mem), total(mem + bins), local(mem + 2 * bins), sorted(mem + 3 * bins),
          mask(mem + 3 * bins + (grid ? kTileSlots : 0)),
          counter(reinterpret_cast<uint16_t*>(mask + (masks ? bins * (blockDim.x / 32) : 0))), bins(bins)
    {
    }
    static size_t bytes(size_t bins, size_t warps, bool grid, bool masks)
    {
        return 12 * bins + (grid ? 4 * kTileSlots : 0) + (masks ? 4 * bins * warps : 0) +
               2 * rsx::align_up(bins * warps, 2);
    }
};

// Where a thread's slots of a tile are: slots first + 32 * i, below end.
struct Run {
    uint32_t first, end;
    __device__ __forceinline__ Run(uint32_t begin, uint32_t len)
    {
        const uint32_t warps = blockDim.x / 32, warp = threadIdx.x / 32;
        const uint32_t per = ((len + warps - 1) / warps + 31) / 32 * 32;
        first = begin + warp * per + threadIdx.x % 32;
        end = min(begin + len, begin + (warp + 1) * per);
    }
};

// Ranks a tile's slots: rank[i] = expert << 16 | slots of that expert before
// this one in the warp's run; the counters end up as the warps' counts.
template <bool MASKS>
__device__ __forceinline__ void rank_tile(const SortParams& p, const Shared& sh, const Run& run,
                                          uint32_t (&rank)[kItems])
{
    if constexpr (MASKS)
        for (uint32_t i = threadIdx.x; i < sh.bins * (blockDim.x / 32); i += blockDim.x) sh.mask[i] = 0;
    uint32_t* pairs = reinterpret_cast<uint32_t*>(sh.counter);  // (a last odd counter is padded)
    for (uint32_t i = threadIdx.x; i < (sh.bins * (blockDim.x / 32) + 1) / 2; i += blockDim.x) pairs[i] = 0;
    uint32_t expert[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t s = run.first + 32 * i;
        expert[i] = s < run.end ? load_expert(p, s) : sh.bins;  // past the end: a value of its own
    }
    __syncthreads();
    const uint32_t lane = threadIdx.x % 32;
    uint16_t* mine = sh.counter + threadIdx.x / 32 * sh.bins;
    uint32_t* mask = sh.mask + threadIdx.x / 32 * sh.bins;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t e = expert[i];
        if (__all_sync(0xFFFFFFFFu, e == sh.bins)) break;  // the run ended (the ranks of the rest are not used)
        const bool real = e < sh.bins;
        uint32_t peers = 0xFFFFFFFFu;
        if constexpr (MASKS) {
            if (real) atomicOr(mask + e, 1u << lane);
            __syncwarp();
            peers = real ? mask[e] : 0u;
        } else {
#pragma unroll
            for (int b = 0; b < 11; ++b) {  // of the largest number ranked, at most RS_EXPERTS_MAX + 1
                const bool bit = e & (1u << b);
                const uint32_t set = __ballot_sync(0xFFFFFFFFu, bit);
                peers &= bit ? set : ~set;
            }
        }
        const uint32_t earlier = __popc(peers & ((1u << lane) - 1));
        const uint32_t before = real ? mine[e] : 0u;
        __syncwarp();
        if (real && earlier == 0) {
            mine[e] = (uint16_t)(before + __popc(peers));
            if constexpr (MASKS) mask[e] = 0;
        }
        __syncwarp();
        rank[i] = e << 16 | (before + earlier);
    }
    __syncthreads();
}

// Counters -> slots of the expert in earlier warps (below kTileSlots, so 16
// bits hold it); total[e] = the tile's count.
__device__ __forceinline__ void scan_warps(const Shared& sh)
{
    const uint32_t warps = blockDim.x / 32;
    for (uint32_t e = threadIdx.x; e < sh.bins; e += blockDim.x) {
        uint32_t at = 0;
#pragma unroll 8
        for (uint32_t w = 0; w < warps; ++w) {
            const uint32_t c = sh.counter[w * sh.bins + e];
            sh.counter[w * sh.bins + e] = (uint16_t)at;
            at += c;
        }
        sh.total[e] = at;
    }
    __syncthreads();
}

// out[e] = the sum of in[0 .. e), for all bins.
__device__ __forceinline__ void scan_bins(uint32_t bins, const uint32_t* in, uint32_t* out)
{
    __shared__ uint32_t warp_sum[kMaxThreads / 32];
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid % 32, warps = blockDim.x / 32;
    uint32_t carry = 0;
    for (uint32_t e0 = 0; e0 < bins; e0 += blockDim.x) {
        const uint32_t e = e0 + tid;
        const uint32_t c = e < bins ? in[e] : 0u;
        uint32_t inc = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, inc, d);
            if (lane >= d) inc += up;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        // every warp scans the warps' sums for itself
        uint32_t sums = lane < warps ? warp_sum[lane] : 0u;
        const uint32_t own = sums;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, sums, d);
            if (lane >= d) sums += up;
        }
        const uint32_t earlier = __shfl_sync(0xFFFFFFFFu, sums - own, warp);
        if (e < bins) out[e] = carry + earlier + inc - c;
        carry += __shfl_sync(0xFFFFFFFFu, sums, 31);
    }
    __syncthreads();
}

// Writes a ranked tile's positions and orders.  In a grid the orders go
// through shared memory: sorted[i] = expert << 16 | slot - begin, i the slot's
// place in the tile by expert.
__device__ __forceinline__ void place_tile(const SortParams& p, const Shared& sh, const Run& run, uint32_t begin,
                                           uint32_t len, const uint32_t (&rank)[kItems])
{
    const uint16_t* mine = sh.counter + threadIdx.x / 32 * sh.bins;
    const bool staged = gridDim.x > 1;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t s = run.first + 32 * i;
        if (s < run.end) {
            const uint32_t e = rank[i] >> 16, nth = mine[e] + (rank[i] & 0xFFFFu), at = sh.base[e] + nth;
            p.position[s] = (int32_t)at;
            if (staged) sh.sorted[sh.local[e] + nth] = e << 16 | (s - begin);
            else if (at < p.n) p.order[at] = (int32_t)s;
        }
    }
    if (!staged) return;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < len; i += blockDim.x) {
        const uint32_t v = sh.sorted[i], e = v >> 16;
        const uint32_t at = sh.base[e] + (i - sh.local[e]);
        if (at < p.n) p.order[at] = (int32_t)(begin + (v & 0xFFFFu));
    }
}

template <bool MASKS>
__global__ void __launch_bounds__(kMaxThreads) k_expert_sort(SortParams p)
{
    extern __shared__ uint32_t mem[];
    const uint32_t bins = p.experts + 1, tid = threadIdx.x;
    const bool grid = gridDim.x > 1;
    const Shared sh(mem, bins, grid, MASKS);
    const uint32_t begin = blockIdx.x * p.chunk, end = min(p.n, begin + p.chunk);  // begin < n by the grid's size
    uint32_t rank[kItems];

    // This block's counts; a chunk of one tile is ranked on the way.
    const bool one_tile = end - begin <= kTileSlots;
    const Run run(begin, min(end - begin, kTileSlots));
    if (one_tile) {
        rank_tile<MASKS>(p, sh, run, rank);
        scan_warps(sh);
    } else {
        for (uint32_t e = tid; e < bins; e += blockDim.x) sh.total[e] = 0;
        __syncthreads();
        for (uint32_t s = begin + tid; s < end; s += blockDim.x) atomicAdd(&sh.total[load_expert(p, s)], 1u);
        __syncthreads();
    }

    if (p.cluster) {
        auto cluster = cooperative_groups::this_cluster();
        scan_bins(bins, sh.total, sh.local);
        cluster.sync();
        uint32_t *sum = sh.sorted, *first = sh.sorted + bins;  // until the tile is placed
        for (uint32_t e = tid; e < bins; e += blockDim.x) {
            uint32_t all = 0, before = 0;
#pragma unroll
            for (uint32_t b = 0; b < kClusterBlocks; ++b) {
                const uint32_t c = b < gridDim.x ? *cluster.map_shared_rank(sh.total + e, b) : 0u;
                all += c;
                before += b < blockIdx.x ? c : 0u;
            }
            sum[e] = all;
            sh.base[e] = before;
        }
        __syncthreads();
        scan_bins(bins, sum, first);
        for (uint32_t e = tid; e < bins; e += blockDim.x) {
            if (blockIdx.x == 0) p.offsets[e] = (int32_t)first[e];
            sh.base[e] += first[e];
        }
        cluster.sync();  // every block has read the counts of the others
    } else if (grid) {
        // every block's counts -> the counts of the blocks before it, and the totals
        uint32_t* mine = p.counts + (size_t)blockIdx.x * bins;
        uint32_t* totals = p.counts + (size_t)gridDim.x * bins;
        for (uint32_t e = tid; e < bins; e += blockDim.x) mine[e] = sh.total[e];
        cooperative_groups::this_grid().sync();
        const uint32_t lane = tid % 32, warps = blockDim.x / 32;
        for (uint32_t e = blockIdx.x + gridDim.x * (tid / 32); e < bins; e += gridDim.x * warps) {
            uint32_t c[kMaxBlocks / 32], carry = 0;
#pragma unroll
            for (uint32_t i = 0; i < kMaxBlocks / 32; ++i) {
                const uint32_t b = i * 32 + lane;
                c[i] = b < gridDim.x ? __ldcg(p.counts + (size_t)b * bins + e) : 0u;
            }
#pragma unroll
            for (uint32_t i = 0; i < kMaxBlocks / 32; ++i) {
                if (i * 32 >= gridDim.x) break;
                uint32_t inc = c[i];
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, inc, d);
                    if (lane >= d) inc += up;
                }
                const uint32_t b = i * 32 + lane;
                if (b < gridDim.x) p.counts[(size_t)b * bins + e] = carry + inc - c[i];
                carry += __shfl_sync(0xFFFFFFFFu, inc, 31);
            }
            if (lane == 0) totals[e] = carry;
        }
        if (one_tile) scan_bins(bins, sh.total, sh.local);
        cooperative_groups::this_grid().sync();
        for (uint32_t e = tid; e < bins; e += blockDim.x) sh.total[e] = __ldcg(totals + e);
        __syncthreads();
        scan_bins(bins, sh.total, sh.base);
        for (uint32_t e = tid; e < bins; e += blockDim.x) {
            if (blockIdx.x == 0) p.offsets[e] = (int32_t)sh.base[e];
            sh.base[e] += __ldcg(mine + e);
        }
    } else {
        scan_bins(bins, sh.total, sh.base);
        for (uint32_t e = tid; e < bins; e += blockDim.x) p.offsets[e] = (int32_t)sh.base[e];
    }
    __syncthreads();

    if (one_tile) {
        place_tile(p, sh, run, begin, end - begin, rank);
        return;
    }
    for (uint32_t at = begin; at < end; at += kTileSlots) {
        const uint32_t len = min(end - at, kTileSlots);
        const Run r(at, len);
        rank_tile<MASKS>(p, sh, r, rank);
        scan_warps(sh);
        scan_bins(bins, sh.total, sh.local);
        place_tile(p, sh, r, at, len, rank);
        __syncthreads();
        for (uint32_t e = tid; e < bins; e += blockDim.x) sh.base[e] += sh.total[e];
        // (rank_tile's barriers come before the next use of base)
    }
}

}  // namespace

extern "C" {

size_t rs_expert_sort_temp_bytes(size_t n, int num_experts)
{
    if (n > RS_EXPERT_SLOTS_MAX || num_experts < 1 || num_experts > RS_EXPERTS_MAX) return (size_t)-1;
    if (n <= kClusterSlots) return 0;
    const size_t blocks = rsx::ceil_div(n, kChunkSlots);
    return rsx::align_up(((blocks < kMaxBlocks ? blocks : kMaxBlocks) + 1) * ((size_t)num_experts + 1) * 4, 256);
}

rs_status rs_expert_sort(const void* ids, int id_bytes, size_t n, int num_experts, int32_t* order,
                         int32_t* position, int32_t* offsets, void* temp, size_t temp_bytes, void* stream)
{
    const size_t need = rs_expert_sort_temp_bytes(n, num_experts);
    if (need == (size_t)-1 || (id_bytes != 4 && id_bytes != 8)) return RS_ERR_INVALID_ARG;
    if (!offsets || (uintptr_t)offsets % 4) return RS_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t bins = (size_t)num_experts + 1;
    if (n == 0) return cudaMemsetAsync(offsets, 0, bins * 4, s) == cudaSuccess ? RS_OK : RS_ERR_CUDA;
    if (!ids || !order || !position || (need && !temp)) return RS_ERR_INVALID_ARG;
    if ((uintptr_t)ids % id_bytes || (uintptr_t)order % 4 || (uintptr_t)position % 4 || (uintptr_t)temp % 256)
        return RS_ERR_INVALID_ARG;
    if (temp_bytes < need) return RS_ERR_TEMP_TOO_SMALL;
    const rsx::Range r[] = {{order, n * 4}, {position, n * 4}, {offsets, bins * 4}, {temp, need},
                            {ids, n * (size_t)id_bytes}};
    if (rsx::any_alias(r, 4, 5)) return RS_ERR_ALIAS;

    SortParams p{};
    p.ids = ids;
    p.id_bytes = id_bytes;
    p.n = (uint32_t)n;
    p.experts = (uint32_t)num_experts;
    p.order = order;
    p.position = position;
    p.offsets = offsets;
    p.counts = static_cast<uint32_t*>(temp);
    const bool masks = bins <= kMaskBins;
    const auto kernel = masks ? k_expert_sort<true> : k_expert_sort<false>;
    const size_t most_smem = Shared::bytes(bins, kMaxThreads / 32, n > kOneBlockSlots, masks);
    if (most_smem > 48 * 1024 - 256 &&
        !rsx::allow_smem(kernel, Shared::bytes(masks ? kMaskBins : RS_EXPERTS_MAX + 1, kMaxThreads / 32, true, masks)))
        return RS_ERR_CUDA;
    if (n <= kOneBlockSlots) {
        p.chunk = (uint32_t)n;
        const unsigned threads = (unsigned)(n < kMaxThreads ? rsx::align_up(n, 32) : kMaxThreads);
        kernel<<<1, threads, Shared::bytes(bins, threads / 32, false, masks), s>>>(p);
    } else if (n <= kClusterSlots) {
        p.chunk = (uint32_t)rsx::ceil_div(n, kClusterBlocks);
        p.cluster = true;
        const int threads = p.chunk < kMaxThreads ? (int)rsx::align_up(p.chunk, 32) : kMaxThreads;
        return rsx::launch_kernel(kernel, dim3(kClusterBlocks), threads,
                                  Shared::bytes(bins, threads / 32, true, masks), s, kClusterBlocks, false, p);
    } else {
        int dev = 0, sms = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
            return RS_ERR_CUDA;
        size_t blocks = rsx::ceil_div(n, kChunkSlots);
        if (blocks > (size_t)sms) blocks = sms;
        if (blocks > kMaxBlocks) blocks = kMaxBlocks;
        p.chunk = (uint32_t)rsx::ceil_div(n, blocks);
        blocks = rsx::ceil_div(n, p.chunk);
        void* args[] = {&p};
        if (cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kernel), dim3((unsigned)blocks),
                                        dim3(kMaxThreads), args, most_smem, s) != cudaSuccess) {
            cudaGetLastError();
            return RS_ERR_CUDA;
        }
    }
    return cudaGetLastError() == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

}  // extern "C"
