// rs_expert_sort.cu -- rs_expert_sort: the slots of a mixture-of-experts layer
// in stable order of their expert, the inverse of that order, and the
// experts' row ranges.
//
// This is one counting-sort pass on a digit of up to 1025 values (the experts
// and one more for dropped slots):
//     position(s) = base(e) + #{s' < s : expert(s') = e},  e = expert(s),
// base the exclusive scan of the experts' counts.  Slots are cut into chunks
// of kSlotsPerBlock in order; each chunk into one run of consecutive slots per
// warp.  Then #{s' < s, same expert} = slots of e in earlier chunks + in
// earlier warps of this chunk + in earlier slots of this warp, and
//   k_expert_count  counts every chunk's experts (integer counters in shared
//                   memory: their order does not matter),
//   k_expert_scan   scans each expert's chunk counts (one warp per expert),
//   k_expert_place  scans the experts' totals, ranks each warp's slots with
//                   __match_any_sync against its own counters, scans those
//                   over the warps and writes order and position.
#include "rs_expert_common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kItems = 16;  // slots per thread
constexpr int kSlotsPerBlock = kThreads * kItems;

struct SortParams {
    const void* ids;
    int id_bytes;
    uint32_t n;
    uint32_t experts;
    uint32_t blocks;
    int32_t* order;
    int32_t* position;
    int32_t* offsets;
    uint32_t* counts;  // [experts + 1][blocks]: first counts, then earlier chunks' sums
    uint32_t* totals;  // [experts + 1]
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

__global__ void __launch_bounds__(kThreads) k_expert_count(SortParams p)
{
    extern __shared__ uint32_t cnt[];
    const uint32_t bins = p.experts + 1;
    for (uint32_t e = threadIdx.x; e < bins; e += kThreads) cnt[e] = 0;
    __syncthreads();
    const uint32_t begin = blockIdx.x * kSlotsPerBlock;
    for (int i = 0; i < kItems; ++i) {
        const uint32_t s = begin + i * kThreads + threadIdx.x;
        if (s < p.n) atomicAdd(&cnt[load_expert(p, s)], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < bins; e += kThreads) p.counts[(size_t)e * p.blocks + blockIdx.x] = cnt[e];
}

__global__ void __launch_bounds__(kThreads) k_expert_scan(SortParams p)
{
    const uint32_t e = blockIdx.x * kWarps + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (e > p.experts) return;
    uint32_t* row = p.counts + (size_t)e * p.blocks;
    uint32_t carry = 0;
    for (uint32_t b0 = 0; b0 < p.blocks; b0 += 32) {
        const uint32_t b = b0 + lane;
        const uint32_t c = b < p.blocks ? row[b] : 0u;
        uint32_t inc = c;
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, inc, d);
            if (lane >= d) inc += up;
        }
        if (b < p.blocks) row[b] = carry + inc - c;
        carry += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
    if (lane == 0) p.totals[e] = carry;
}

__global__ void __launch_bounds__(kThreads) k_expert_place(SortParams p)
{
    // [bins] the first row of the chunk's slots of each expert, then [warps][bins] counters
    extern __shared__ uint32_t sm[];
    __shared__ uint32_t warp_sum[kWarps];
    const uint32_t bins = p.experts + 1, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    uint32_t* base = sm;
    uint32_t* mine = sm + bins + warp * bins;
    for (uint32_t e = tid; e < bins * kWarps; e += kThreads) sm[bins + e] = 0;

    // base = exclusive scan of the totals + this expert's slots in earlier chunks
    uint32_t carry = 0;
    for (uint32_t e0 = 0; e0 < bins; e0 += kThreads) {
        const uint32_t e = e0 + tid;
        const uint32_t c = e < bins ? p.totals[e] : 0u;
        uint32_t inc = c;
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, inc, d);
            if (lane >= d) inc += up;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        uint32_t before = carry, all = 0;
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? warp_sum[w] : 0u;
            all += warp_sum[w];
        }
        if (e < bins) {
            const uint32_t first = before + inc - c;
            base[e] = first + p.counts[(size_t)e * p.blocks + blockIdx.x];
            if (blockIdx.x == 0) p.offsets[e] = (int32_t)first;
        }
        carry += all;
    }
    __syncthreads();

    // rank among the warp's own earlier slots of the same expert
    const uint32_t begin = blockIdx.x * kSlotsPerBlock + warp * (32 * kItems) + lane;
    uint32_t packed[kItems];  // expert << 16 | rank; rank < 512
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t s = begin + i * 32;
        const uint32_t e = s < p.n ? load_expert(p, s) : bins;  // past the end: a value of its own
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, e);
        const uint32_t earlier = __popc(peers & ((1u << lane) - 1));
        uint32_t before = 0;
        if (e < bins) before = mine[e];
        __syncwarp();
        if (e < bins && earlier == 0) mine[e] = before + __popc(peers);
        __syncwarp();
        packed[i] = e << 16 | (before + earlier);
    }
    __syncthreads();
    // counters -> first row of each warp's slots
    for (uint32_t e = tid; e < bins; e += kThreads) {
        uint32_t at = base[e];
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t c = sm[bins + w * bins + e];
            sm[bins + w * bins + e] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t s = begin + i * 32;
        if (s < p.n) {
            const uint32_t at = mine[packed[i] >> 16] + (packed[i] & 0xFFFFu);
            p.position[s] = (int32_t)at;
            if (at < p.n) p.order[at] = (int32_t)s;
        }
    }
}

}  // namespace

extern "C" {

size_t rs_expert_sort_temp_bytes(size_t n, int num_experts)
{
    if (n > RS_EXPERT_SLOTS_MAX || num_experts < 1 || num_experts > RS_EXPERTS_MAX) return (size_t)-1;
    if (n == 0) return 0;
    const size_t bins = (size_t)num_experts + 1;
    return rsx::align_up((bins * rsx::ceil_div(n, kSlotsPerBlock) + bins) * 4, 256);
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
    if (!ids || !order || !position || !temp) return RS_ERR_INVALID_ARG;
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
    p.blocks = (uint32_t)rsx::ceil_div(n, kSlotsPerBlock);
    p.order = order;
    p.position = position;
    p.offsets = offsets;
    p.counts = static_cast<uint32_t*>(temp);
    p.totals = p.counts + bins * p.blocks;
    k_expert_count<<<p.blocks, kThreads, bins * 4, s>>>(p);
    k_expert_scan<<<(unsigned)rsx::ceil_div(bins, kWarps), kThreads, 0, s>>>(p);
    k_expert_place<<<p.blocks, kThreads, bins * 4 * (kWarps + 1), s>>>(p);
    return cudaGetLastError() == cudaSuccess ? RS_OK : RS_ERR_CUDA;
}

}  // extern "C"
