// rs_tc.cuh -- the tensor-core side of sm_103a in inline PTX: mbarriers with
// bounded waits, tiled bulk copies (TMA), tensor memory and tcgen05.mma, and
// the descriptors they take.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rstc {

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// One lane of the (converged) warp, the same one each time.  Code that only
// it runs still has warp-uniform operands, which the tensor and copy
// instructions take from uniform registers.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
}

// ---- mbarriers

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}

// Makes initialised barriers visible to the async proxy and the cluster.
__device__ __forceinline__ void bar_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }

__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void bar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// A wait gives up after this many SM clocks (about two seconds), short enough
// that a call with a fault still ends, and far longer than a working kernel
// waits for a copy, a free stage or another block.  A wait for a whole
// reduction has kSliceClocks more (4 us) for each of the reduction's 64-deep
// slices, which take 0.2 to 0.8 us: 2^30 rows in one tile take four seconds.
constexpr long long kWaitClocks = 1ll << 32, kSliceClocks = 1 << 13;

// The thread may sleep this long (ns) in one try.
constexpr uint32_t kTryNs = 1000000;

__device__ __forceinline__ bool bar_try(uint64_t* bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "r"(kTryNs)
        : "memory");
    return done != 0;
}

// Waits for phase `parity` of bar to complete, which may take as long as
// `slices` of a reduction; false if the time ran out.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, uint32_t slices = 0)
{
    if (bar_try(bar, parity)) return true;
    const long long start = clock64();
    while (clock64() - start < kWaitClocks + slices * kSliceClocks)
        if (bar_try(bar, parity)) return true;
    return false;
}

// The same for arrivals from the other block of a pair.
__device__ __forceinline__ bool bar_wait_cluster(uint64_t* bar, uint32_t parity, uint32_t slices = 0)
{
    const long long start = clock64();
    do {
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity), "r"(kTryNs)
            : "memory");
        if (done) return true;
    } while (clock64() - start < kWaitClocks + slices * kSliceClocks);
    return false;
}

// The same for a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool bar_wait_warp(uint64_t* bar, uint32_t parity, uint32_t slices = 0)
{
    return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, slices));
}

__device__ __forceinline__ bool bar_wait_cluster_warp(uint64_t* bar, uint32_t parity, uint32_t slices = 0)
{
    return __all_sync(0xFFFFFFFFu, bar_wait_cluster(bar, parity, slices));
}

// This thread's ordinary writes before later accesses of the async proxy
// (tensor cores, bulk copies), from either block of a pair.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// The same for writes to shared memory alone, which do not wait for the rest.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Two warps meet at barrier `id` (1 to 15): true if both bring true.
__device__ __forceinline__ bool meet_two_warps(uint32_t id, bool ok)
{
    uint32_t both;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.and.pred q, %1, 64, p;\n"
        " selp.u32 %0, 1, 0, q;\n}"
        : "=r"(both)
        : "r"(id), "r"((uint32_t)ok)
        : "memory");
    return both != 0;
}

// ---- clusters of blocks

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// The address, in the cluster's window, of `p` in block `rank`'s shared memory.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}

// An arrival on a barrier of any block of the cluster.  RELEASE: this thread's
// writes are visible to that block first, which waits for every store it has in
// flight; without, the arrival only says that what the thread waited for
// itself (loads from tensor memory) is done.
template <bool RELEASE>
__device__ __forceinline__ void bar_arrive_cluster(uint32_t cluster_bar)
{
    if constexpr (!RELEASE)
        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
    else
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void bar_expect_cluster(uint32_t cluster_bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_bar),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}

// ---- tiled copies into this block's shared memory, counted on bar.  PAIR:
// bar is an address in the cluster's window (the leader's barrier).

__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)map) : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
            "[%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
            "l"((uint64_t)map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
            "[%4];" ::"r"(smem_addr(dst)),
            "l"((uint64_t)map), "r"(x), "r"(y), "r"(bar)
            : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
            "[%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
            "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
            "%4}], [%5];" ::"r"(smem_addr(dst)),
            "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}

// ---- 32 bytes of global memory, 32-byte aligned: one sector in one access

__device__ __forceinline__ void load_sector(uint32_t (&r)[8], const void* p)
{
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
}

__device__ __forceinline__ void store_sector(void* p, const uint32_t (&r)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// ---- tensor memory

// One whole warp (PAIR: of each block of the pair); the address of `cols`
// columns (a power of two >= 32) lands in *slot (shared memory).
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols)
{
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}

template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols)
{
    if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 columns of this warp's 32 lanes: r[c] = column addr + c of lane laneid.
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t addr)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

// The loads so far are in their registers (which this names, so that no use of
// them moves ahead of the wait).
__device__ __forceinline__ void tmem_load_wait(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// The reverse of tmem_load16; tmem_store_wait before the columns are read again.
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---- the matrix instruction

// D (tensor memory, float32) = or += A B^T for K = 16 of 16-bit elements.
// PAIR: issued by the leader; each block holds half of A's rows, half of B's
// and half of D's rows.
template <bool PAIR>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
            : "memory");
}

// The same for K = 32 of e4m3 elements with a scale (a power of two, e8m0) for
// each row of A and of B: scales are in tensor memory, four to a 32-bit word, of
// which `idesc` names the byte.  Row 32 c + l of an operand has its word in
// column c of lane l, and again in the same columns 32, 64 and 96 lanes on.
// PAIR: each block has the scales of its own rows of A and of all rows of B.
template <bool PAIR>
__device__ __forceinline__ void mma_e4m3_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t scale_a,
                                                uint32_t scale_b, bool accumulate)
{
    if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(scale_a), "r"(scale_b)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(scale_a), "r"(scale_b)
            : "memory");
}

// Copies 32 rows of 16 bytes, 512 adjacent bytes of shared memory (scales_desc), to
// the four columns from `addr` of lanes 0..31 and of each 32 lanes after them.
// Matrix instructions that the thread issues later see them.  PAIR: issued by
// the leader; each block's tensor memory receives its own shared memory's.
template <bool PAIR>
__device__ __forceinline__ void tmem_copy_scales(uint32_t addr, uint64_t desc)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(addr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(addr), "l"(desc) : "memory");
}

// An arrival on bar (PAIR: on that barrier of both blocks) once every mma and
// copy to tensor memory that this thread issued so far is done.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint64_t* bar)
{
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_addr(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         smem_addr(bar))
                     : "memory");
}

// Instruction descriptor: float32 accumulator, A and B both binary16 or both
// bfloat16, each either with the reduction index adjacent in memory (K-major)
// or with the row index adjacent (MN-major); m x n tile.
__host__ __device__ constexpr uint32_t mma_desc(bool bf16, bool a_mn, bool b_mn, uint32_t m, uint32_t n)
{
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// The same for mma_e4m3_scaled, both operands K-major; `byte` of the scales' words.
__host__ __device__ constexpr uint32_t mma_scaled_desc(uint32_t m, uint32_t n)
{
    return ((n >> 3) << 17) | (1u << 23) | ((m >> 7) << 27);
}
__host__ __device__ constexpr uint32_t mma_scale_byte(uint32_t byte) { return (byte << 29) | (byte << 4); }

// Shared-memory operand descriptor for tiles copied with the 128-byte
// swizzle (rows of 128 bytes, groups of 8 rows = 1024 bytes, 1024-aligned).
//   K-major:  a row holds 64 reduction elements of one operand row; the next
//             8 operand rows are 1024 bytes on; a step of 16 in the reduction
//             is 32 bytes.
//   MN-major: a row holds 64 operand rows of one reduction index; the next 8
//             reduction indexes are 1024 bytes on, the next 64 operand rows
//             `mn_stride` bytes on; a step of 16 in the reduction is 2048.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t mn_stride)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((mn_stride >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// 512 bytes of scales, not swizzled: groups of 8 rows of 16 bytes, one after the
// other.
__device__ __forceinline__ uint64_t scales_desc(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(128u >> 4) << 32) | (1ull << 46);
}

// ---- host side

// cuTensorMapEncodeTiled through the runtime (no link dependency on the
// driver library); nullptr if there is none.
inline decltype(&cuTensorMapEncodeTiled) tensor_map_encoder()
{
    static const auto fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(p);
    }();
    return fn;
}

// A map with the 128-byte swizzle: dims[0] adjacent, strides (bytes) of dims
// 1.., boxes of 128 bytes x box1 (x 1).
inline bool encode_tiles(CUtensorMap* map, CUtensorMapDataType type, uint32_t elem_bytes, int rank, const void* base,
                         const uint64_t* dims, const uint64_t* strides, uint32_t box1)
{
    const auto encode = tensor_map_encoder();
    if (!encode) return false;
    cuuint64_t d[3], s[2];
    cuuint32_t box[3] = {128 / elem_bytes, box1, 1}, step[3] = {1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        if (dims[i] == 0 || dims[i] > 0xFFFFFFFFull) return false;
        d[i] = dims[i];
    }
    for (int i = 0; i + 1 < rank; ++i) {
        if (strides[i] == 0 || strides[i] % 16 || strides[i] >= (1ull << 40)) return false;
        s[i] = strides[i];
    }
    if ((uintptr_t)base % 16) return false;
    return encode(map, type, (cuuint32_t)rank, const_cast<void*>(base), d, s, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Of 16-bit elements.
inline bool encode_map(CUtensorMap* map, bool bf16, int rank, const void* base, const uint64_t* dims,
                       const uint64_t* strides, uint32_t box1)
{
    return encode_tiles(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, rank, base, dims,
                        strides, box1);
}

}  // namespace rstc
