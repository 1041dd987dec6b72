// rs_expert_norm_launch.cuh -- the host side of rs_expert_norm.cuh: which
// kernel takes which width.  Included by one translation unit per type.
#pragma once

#include <type_traits>

#include "rs_expert_norm.cuh"

namespace rsx {

// The shape for a width: one vector per thread up to 512 threads, rows through
// shared memory, but two where a row has 65 to 256 of them (unless it is the
// forward call with a block): what a thread does once per row then counts for more
// elements (16384 x 2048 bf16: gradient 86 -> 73 us, norm alone 22.8 -> 20.7, but with a
// block 48 -> 50; rows of 256 33 -> 43 and more).  Past 512 vectors two (or four) of
// them in up to 1024 threads, through registers; strided elements up to 2048 four
// per thread with a block and eight without (a gradient of 4099 x 1037 float32 without a block 29 us with four
// and 20 with eight; with one, 16 bits, 51 and 79), else 16.
template <typename T, bool BLOCK, bool TWO, typename F>
rs_status norm_shape(uint32_t width, bool vectors, F run)
{
    constexpr int N = kVec<T>;
    auto with = [&](auto shape) {
        using S = decltype(shape);
        return run(shape, (unsigned)align_up(ceil_div(width, (size_t)S::N * S::V), 32));
    };
    if (!vectors) {
        using Short = std::conditional_t<BLOCK, NormShape<4, 1, 512, kRegisters, true>, NormShape<8, 1, 256, kRegisters, true>>;
        if (width <= 2048) return with(Short{});
        if (width <= 8192) return with(NormShape<4, 4, 512, kRegisters, true>{});
        return with(NormShape<4, 4, 1024, kRegisters, true>{});
    }
    if constexpr (TWO)
        if (width > 64 * N && width <= 256 * N) return with(NormShape<N, 2, 128, kOwn, false>{});
    if (width <= (TWO ? 64 : 256) * N) return with(NormShape<N, 1, 256, kOwn, false>{});
    if (width <= 512 * N) return with(NormShape<N, 1, 512, kOwn, false>{});
    if constexpr (sizeof(T) == 4) {
        if (width <= 1024 * N) return with(NormShape<N, 2, 512, kRegisters, false>{});
        if (width <= 2048 * N) return with(NormShape<N, 4, 512, kRegisters, false>{});
        return with(NormShape<N, 4, 1024, kRegisters, false>{});
    } else {
        if (width <= 1024 * N) return with(NormShape<N, 2, 512, kRegisters, false>{});
        return with(NormShape<N, 2, 1024, kRegisters, false>{});
    }
}

template <typename K, typename T>
rs_status norm_launch(K kernel, size_t blocks, unsigned threads, size_t smem, const NormArgs<T>& p, cudaStream_t s)
{
    constexpr size_t unasked = 48 * 1024 - 1024;  // beside the kernels' own
    if (smem > unasked && !allow_smem(kernel, kNormSmem)) return RS_ERR_CUDA;
    return launch_kernel(kernel, dim3((unsigned)blocks), dim3(threads), smem, s, 1, false, p);
}

template <typename T>
rs_status norm_forward(const NormArgs<T>& p, bool vectors, cudaStream_t s)
{
    auto launch = [&](auto block) {
        constexpr bool BLOCK = decltype(block)::value != 0;
        return norm_shape<T, BLOCK, !BLOCK>(p.width, vectors, [&](auto shape, unsigned threads) {
            using S = decltype(shape);
            // as many blocks as an SM holds at once
            const size_t of = S::V == 1 ? 1024 : S::THREADS == 128 ? 768 : 512, per = threads > of ? 1 : of / threads < 16 ? of / threads : 16;
            return norm_launch(k_norm<T, S, BLOCK>, p.rows < kSms * per ? p.rows : kSms * per, threads,
                               Feed<T, S, BLOCK ? 2 : 1>::smem(threads), p, s);
        });
    };
    return p.block ? launch(Int<1>{}) : launch(Int<0>{});
}

template <typename T>
rs_status norm_gradient(const NormArgs<T>& p, bool vectors, uint32_t blocks, cudaStream_t s)
{
    auto launch = [&](auto block) {
        constexpr bool BLOCK = decltype(block)::value != 0;
        return norm_shape<T, BLOCK, true>(p.width, vectors, [&](auto shape, unsigned threads) {
            using S = decltype(shape);
            return norm_launch(k_norm_grad<T, S, BLOCK>, blocks, threads, Feed<T, S, BLOCK ? 4 : 3>::smem(threads), p, s);
        });
    };
    const rs_status st = p.block ? launch(Int<1>{}) : launch(Int<0>{});
    if (st != RS_OK || (!p.dweight && !p.dblock_weight && !p.dgate)) return st;
    const bool by_gate = p.gate_rows < blocks;
    const unsigned jobs = 2 + (p.dgate ? by_gate ? p.gate_rows : blocks - 1 : 0);
    const dim3 threads(kFinishThreads, kFinishRows);
    auto finish = [&](auto kernel, int cols) {
        return launch_kernel(kernel, dim3((unsigned)ceil_div(p.width, (size_t)kFinishThreads * cols), jobs), threads, 0, s, 1, true, p,
                             blocks, by_gate);
    };
    return p.width % 4 == 0 ? finish(k_norm_finish<T, 4>, 4) : finish(k_norm_finish<T, 1>, 1);
}

}  // namespace rsx
