// rs_expert_norm_launch.cuh -- the host side of rs_expert_norm.cuh: which
// kernel takes which width.  Included by one translation unit per type.
#pragma once

#include "rs_expert_norm.cuh"

namespace rsx {

// The shape for a width: one vector per thread up to 512 threads, rows through
// shared memory; past 512 vectors two (or four) of them in up to 1024 threads,
// through registers; strided elements, eight per thread through shared memory up
// to 2048, else 16 through registers.
template <typename T, typename F>
rs_status norm_shape(uint32_t width, bool vectors, F run)
{
    constexpr int N = kVec<T>;
    auto with = [&](auto shape) {
        using S = decltype(shape);
        return run(shape, (unsigned)align_up(ceil_div(width, (size_t)S::N * S::V), 32));
    };
    if (!vectors) {
        if (width <= 2048) return with(NormShape<8, 1, 256, kShared, true>{});
        if (width <= 8192) return with(NormShape<4, 4, 512, kRegisters, true>{});
        return with(NormShape<4, 4, 1024, kRegisters, true>{});
    }
    if (width <= 256 * N) return with(NormShape<N, 1, 256, kOwn, false>{});
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
    return norm_shape<T>(p.width, vectors, [&](auto shape, unsigned threads) {
        using S = decltype(shape);
        // as many blocks as an SM holds at once
        const size_t of = S::V == 1 ? 1024 : 512, per = threads > of ? 1 : of / threads < 16 ? of / threads : 16;
        const size_t blocks = p.rows < 152 * per ? p.rows : 152 * per;
        if (p.block)
            return norm_launch(k_norm<T, S, true>, blocks, threads, Feed<T, S, 2>::smem(p.width, threads), p, s);
        return norm_launch(k_norm<T, S, false>, blocks, threads, Feed<T, S, 1>::smem(p.width, threads), p, s);
    });
}

template <typename T>
rs_status norm_gradient(const NormArgs<T>& p, bool vectors, uint32_t blocks, cudaStream_t s)
{
    const rs_status st = norm_shape<T>(p.width, vectors, [&](auto shape, unsigned threads) {
        using S = decltype(shape);
        if (p.block)
            return norm_launch(k_norm_grad<T, S, true>, blocks, threads, Feed<T, S, 4>::smem(p.width, threads), p, s);
        return norm_launch(k_norm_grad<T, S, false>, blocks, threads, Feed<T, S, 3>::smem(p.width, threads), p, s);
    });
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
