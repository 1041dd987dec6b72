// rs_expert_norm_launch.cuh -- the host side of rs_expert_norm.cuh: which
// kernel takes which width.  Included by one translation unit per type.
#pragma once

#include "rs_expert_norm.cuh"

namespace rsx {

// Accesses per thread, the most threads that a kernel is compiled for and whether
// rows go through shared memory: one access each up to 512 threads, then two;
// rows past 16 KB two (or four) in up to 1024 threads, through registers; single
// elements (rows that are only element-aligned) four, then sixteen.
template <typename T, typename F>
rs_status norm_shape(uint32_t width, bool vectors, F run)
{
    constexpr int N = kVec<T>;
    auto with = [&](auto n, auto v, auto most, auto ring) {
        const uint32_t accesses = width / decltype(n)::value;
        return run(n, v, most, ring, (unsigned)align_up(ceil_div(accesses, decltype(v)::value), 32));
    };
    if (!vectors) {
        if (width <= 2048) return with(Int<1>{}, Int<4>{}, Int<512>{}, Int<0>{});
        if (width <= 8192) return with(Int<1>{}, Int<16>{}, Int<512>{}, Int<0>{});
        return with(Int<1>{}, Int<16>{}, Int<1024>{}, Int<0>{});
    }
    if (width <= 256 * N) return with(Int<N>{}, Int<1>{}, Int<256>{}, Int<1>{});
    if (width <= 512 * N) return with(Int<N>{}, Int<1>{}, Int<512>{}, Int<1>{});
    if constexpr (sizeof(T) == 4) {
        if (width <= 1024 * N) return with(Int<N>{}, Int<2>{}, Int<512>{}, Int<0>{});
        if (width <= 2048 * N) return with(Int<N>{}, Int<4>{}, Int<512>{}, Int<0>{});
        return with(Int<N>{}, Int<4>{}, Int<1024>{}, Int<0>{});
    } else {
        if (width <= 1024 * N) return with(Int<N>{}, Int<2>{}, Int<512>{}, Int<0>{});
        return with(Int<N>{}, Int<2>{}, Int<1024>{}, Int<0>{});
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
    return norm_shape<T>(p.width, vectors, [&](auto n, auto v, auto most, auto ring, unsigned threads) {
        constexpr int N = decltype(n)::value, V = decltype(v)::value, M = decltype(most)::value;
        constexpr int D = decltype(ring)::value ? kNormDepth : 0;
        // as many blocks as an SM holds at once
        const size_t of = V == 1 ? 1024 : N == 1 && V == 4 ? 768 : 512;
        const size_t per = threads > of ? 1 : of / threads < 16 ? of / threads : 16, blocks = p.rows < 152 * per ? p.rows : 152 * per;
        if (p.block)
            return norm_launch(k_norm<T, N, V, M, true, D>, blocks, threads, Feed<T, N, V, 2, D>::smem(threads), p, s);
        return norm_launch(k_norm<T, N, V, M, false, D>, blocks, threads, Feed<T, N, V, 1, D>::smem(threads), p, s);
    });
}

template <typename T>
rs_status norm_gradient(const NormArgs<T>& p, bool vectors, uint32_t blocks, cudaStream_t s)
{
    const rs_status st = norm_shape<T>(p.width, vectors, [&](auto n, auto v, auto most, auto ring, unsigned threads) {
        constexpr int N = decltype(n)::value, V = decltype(v)::value, M = decltype(most)::value;
        constexpr int D = decltype(ring)::value ? kGradDepth : 0;
        if (p.block)
            return norm_launch(k_norm_grad<T, N, V, M, true, D>, blocks, threads, Feed<T, N, V, 4, D>::smem(threads), p, s);
        return norm_launch(k_norm_grad<T, N, V, M, false, D>, blocks, threads, Feed<T, N, V, 3, D>::smem(threads), p, s);
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
