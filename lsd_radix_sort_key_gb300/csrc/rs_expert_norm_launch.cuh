// rs_expert_norm_launch.cuh -- the host side of rs_expert_norm.cuh: which
// kernel takes which width.  Included by one translation unit per type.
#pragma once

#include "rs_expert_norm.cuh"

namespace rsx {

// Accesses per thread, and the most threads that a kernel is compiled for: one
// access each up to 512 threads, then two, then up to 1024 threads; single
// elements (rows that are only element-aligned) four, then sixteen.
template <typename T, typename F>
rs_status norm_shape(uint32_t width, bool vectors, F run)
{
    constexpr int N = kVec<T>;
    auto with = [&](auto n, auto v, auto threads) {
        const uint32_t accesses = width / decltype(n)::value;
        return run(n, v, threads, (unsigned)align_up(ceil_div(accesses, decltype(v)::value), 32));
    };
    if (!vectors) {
        if (width <= 2048) return with(Int<1>{}, Int<4>{}, Int<512>{});
        if (width <= 8192) return with(Int<1>{}, Int<16>{}, Int<512>{});
        return with(Int<1>{}, Int<16>{}, Int<1024>{});
    }
    if (width <= 256 * N) return with(Int<N>{}, Int<1>{}, Int<256>{});
    if (width <= 512 * N) return with(Int<N>{}, Int<1>{}, Int<512>{});
    if (width <= 1024 * N) return with(Int<N>{}, Int<2>{}, Int<512>{});
    if constexpr (sizeof(T) == 4) {
        if (width <= 2048 * N) return with(Int<N>{}, Int<4>{}, Int<512>{});
        return with(Int<N>{}, Int<4>{}, Int<1024>{});
    } else {
        return with(Int<N>{}, Int<2>{}, Int<1024>{});
    }
}

template <typename T>
rs_status norm_forward(const NormArgs<T>& p, bool vectors, cudaStream_t s)
{
    return norm_shape<T>(p.width, vectors, [&](auto n, auto v, auto most, unsigned threads) {
        constexpr int N = decltype(n)::value, V = decltype(v)::value, M = decltype(most)::value;
        // as many as an SM holds at once
        const size_t blocks = 152 * norm_blocks_per_sm(threads, V == 1 ? 1024 : N == 1 && V == 4 ? 768 : 512);
        const dim3 grid((unsigned)(p.rows < blocks ? p.rows : blocks));
        if (p.block) return launch_kernel(k_norm<T, N, V, M, true>, grid, dim3(threads), 0, s, 1, false, p);
        return launch_kernel(k_norm<T, N, V, M, false>, grid, dim3(threads), 0, s, 1, false, p);
    });
}

template <typename T>
rs_status norm_gradient(const NormArgs<T>& p, bool vectors, uint32_t blocks, cudaStream_t s)
{
    const rs_status st = norm_shape<T>(p.width, vectors, [&](auto n, auto v, auto most, unsigned threads) {
        constexpr int N = decltype(n)::value, V = decltype(v)::value, M = decltype(most)::value;
        if (p.block) return launch_kernel(k_norm_grad<T, N, V, M, true>, dim3(blocks), dim3(threads), 0, s, 1, false, p);
        return launch_kernel(k_norm_grad<T, N, V, M, false>, dim3(blocks), dim3(threads), 0, s, 1, false, p);
    });
    if (st != RS_OK || (!p.dweight && !p.dblock_weight && !p.dgate)) return st;
    const bool by_gate = p.gate_rows < blocks;
    const unsigned jobs = 2 + (p.dgate ? by_gate ? p.gate_rows : blocks - 1 : 0);
    return launch_kernel(k_norm_finish<T>, dim3((unsigned)ceil_div(p.width, kFinishCols), jobs), dim3(kFinishCols, kFinishRows),
                         0, s, 1, true, p, blocks, by_gate);
}

}  // namespace rsx
