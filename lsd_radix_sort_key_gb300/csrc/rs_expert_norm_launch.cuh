// rs_expert_norm_launch.cuh -- the host side of rs_expert_norm.cuh: which
// kernel takes which width.  Included by one translation unit per type.
#pragma once

#include "rs_expert_norm.cuh"

namespace rsx {

inline unsigned norm_threads(size_t accesses, int v) { return (unsigned)align_up(ceil_div(accesses, v), 32); }

// Rows that fit 32 threads go to one warp each, 8 to a block, longer ones to a
// block each.  Accesses per thread: one where there are few rows, so that a row's
// loads are spread widest, else four (eight in a warp).
template <typename T>
rs_status norm_forward(const NormArgs<T>& p, bool vectors, cudaStream_t s)
{
    auto run = [&](auto kernel, size_t accesses, int v) {
        const unsigned x = norm_threads(accesses, v), y = x == 32 ? 8 : 1;
        kernel<<<(unsigned)ceil_div(p.rows, (size_t)y), dim3(x, y), 0, s>>>(p);
        return cudaGetLastError() == cudaSuccess ? RS_OK : RS_ERR_CUDA;
    };
    if (!vectors) {
        if (p.width <= 8192) return run(k_norm<T, 1, 8, 1024>, p.width, 8);
        return run(k_norm<T, 1, 16, 1024>, p.width, 16);
    }
    constexpr int N = kVec<T>;
    const size_t n = p.width / N;
    const bool few = p.rows <= 4 * 152;
    if (n <= 32 || (few && n <= 1024)) return run(k_norm<T, N, 1, 1024>, n, 1);
    if (n <= 64 || (few && n <= 2048)) return run(k_norm<T, N, 2, 1024>, n, 2);
    if (n <= 128 || (n > 256 && n <= 2048)) return run(k_norm<T, N, 4, 512>, n, 4);
    return run(k_norm<T, N, 8, 512>, n, 8);
}

template <typename T>
rs_status norm_gradient(const NormArgs<T>& p, bool vectors, uint32_t blocks, cudaStream_t s)
{
    auto run = [&](auto kernel, size_t accesses, int v) {
        return launch_kernel(kernel, dim3(blocks), dim3(norm_threads(accesses, v)), 0, s, 1, false, p);
    };
    constexpr int N = kVec<T>;
    const size_t n = p.width / N;
    rs_status st;
    if (!vectors) {
        if (p.width <= 2048) st = run(k_norm_grad<T, 1, 4, 512>, p.width, 4);
        else if (p.width <= 8192) st = run(k_norm_grad<T, 1, 16, 512>, p.width, 16);
        else st = run(k_norm_grad<T, 1, 16, 1024>, p.width, 16);
    } else if (n <= 512) {
        st = run(k_norm_grad<T, N, 1, 512>, n, 1);
    } else if (n <= 1024) {
        st = run(k_norm_grad<T, N, 2, 512>, n, 2);
    } else if constexpr (sizeof(T) == 4) {
        if (n <= 2048) st = run(k_norm_grad<T, N, 4, 512>, n, 4);
        else st = run(k_norm_grad<T, N, 4, 1024>, n, 4);
    } else {
        st = run(k_norm_grad<T, N, 2, 1024>, n, 2);
    }
    if (st != RS_OK || (!p.dweight && !p.dblock_weight && !p.dgate)) return st;
    const bool by_gate = p.gate_rows < blocks;
    const unsigned jobs = 2 + (p.dgate ? by_gate ? p.gate_rows : blocks - 1 : 0);
    return launch_kernel(k_norm_finish<T>, dim3((unsigned)ceil_div(p.width, kFinishCols), jobs), dim3(kFinishCols, kFinishRows),
                         0, s, 1, true, p, blocks, by_gate);
}

}  // namespace rsx
