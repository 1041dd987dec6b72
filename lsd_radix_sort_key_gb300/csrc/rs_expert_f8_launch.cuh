// rs_expert_f8_launch.cuh -- the host side of rs_expert_f8.cuh: tensor maps,
// the choice of a form, launches.  Included by one translation unit per type.
#pragma once

#include "rs_expert_f8.cuh"
#include "rs_expert_tc_launch.cuh"

namespace rsx {

template <typename T, bool PAIR, bool QUANT, bool RESIDUAL>
rs_status f8_launch(const F8Operands& o, const F8Args<T>& args, int sms, cudaStream_t s)
{
    using S = F8Shape<PAIR, QUANT>;
    const auto kernel = k_product_f8<T, PAIR, QUANT, RESIDUAL>;
    constexpr size_t most = S::smem(RS_EXPERTS_MAX);
    static_assert(most <= kBlockSmem);
    if (!allow_smem(kernel, most)) return RS_ERR_CUDA;
    CUtensorMap ma, mb;
    const uint64_t da[2] = {args.reduce, args.rows}, sa[1] = {o.x_stride};
    const uint64_t db[2] = {args.reduce, (uint64_t)args.experts * args.cols}, sb[1] = {o.w_stride};
    if (!rstc::encode_tiles(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 2, o.x, da, sa, PAIR ? kTcRows : 16) ||
        !rstc::encode_tiles(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 2, o.w, db, sb, 128))
        return RS_ERR_CUDA;
    constexpr int blocks = PAIR ? 2 : 1;
    const size_t tiles = max_tiles(args.rows, args.experts, S::kRows) * ceil_div(args.cols, S::kCols);
    size_t clusters = (size_t)(sms < kTcMaxBlocks ? sms : kTcMaxBlocks) / blocks;
    if (tiles < clusters) clusters = tiles;
    return launch_kernel(kernel, dim3((unsigned)(clusters * blocks)), S::kThreads, S::smem(args.experts), s, blocks, false, ma,
                         mb, args);
}

// Pairs or single blocks, by a model of the time (us): the waves of tiles over the
// SMs, each of
//   narrow  0.31 per slice of 128, and 0.8
//   pair    0.27 per slice, and 2.6 (its epilogue is four times the work of a narrow
//           tile's); 2.5 once, to start and to end
// but 0.38 per slice where every block reads weights that nobody has read yet, as
// long as device memory needs when all SMs ask at once.  A fit to timings on GB300 of
// 1 to 16 experts with 8 to 2048 rows each, narrow / pair, us:
//   1 expert,    512 rows, 4096 x 4096   20.5   22.5
//   1 expert,   2048 rows, 4096 x 4096   51.2   34.8
//   8 experts, 3001 rows in all, 1000 x 1160   14.5   16.4
//   8 experts,  1000 rows, 1024 x 1024   22.5   20.5
//   16 experts, 2048 rows, 512 x 1024    38.9   34.8
//   16 experts, 2048 rows, 4096 x 4096    567    311
inline bool f8_pairs(size_t rows, size_t experts, size_t cols, size_t slices, int sms)
{
    if (cols <= 128) return false;
    // The offsets are on the device: with `owners` experts that can have rows,
    // half of them are taken to end in a partly filled tile.
    const size_t owners = rows < experts ? rows : experts;
    auto time = [&](double slice, double wave, size_t tile_rows, size_t tile_cols, int at_once) {
        const size_t t = rows / tile_rows + owners / 2, down = t > owners ? t : owners;
        const double first = 0.38 * (double)owners / (double)down;
        return ((slice > first ? slice : first) * (double)slices + wave) *
               (double)ceil_div(down * ceil_div(cols, tile_cols), at_once);
    };
    return time(0.27, 2.6, 2 * kTcRows, 256, sms / 2) + 2.5 < time(0.31, 0.8, kTcRows, 128, sms);
}

template <typename T, bool QUANT, bool RESIDUAL>
rs_status f8_run(const F8Operands& o, const F8Args<T>& args, cudaStream_t s)
{
    const int sms = sm_count();
    if (sms < 2) return RS_ERR_CUDA;
    const bool pair = f8_pairs(args.rows, args.experts, args.cols, ceil_div(args.reduce, kF8Depth), sms);
    return pair ? f8_launch<T, true, QUANT, RESIDUAL>(o, args, sms, s) : f8_launch<T, false, QUANT, RESIDUAL>(o, args, sms, s);
}

template <typename T>
rs_status f8_product(const F8Operands& o, const F8Args<T>& args, cudaStream_t s)
{
    return args.q ? f8_run<T, true, false>(o, args, s) : args.residual ? f8_run<T, false, true>(o, args, s) : f8_run<T, false, false>(o, args, s);
}

}  // namespace rsx
