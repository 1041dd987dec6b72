// rs_expert_f8_launch.cuh -- the host side of rs_expert_f8.cuh: tensor maps,
// the choice of a form, launches.  Included by one translation unit per type.
#pragma once

#include "rs_expert_f8.cuh"
#include "rs_expert_tc_launch.cuh"

namespace rsx {

template <typename T, bool PAIR, bool QUANT>
rs_status f8_launch(const F8Operands& o, const F8Args<T>& args, int sms, cudaStream_t s)
{
    using S = F8Shape<PAIR, QUANT>;
    const auto kernel = k_product_f8<T, PAIR, QUANT>;
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

// Pairs or single blocks, by a model of the time (us) as for the 16-bit products:
// a block's slices times the waves of tiles over the SMs, 0.33 per slice of a
// narrow tile, 0.34 of a pair's and 2 to start, and 0.38 where every block reads
// weights that nobody has read yet.
inline bool f8_pairs(size_t rows, size_t experts, size_t cols, size_t slices, int sms)
{
    if (cols <= 128) return false;
    // The offsets are on the device: with `owners` experts that can have rows,
    // half of them are taken to end in a partly filled tile.
    const size_t owners = rows < experts ? rows : experts;
    auto down = [&](size_t tile_rows) {
        const size_t t = rows / tile_rows + owners / 2;
        return t > owners ? t : owners;
    };
    auto time = [&](double slice, size_t tile_rows, size_t tile_cols, int at_once) {
        const size_t d = down(tile_rows);
        const double first = 0.38 * (double)owners / (double)d;
        return (slice > first ? slice : first) * (double)slices * (double)ceil_div(d * ceil_div(cols, tile_cols), at_once);
    };
    return time(0.34, 2 * kTcRows, 256, sms / 2) + 2.0 < time(0.33, kTcRows, 128, sms);
}

template <typename T, bool QUANT>
rs_status f8_run(const F8Operands& o, const F8Args<T>& args, cudaStream_t s)
{
    const int sms = sm_count();
    if (sms < 2) return RS_ERR_CUDA;
    const bool pair = f8_pairs(args.rows, args.experts, args.cols, ceil_div(args.reduce, kF8Depth), sms);
    return pair ? f8_launch<T, true, QUANT>(o, args, sms, s) : f8_launch<T, false, QUANT>(o, args, sms, s);
}

template <typename T>
rs_status f8_product(const F8Operands& o, const F8Args<T>& args, cudaStream_t s)
{
    return args.q ? f8_run<T, true>(o, args, s) : f8_run<T, false>(o, args, s);
}

}  // namespace rsx
