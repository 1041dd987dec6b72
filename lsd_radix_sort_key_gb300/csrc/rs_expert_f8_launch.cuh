// rs_expert_f8_launch.cuh -- the host side of rs_expert_f8.cuh: tensor maps,
// the choice of a form, launches.  Included by one translation unit per type.
#pragma once

#include "rs_expert_f8.cuh"
#include "rs_expert_tc_launch.cuh"

namespace rsx {

template <typename T, bool PAIR, bool QUANT>
rs_status f8_launch(const CUtensorMap& ma, const CUtensorMap& mb, const F8Args<T>& args, size_t tiles, int sms, cudaStream_t s)
{
    const auto kernel = k_product_f8<T, PAIR, QUANT>;
    constexpr size_t most = F8Shape<PAIR>::smem(RS_EXPERTS_MAX);
    static_assert(most <= kBlockSmem);
    if (!allow_smem(kernel, most)) return RS_ERR_CUDA;
    constexpr int blocks = PAIR ? 2 : 1;
    size_t clusters = (size_t)(sms < kTcMaxBlocks ? sms : kTcMaxBlocks) / blocks;
    if (tiles < clusters) clusters = tiles;
    return launch_kernel(kernel, dim3((unsigned)(clusters * blocks)), kF8Threads, F8Shape<PAIR>::smem(args.experts), s,
                         blocks, false, ma, mb, args);
}

template <typename T>
rs_status f8_product(const F8Operands& o, const F8Args<T>& args, cudaStream_t s)
{
    const int sms = sm_count();
    if (sms < 2) return RS_ERR_CUDA;
    const size_t owners = args.rows < args.experts ? args.rows : args.experts;
    auto down = [&](size_t tile_rows) {
        const size_t t = args.rows / tile_rows + owners / 2;
        return t > owners ? t : owners;
    };
    const size_t by128 = ceil_div(args.cols, 128), by256 = ceil_div(args.cols, 256);
    const Choice c = choose(down(kTcRows) * by128, 0, args.cols > 128 ? down(2 * kTcRows) * by256 : 0, 0,
                            ceil_div(args.reduce, kF8Depth), (double)owners / (double)down(kTcRows),
                            (double)owners / (double)down(2 * kTcRows), sms, [](int) { return (size_t)0; });
    const bool pair = c.form == Form::kPair;
    CUtensorMap ma, mb;
    const uint64_t da[2] = {args.reduce, args.rows}, sa[1] = {o.x_stride};
    const uint64_t db[2] = {args.reduce, (uint64_t)args.experts * args.cols}, sb[1] = {o.w_stride};
    if (!rstc::encode_tiles(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 2, o.x, da, sa, pair ? kTcRows : 16) ||
        !rstc::encode_tiles(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 2, o.w, db, sb, 128))
        return RS_ERR_CUDA;
    const size_t tiles = max_tiles(args.rows, args.experts, pair ? 2 * kTcRows : kTcRows) * (pair ? by256 : by128);
    if (pair)
        return args.q ? f8_launch<T, true, true>(ma, mb, args, tiles, sms, s)
                      : f8_launch<T, true, false>(ma, mb, args, tiles, sms, s);
    return args.q ? f8_launch<T, false, true>(ma, mb, args, tiles, sms, s)
                  : f8_launch<T, false, false>(ma, mb, args, tiles, sms, s);
}

}  // namespace rsx
