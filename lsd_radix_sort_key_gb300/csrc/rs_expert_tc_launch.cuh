// rs_expert_tc_launch.cuh -- the host side of rs_expert_tc.cuh: tensor maps
// and launches.  Included by one translation unit per element type.
#pragma once

#include "rs_expert_tc.cuh"

namespace rsx {

constexpr int kMaxDevices = 64;

// SMs of the current device; 0 on failure.
inline int sm_count()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

template <typename T, int BN, bool RAGGED_K, bool B_MN, bool PAIR, bool FEW = false>
rs_status tc_launch(const CUtensorMap& ma, const CUtensorMap& mb, const TcArgs<T>& args, size_t tiles, cudaStream_t s)
{
    const auto kernel = k_product_tc<T, BN, RAGGED_K, B_MN, PAIR, FEW>;
    const size_t smem = TcShape<BN, PAIR>::smem(args.experts);
    const int sms = sm_count();
    if (sms < 2) return RS_ERR_CUDA;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return RS_ERR_CUDA;
    size_t grid = (size_t)sms < kTcMaxBlocks ? (size_t)sms : kTcMaxBlocks;
    if constexpr (PAIR) grid = grid / 2 * 2 < tiles * 2 ? grid / 2 * 2 : tiles * 2;
    else grid = grid < tiles ? grid : tiles;
    return launch_kernel(kernel, dim3((unsigned)grid), kTcThreads, smem, s, PAIR ? 2 : 1, args.dependent != 0, ma, mb,
                         args);
}

// Up to this many rows per expert (on average) the weights' bytes bound the
// product, and 128-column tiles spread them more evenly over the SMs: 128 rows,
// 64 experts of 2048 x 2048 83.6 us against 86.6 with 256 columns, 64 rows of
// one expert of 4096 x 4096 21.1 against 29.2, 64 rows each of 128 experts of
// 1536 x 2048 143.5 against 147.3; at 256 rows each 224 against 203.
constexpr size_t kFewRows = 64;

// Pairs of blocks from this many rows per expert on (on average).
constexpr size_t kPairRows = 512;

template <typename T>
rs_status tc_ragged_rows(const TcOperand<T>& a, const TcOperand<T>& b, TcArgs<T> args, cudaStream_t stream)
{
    constexpr bool kBf16 = !__is_same(T, __half);
    const bool few = args.rows <= kFewRows * args.experts;
    const bool wide = args.cols > 128 && !few, pair = wide && args.rows >= kPairRows * args.experts;
    const uint64_t experts = b.expert_stride ? args.experts : 1;
    args.b_expert = b.expert_stride ? 1 : 0;
    CUtensorMap ma, mb;
    const uint64_t da[2] = {args.reduce, args.rows}, sa[1] = {(uint64_t)a.row_stride * 2};
    const uint64_t db[3] = {b.mn ? args.cols : args.reduce, b.mn ? args.reduce : args.cols, experts};
    const uint64_t sb[2] = {(uint64_t)b.row_stride * 2,
                            experts > 1 ? (uint64_t)b.expert_stride * 2 : (uint64_t)b.row_stride * 2};
    if (!rstc::encode_map(&ma, kBf16, 2, a.p, da, sa, few ? 16 : kTcRows) ||
        !rstc::encode_map(&mb, kBf16, 3, b.p, db, sb, b.mn ? 64 : wide && !pair ? 256 : 128))
        return RS_ERR_UNSUPPORTED;
    const size_t tiles =
        max_tiles(args.rows, args.experts, pair ? 2 * kTcRows : kTcRows) * ceil_div(args.cols, wide ? 256 : 128);
    if (pair)
        return b.mn ? tc_launch<T, 256, false, true, true>(ma, mb, args, tiles, stream)
                    : tc_launch<T, 256, false, false, true>(ma, mb, args, tiles, stream);
    if (wide)
        return b.mn ? tc_launch<T, 256, false, true, false>(ma, mb, args, tiles, stream)
                    : tc_launch<T, 256, false, false, false>(ma, mb, args, tiles, stream);
    if (few)
        return b.mn ? tc_launch<T, 128, false, true, false, true>(ma, mb, args, tiles, stream)
                    : tc_launch<T, 128, false, false, false, true>(ma, mb, args, tiles, stream);
    return b.mn ? tc_launch<T, 128, false, true, false>(ma, mb, args, tiles, stream)
                : tc_launch<T, 128, false, false, false>(ma, mb, args, tiles, stream);
}

template <typename T>
rs_status tc_ragged_reduce(const TcOperand<T>& a, const TcOperand<T>& b, TcArgs<T> args, cudaStream_t stream)
{
    constexpr bool kBf16 = !__is_same(T, __half);
    const bool wide = args.cols > 128, pair = wide && args.out_rows > 128;
    CUtensorMap ma, mb;
    const uint64_t da[2] = {args.out_rows, args.rows}, sa[1] = {(uint64_t)a.row_stride * 2};
    const uint64_t db[2] = {args.cols, args.rows}, sb[1] = {(uint64_t)b.row_stride * 2};
    if (!rstc::encode_map(&ma, kBf16, 2, a.p, da, sa, 64) || !rstc::encode_map(&mb, kBf16, 2, b.p, db, sb, 64))
        return RS_ERR_UNSUPPORTED;
    const size_t tiles =
        ceil_div(args.out_rows, pair ? 2 * kTcRows : kTcRows) * args.experts * ceil_div(args.cols, wide ? 256 : 128);
    if (pair) return tc_launch<T, 256, true, true, true>(ma, mb, args, tiles, stream);
    return wide ? tc_launch<T, 256, true, true, false>(ma, mb, args, tiles, stream)
                : tc_launch<T, 128, true, true, false>(ma, mb, args, tiles, stream);
}

}  // namespace rsx
