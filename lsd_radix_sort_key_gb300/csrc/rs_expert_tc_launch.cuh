// rs_expert_tc_launch.cuh -- the host side of rs_expert_tc.cuh: tensor maps
// and launches.  Included by one translation unit per element type.
#pragma once

#include <atomic>

#include "rs_expert_split.cuh"
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

template <typename T, int BN, bool RAGGED_K, bool B_MN, bool PAIR>
rs_status tc_launch(const CUtensorMap& ma, const CUtensorMap& mb, const TcArgs<T>& args, size_t tiles, cudaStream_t s)
{
    const auto kernel = k_product_tc<T, BN, RAGGED_K, B_MN, PAIR>;
    const size_t smem = TcShape<BN, PAIR>::smem(args.experts);
    const int sms = sm_count();
    if (sms < 2) return RS_ERR_CUDA;
    constexpr size_t most = TcShape<BN, PAIR>::smem(RS_EXPERTS_MAX);
    static_assert(most <= kBlockSmem);
    if (!allow_smem(kernel, most)) return RS_ERR_CUDA;
    size_t grid = (size_t)sms < kTcMaxBlocks ? (size_t)sms : kTcMaxBlocks;
    if constexpr (PAIR) grid = grid / 2 * 2 < tiles * 2 ? grid / 2 * 2 : tiles * 2;
    else grid = grid < tiles ? grid : tiles;
    return launch_kernel(kernel, dim3((unsigned)grid), kTcThreads, smem, s, PAIR ? 2 : 1, args.dependent != 0, ma, mb,
                         args);
}

template <typename T, bool RAGGED_K, bool B_MN>
rs_status split_launch(const CUtensorMap& ma, const CUtensorMap& mb, const TcArgs<T>& args, size_t tiles, int blocks,
                       int sms, cudaStream_t s)
{
    const auto kernel = k_product_split<T, RAGGED_K, B_MN>;
    const size_t smem = SplitShape::smem(args.experts);
    constexpr size_t most = SplitShape::smem(RS_EXPERTS_MAX);
    static_assert(most <= kBlockSmem);
    if (!allow_smem(kernel, most)) return RS_ERR_CUDA;
    size_t clusters = (size_t)(sms < kTcMaxBlocks ? sms : kTcMaxBlocks) / blocks;
    if (tiles < clusters) clusters = tiles;
    return launch_kernel(kernel, dim3((unsigned)(clusters * blocks)), kTcThreads, smem, s, blocks, args.dependent != 0,
                         ma, mb, args);
}

// Which kernel runs a product.  All tile the same work, so the choice is made
// by a model of the time: a block's slices of 64 times the waves of tiles over
// the SMs, in us,
//   narrow  128 x 128 tiles, one block each       0.27 per slice
//   wide    128 x 256, one block each             0.39 (shared memory bounds it)
//   pair    256 x 256, two blocks each            0.30, and 3 to start
//   split   128 x 128, 2, 4 or 8 blocks each, one wave only: 0.27 per slice of
//           a block, and 2.5 to join.
// but a slice that brings weights nobody has read yet takes as long as device
// memory needs for it when every SM asks at once, 0.38 per 128 columns (6.5 TB/s;
// 128 rows of 64 experts of 2048 x 2048: narrow 77, wide 87).
// The constants are a fit to timings on GB300 of 200 products (1 to 16 experts, 8
// to 2048 rows each, inner x outer from 512 x 2048 to 4096 x 4096) by every
// kernel: the choice was on average 2.5% above the best of them where they were
// fitted and 4.6% on another box, at worst 1.6 times.
// Some of them, narrow / wide / pair / split by 2 / 4 / 8, us:
//   1 expert,      8 rows, 4096 x 1024   18.0  22.1  23.6  13.0  10.0   8.7
//   1 expert,    128 rows, 4096 x 4096   23.4  23.6  25.3  17.4  13.4
//   1 expert,    400 rows, 2048 x 2048   14.4  15.4  16.7  13.1  20.4
//   8 experts,   100 rows, 2048 x 2048   15.0  18.3  18.1
//   8 experts,   128 rows, 2048 x 2048   24.6  16.4  18.3
//   4 experts,  2048 rows, 2048 x 2048   73.8  53.4  47.0
// (A split that needs a second wave is the 20.4: the others then do better.)
enum class Form { kNarrow, kWide, kPair, kSplit };

struct Choice {
    Form form;
    int blocks;  // kSplit
};

// Clusters of `blocks` of a split kernel that the device holds at once, with
// shared memory for any number of experts.
template <auto kernel>
size_t resident_clusters(int blocks)
{
    static std::atomic<int> known[kMaxDevices][4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    std::atomic<int>& n = known[dev][blocks == 2 ? 0 : blocks == 4 ? 1 : 2];
    int v = n.load(std::memory_order_relaxed);
    if (v == 0) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(kTcThreads);
        cfg.dynamicSmemBytes = SplitShape::smem(RS_EXPERTS_MAX);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)blocks;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (!allow_smem(kernel, cfg.dynamicSmemBytes)) return 0;
        if (cudaOccupancyMaxActiveClusters(&v, kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        n.store(v, std::memory_order_relaxed);
    }
    return (size_t)v;
}

// narrow, wide, pair: tiles of each form (expected); most: 128 x 128 tiles that
// there can be; slices: of the reduction; first, first_pair: the share of
// tiles that are the first to read their weights; clusters(c): resident
// clusters of c.
template <typename F>
Choice choose(size_t narrow, size_t wide, size_t pair, size_t most, size_t slices, double first, double first_pair,
              int sms, F clusters)
{
    const double n = (double)slices, memory = 0.38;
    auto larger = [](double a, double b) { return a > b ? a : b; };
    Choice best{Form::kNarrow, 1};
    double time = larger(0.27, memory * first) * n * (double)ceil_div(narrow, sms);
    auto offer = [&](Form form, int blocks, double t) {
        if (t < time) time = t, best = Choice{form, blocks};
    };
    if (wide) offer(Form::kWide, 1, larger(0.39, 2 * memory * first) * n * (double)ceil_div(wide, sms));
    if (pair) offer(Form::kPair, 2, larger(0.30, memory * first_pair) * n * (double)ceil_div(pair, sms / 2) + 3.0);
    for (int c = 2; c <= 8 && slices >= (size_t)(2 * c) && most * c <= (size_t)sms; c *= 2)
        if (most <= clusters(c)) offer(Form::kSplit, c, 0.27 * (double)ceil_div(slices, c) + 2.5);
    return best;
}

template <typename T>
rs_status tc_ragged_rows(const TcOperand<T>& a, const TcOperand<T>& b, TcArgs<T> args, cudaStream_t stream)
{
    constexpr bool kBf16 = !__is_same(T, __half);
    const int sms = sm_count();
    if (sms < 2) return RS_ERR_CUDA;
    const uint64_t experts = b.expert_stride ? args.experts : 1;
    args.b_expert = b.expert_stride ? 1 : 0;
    // The offsets are on the device: with `owners` experts that can have rows,
    // half of them are taken to end in a partly filled tile.
    const size_t owners = args.rows < args.experts ? args.rows : args.experts;
    auto down = [&](size_t tile_rows) {
        const size_t t = args.rows / tile_rows + owners / 2;
        return t > owners ? t : owners;
    };
    const size_t by128 = ceil_div(args.cols, 128), by256 = ceil_div(args.cols, 256);
    const Choice c = choose(down(kTcRows) * by128, args.cols > 128 ? down(kTcRows) * by256 : 0,
                            args.cols > 128 ? down(2 * kTcRows) * by256 : 0, (owners + args.rows / kTcRows) * by128,
                            ceil_div(args.reduce, kTcDepth), (double)owners / (double)down(kTcRows),
                            (double)owners / (double)down(2 * kTcRows), sms, [&](int n) {
                                return b.mn ? resident_clusters<k_product_split<T, false, true>>(n)
                                            : resident_clusters<k_product_split<T, false, false>>(n);
                            });
    const bool narrow = c.form == Form::kNarrow || c.form == Form::kSplit, pair = c.form == Form::kPair;
    CUtensorMap ma, mb;
    const uint64_t da[2] = {args.reduce, args.rows}, sa[1] = {(uint64_t)a.row_stride * 2};
    const uint64_t db[3] = {b.mn ? args.cols : args.reduce, b.mn ? args.reduce : args.cols, experts};
    const uint64_t sb[2] = {(uint64_t)b.row_stride * 2,
                            experts > 1 ? (uint64_t)b.expert_stride * 2 : (uint64_t)b.row_stride * 2};
    if (!rstc::encode_map(&ma, kBf16, 2, a.p, da, sa, narrow ? 16 : kTcRows) ||
        !rstc::encode_map(&mb, kBf16, 3, b.p, db, sb, b.mn ? 64 : narrow || pair ? 128 : 256))
        return RS_ERR_CUDA;
    const size_t tiles = max_tiles(args.rows, args.experts, pair ? 2 * kTcRows : kTcRows) * (narrow ? by128 : by256);
    switch (c.form) {
    case Form::kSplit:
        return b.mn ? split_launch<T, false, true>(ma, mb, args, tiles, c.blocks, sms, stream)
                    : split_launch<T, false, false>(ma, mb, args, tiles, c.blocks, sms, stream);
    case Form::kPair:
        return b.mn ? tc_launch<T, 256, false, true, true>(ma, mb, args, tiles, stream)
                    : tc_launch<T, 256, false, false, true>(ma, mb, args, tiles, stream);
    case Form::kWide:
        return b.mn ? tc_launch<T, 256, false, true, false>(ma, mb, args, tiles, stream)
                    : tc_launch<T, 256, false, false, false>(ma, mb, args, tiles, stream);
    default:
        return b.mn ? tc_launch<T, 128, false, true, false>(ma, mb, args, tiles, stream)
                    : tc_launch<T, 128, false, false, false>(ma, mb, args, tiles, stream);
    }
}

template <typename T>
rs_status tc_ragged_reduce(const TcOperand<T>& a, const TcOperand<T>& b, TcArgs<T> args, cudaStream_t stream)
{
    constexpr bool kBf16 = !__is_same(T, __half);
    const int sms = sm_count();
    if (sms < 2) return RS_ERR_CUDA;
    const size_t down = ceil_div(args.out_rows, kTcRows) * args.experts, by128 = ceil_div(args.cols, 128);
    const size_t by256 = ceil_div(args.cols, 256);
    const size_t down256 = ceil_div(args.out_rows, 2 * kTcRows) * args.experts;
    const bool wide = args.cols > 128;
    const Choice c = choose(down * by128, wide ? down * by256 : 0, wide && args.out_rows > 128 ? down256 * by256 : 0,
                            down * by128, ceil_div(args.rows, args.experts * (size_t)kTcDepth), 0.0, 0.0, sms, [&](int n) {
                                return resident_clusters<k_product_split<T, true, true>>(n);
                            });
    CUtensorMap ma, mb;
    const uint64_t da[2] = {args.out_rows, args.rows}, sa[1] = {(uint64_t)a.row_stride * 2};
    const uint64_t db[2] = {args.cols, args.rows}, sb[1] = {(uint64_t)b.row_stride * 2};
    if (!rstc::encode_map(&ma, kBf16, 2, a.p, da, sa, 64) || !rstc::encode_map(&mb, kBf16, 2, b.p, db, sb, 64))
        return RS_ERR_CUDA;
    switch (c.form) {
    case Form::kSplit: return split_launch<T, true, true>(ma, mb, args, down * by128, c.blocks, sms, stream);
    case Form::kPair: return tc_launch<T, 256, true, true, true>(ma, mb, args, down256 * by256, stream);
    case Form::kWide: return tc_launch<T, 256, true, true, false>(ma, mb, args, down * by256, stream);
    default: return tc_launch<T, 128, true, true, false>(ma, mb, args, down * by128, stream);
    }
}

}  // namespace rsx
