// rs_expert_f8.cuh -- the experts' products of rows and weights in 8 bits with
// block scales, on the tensor cores (definitions in rs_expert_block.h).
//
// D = A B^T, tiles of D per persistent block (128 x 128) or pair of blocks (PAIR:
// 256 x 256, a cluster of two on neighbouring SMs).  Scales are powers of two,
// which tcgen05.mma.kind::mxf8f6f4 applies itself to every 32 products that it
// adds, exactly, so the sums stay in one float32 accumulator in tensor memory
// and nothing is added up outside the tensor pipe.  (Each instruction's addition to
// it, of 32 products, cuts off below float32's last bit, where an adder in registers
// would round.)  Warp 0 copies 128-deep slices of A and B, one scale block each, into
// a ring of shared-memory stages (TMA, 128-byte swizzle); warp 3 gathers the scales of
// eight slices at a time, a 32-bit word for each four of a row, into a ring of its
// own; one thread of warp 1 has those of four slices at a time copied to tensor memory
// and issues the products; 16 epilogue warps read finished accumulators, apply the
// epilogue and store.
//
// Tensor memory (512 columns): two accumulators and two sets of scales.  A
// pair's accumulators are 256 columns each and there is room for 480: they
// overlap by 32 columns, which the epilogue reads first (`early`).
//
// What bounds it: the tensor pipe and, over a second, power.  8192^3 takes 297 us
// (3.7 PFLOP/s; 4.1 with neither copies nor scales), 32768 x 2048 x 4096 of 16 even
// groups in a short burst 168 us without an activation, 174 with gelu and 203 with the
// values before it kept; in longer runs, where power counts, 182, 188 and 217, and
// 226 with uneven groups.  Quantised results are bound by their epilogue: 16384 x
// 2048 x 2048 with silu 63 us.  A tile of 16 slices is 8200 cycles of the pipe and
// about 1300 until the next one's first instruction.  Copying A once for two pairs
// (multicast in clusters of four) changed nothing and left 8 SMs idle (36 such
// clusters fit).  Few rows are bound by the weights' way from device memory (128 rows,
// 64 experts of 2048 x 2048: 48 us, 5.6 TB/s).
#pragma once

#include "rs_expert_e4m3.cuh"
#include "rs_expert_tc.cuh"

namespace rsx {

constexpr int kF8Depth = 128;  // reduction elements per stage: one swizzled row of 128 bytes, one scale block

template <typename T>
struct F8Args {
    const int32_t* offsets;
    uint32_t experts, rows;
    uint32_t cols;    // of D
    uint32_t reduce;  // the reduction's length
    int act;          // rs_activation
    const uint8_t* a_scales;
    size_t a_scales_i;
    const uint8_t* b_scales;  // [experts][blocks of cols][blocks of reduce]
    const T* bias;
    size_t bias_e;
    const T* residual;
    size_t residual_i;
    T* d;
    size_t d_i;
    uint8_t* q;  // or D quantised
    size_t q_i;
    uint8_t* q_scales;
    size_t q_scales_i;
    T* pre;
    size_t pre_i;
    uint32_t* status;  // as in TcArgs
    uint32_t status_words;
    uint32_t stall;    // testing hook: tile stall - 1 is never copied
};

// 16 epilogue warps of 64 columns each: with 8 the epilogue was what lasted
// (32768 x 2048 x 4096 with gelu 250 us, 200 without an activation).
template <bool PAIR, bool QUANT>
struct F8Shape {
    static constexpr int kWarps = 16, kThreads = 32 * (kTcFirstEpilogueWarp + kWarps);
    // Columns of an epilogue warp, and whether half of the warps take every other
    // tile.  A single block's 128 columns go to all warps, 32 each, as few rows make
    // few tiles; half a scale block, 64, to each where the result is quantised.
    static constexpr uint32_t kWarpCols = PAIR || QUANT ? 64 : 32;
    static constexpr bool kTurns = !PAIR && QUANT;
    static constexpr uint32_t kReaders = PAIR ? 2 * kWarps : kTurns ? kWarps / 2 : kWarps;  // of an accumulator
    static constexpr uint32_t kCols = PAIR ? 256 : 128, kRows = PAIR ? 2 * kTcRows : kTcRows;  // of a tile
    static constexpr uint32_t kA = kTcRows * kF8Depth, kB = 128 * kF8Depth, kStage = kA + kB;   // of a block
    static constexpr int kStages = 6;
    static constexpr uint32_t kScales = 512 + kCols * 4;  // of four slices
    static constexpr uint32_t kScaleStage = 2 * kScales;  // of eight
    static constexpr int kScaleStages = 2;
    static constexpr uint32_t kStaging = 32 * 32;  // per epilogue warp: 32 rows of 16 elements
    static constexpr uint32_t kOverlap = PAIR ? 32 : 0;
    static constexpr uint32_t kAccStep = kCols - kOverlap;  // columns from one accumulator to the other
    static constexpr uint32_t kScaleCols = PAIR ? 480 : 256, kScaleStep = 16;
    static constexpr size_t smem(size_t experts)
    {
        return 1024 + (size_t)kStages * kStage + kScaleStages * kScaleStage + kWarps * kStaging +
               (2 * kStages + 2 * kScaleStages + 6) * 8 + 16 + Groups::words(experts) * 4;
    }
};

// Eight adjacent scales as two words: from the three aligned words around them, so
// that any base and stride will do, loaded in one go (load) before the first is
// looked at (get).  The words may hold other rows' scales, which are not used;
// those that do not lie wholly inside the scales, [begin, end), are read byte by
// byte.
struct Scales8 {
    uint32_t w[3];
    __device__ __forceinline__ static bool inside(uintptr_t a, const uint8_t* begin, const uint8_t* end)
    {
        return a >= (uintptr_t)begin && a + 4 <= (uintptr_t)end;
    }
    __device__ __forceinline__ void load(const uint8_t* from, const uint8_t* begin, const uint8_t* end)
    {
        const uintptr_t a = (uintptr_t)from & ~(uintptr_t)3;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            w[i] = 0;
            if (inside(a + 4 * i, begin, end)) w[i] = __ldg(reinterpret_cast<const uint32_t*>(a + 4 * i));
        }
    }
    __device__ __forceinline__ void get(uint32_t (&out)[2], const uint8_t* from, const uint8_t* begin, const uint8_t* end)
    {
        const uintptr_t a = (uintptr_t)from & ~(uintptr_t)3;
        if (!inside(a, begin, end) || !inside(a + 8, begin, end)) {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (!inside(a + 4 * i, begin, end))
                    for (int c = 0; c < 4; ++c) {
                        const uint8_t* at = reinterpret_cast<const uint8_t*>(a) + 4 * i + c;
                        if (at >= begin && at < end) w[i] |= (uint32_t)__ldg(at) << 8 * c;
                    }
        }
        const uint32_t bits = (uint32_t)((uintptr_t)from & 3) * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) out[i] = __funnelshift_r(w[i], w[i + 1], bits);
    }
};

// The epilogue's arithmetic on 16 values, two to an instruction (the same formulas
// as in rs_expert_groups.cuh): with gelu the issue slots are what lasts.
template <typename T>
__device__ __forceinline__ void add_pairs(uint32_t (&z)[16], const uint32_t (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = unpack2<T>(v[i]);
        const uint64_t sum = add2((uint64_t)z[2 * i + 1] << 32 | z[2 * i], pair_of(f.x, f.y));
        z[2 * i] = (uint32_t)sum;
        z[2 * i + 1] = (uint32_t)(sum >> 32);
    }
}

template <typename F>
__device__ __forceinline__ uint64_t both(F f, uint64_t v)
{
    return pair_of(f(__uint_as_float((uint32_t)v)), f(__uint_as_float((uint32_t)(v >> 32))));
}

template <int ACT>
__device__ __forceinline__ uint64_t activate_pair(uint64_t z)
{
    constexpr auto two = [](float c) { return pair_of(c, c); };
    if constexpr (ACT == RS_ACT_RELU) {
        return both(activate<RS_ACT_RELU, true>, z);
    } else if constexpr (ACT == RS_ACT_SILU) {
        const uint64_t e = both(fast_exp2, mul2(z, two(-kLog2e)));
        return mul2(z, both(fast_reciprocal, add2(e, two(1.0f))));
    } else {
        // z Phi(z) = max(z, 0) - |z| Phi(-|z|), so that no sign decides; `minus` is -|z|,
        // finite, as infinity times the zero of Phi would be NaN.
        const uint64_t minus = both([](float v) { return fmaxf(-fabsf(v), -3.402823466e38f); }, z);
        const uint64_t above = both([](float v) { return fmaxf(v, 0.0f); }, z);
        const uint64_t t = both(fast_reciprocal, fma2(two(-0.3275911f * 0.70710678118654752f), minus, two(1.0f)));
        const uint64_t e = both(fast_exp2, mul2(mul2(z, z), two(-0.5f * kLog2e)));
        uint64_t poly = fma2(t, two(0.5f * 1.061405429f), two(0.5f * -1.453152027f));
        poly = fma2(t, poly, two(0.5f * 1.421413741f));
        poly = fma2(t, poly, two(0.5f * -0.284496736f));
        poly = fma2(t, poly, two(0.5f * 0.254829592f));
        return fma2(minus, mul2(mul2(t, poly), e), above);
    }
}

template <int ACT>
__device__ __forceinline__ void activate_pairs(uint32_t (&z)[16])
{
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const uint64_t v = activate_pair<ACT>((uint64_t)z[i + 1] << 32 | z[i]);
        z[i] = (uint32_t)v;
        z[i + 1] = (uint32_t)(v >> 32);
    }
}

__device__ __forceinline__ void activate_pairs(uint32_t (&z)[16], int act)
{
    if (act == RS_ACT_RELU) activate_pairs<RS_ACT_RELU>(z);
    else if (act == RS_ACT_GELU) activate_pairs<RS_ACT_GELU>(z);
    else if (act == RS_ACT_SILU) activate_pairs<RS_ACT_SILU>(z);
}

// Activations of a result that is quantised from its float32 value, to float32's
// precision: with u = 2^-24, of the value,
//   silu  8 u + 1.25 |z| u: the form above.
//   gelu  16 u + 1.25 z^2 u.  (As above it is off by 1e-7 whatever the value, which
//         16 bits hide and a scale of the block's own does not.)  z Phi(z) as above with
//         Phi(-|z|) = t P(t) exp(-z^2 / 2), t = 1 / (1 + 0.305 |z|), and P of degree 7, a
//         minimax fit of the relative error for |z| to 14.5 (by Lawson's iteration; 6.5 u
//         as evaluated here).
// Half a step of z is |z| u and z^2 u of a value far below zero.  Where the exponential
// leaves the normal range, silu below -87 and gelu below -13, the scales still reach.
// 16384 x 2048 x 2048 takes 63 us with silu and 75 with gelu (61 and 70 by the forms
// above, 90 and 119 with the library's expf, erfcf and divisions).
__device__ __forceinline__ float exp2_below(float x)  // also below the normal range
{
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint64_t gelu_pair_float32(uint64_t z)
{
    constexpr auto two = [](float c) { return pair_of(c, c); };
    const uint64_t minus = both([](float v) { return fmaxf(-fabsf(v), -3.402823466e38f); }, z);
    const uint64_t above = both([](float v) { return fmaxf(v, 0.0f); }, z);
    const uint64_t t = both(fast_reciprocal, fma2(two(-0.305f), minus, two(1.0f)));
    const uint64_t e = both(exp2_below, mul2(mul2(z, z), two(-0.5f * kLog2e)));
    uint64_t poly = fma2(t, two(0.0366390459f), two(-0.152746767f));
    poly = fma2(t, poly, two(0.185315982f));
    poly = fma2(t, poly, two(-0.0376215354f));
    poly = fma2(t, poly, two(0.120840795f));
    poly = fma2(t, poly, two(0.103473589f));
    poly = fma2(t, poly, two(0.122458696f));
    poly = fma2(t, poly, two(0.121640243f));
    return fma2(minus, mul2(mul2(t, poly), e), above);
}

// silu where 1 + exp(z) is 1 and exp(-z) may be infinite, else as above.
__device__ __forceinline__ uint64_t silu_pair_below(uint64_t z)
{
    float v[2], y[2];
    unpair(z, v[0], v[1]);
    unpair(activate_pair<RS_ACT_SILU>(z), y[0], y[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (v[i] < -87.0f) y[i] = v[i] * exp2_below(v[i] * kLog2e);
    return pair_of(y[0], y[1]);
}

__device__ __forceinline__ void activate_float32(uint32_t (&z)[16], int act)  // by a whole warp
{
    if (act == RS_ACT_RELU) {
        activate_pairs<RS_ACT_RELU>(z);
    } else if (act == RS_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const uint64_t v = gelu_pair_float32((uint64_t)z[i + 1] << 32 | z[i]);
            z[i] = (uint32_t)v;
            z[i + 1] = (uint32_t)(v >> 32);
        }
    } else if (act == RS_ACT_SILU) {
        uint32_t most = 0;  // as bits the lowest of negative values is the largest
#pragma unroll
        for (int i = 0; i < 16; ++i) most = max(most, z[i]);
        if (__builtin_expect(__any_sync(0xFFFFFFFFu, most > __float_as_uint(-87.0f)), 0)) {
            // Seldom, so short: the pairs take turns in the first two places.  (Unrolled,
            // and with it all of the epilogue's code, 512 deep results took 2% longer.)
#pragma unroll 1
            for (int n = 0; n < 8; ++n) {
                const uint64_t v = silu_pair_below((uint64_t)z[1] << 32 | z[0]);
#pragma unroll
                for (int i = 0; i < 14; ++i) z[i] = z[i + 2];
                z[14] = (uint32_t)v;
                z[15] = (uint32_t)(v >> 32);
            }
        } else {
            activate_pairs<RS_ACT_SILU>(z);
        }
    }
}

// The larger of this lane's value and that of the same lane in the warp that has the
// other half of its columns.  mine, other: shared memory of the two warps, 32
// words each; both come here together (barrier `id`).
__device__ __forceinline__ uint32_t max_of_both(uint32_t v, uint32_t* mine, const uint32_t* other, uint32_t id)
{
    mine[threadIdx.x % 32] = v;
    rstc::meet_two_warps(id, true);
    v = max(v, other[threadIdx.x % 32]);
    rstc::meet_two_warps(id, true);  // both have read: the memory may be used again
    return v;
}

// The largest magnitude of 16 values (NaN, as bits above all others, if one is NaN).
__device__ __forceinline__ uint32_t largest16(const uint32_t (&z)[16])
{
    float most = 0.0f;
#pragma unroll
    for (uint32_t c = 0; c < 16; ++c)
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(fabsf(__uint_as_float(z[c]))));
    return __float_as_uint(most);
}

// The largest magnitude of the finite ones among 16 values.
__device__ __forceinline__ uint32_t largest_finite16(const uint32_t (&z)[16])
{
    uint32_t most = 0;
#pragma unroll
    for (uint32_t c = 0; c < 16; ++c) {
        const uint32_t m = z[c] & 0x7FFFFFFFu;
        most = max(most, m >= kNotFinite ? 0u : m);
    }
    return most;
}

// 16 values rounded to 8 bits.
__device__ __forceinline__ uint4 quantized16(const uint32_t (&z)[16], float inverse, bool all_finite)
{
    const uint64_t by = pair_of(inverse, inverse);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float f[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            f[c] = __uint_as_float(z[4 * k + c]);
            if (!all_finite) f[c] = finite_or_nan(f[c]);
        }
#pragma unroll
        for (int c = 0; c < 4; c += 2) unpair(mul2(pair_of(f[c], f[c + 1]), by), f[c], f[c + 1]);
        w[k] = to_e4m3x4(f[0], f[1], f[2], f[3]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A is rows of map_a, B is rows of map_b, expert e's from row e * cols; both
// have the reduction index adjacent.  QUANT: D leaves in 8 bits.  RESIDUAL: p.residual
// is added; a form of its own, as the registers that fetch it ahead keep the
// activations of one piece from overlapping (32768 x 512 x 4096 with gelu 152 us with
// them and 133 without).
template <typename T, bool PAIR, bool QUANT, bool RESIDUAL>
__global__ void __launch_bounds__((F8Shape<PAIR, QUANT>::kThreads), 1)
    k_product_f8(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, F8Args<T> p)
{
    using namespace rstc;
    using S = F8Shape<PAIR, QUANT>;
    constexpr uint32_t BN = S::kCols;
    extern __shared__ unsigned char raw[];
    unsigned char* ring = raw + (1024 - smem_addr(raw) % 1024) % 1024;  // stages are 1024-byte aligned
    unsigned char* scales = ring + S::kStages * S::kStage;
    unsigned char* staging = scales + S::kScaleStages * S::kScaleStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + S::kWarps * S::kStaging);
    uint64_t* empty = full + S::kStages;
    uint64_t* scales_full = empty + S::kStages;
    uint64_t* scales_empty = scales_full + S::kScaleStages;
    uint64_t* acc_full = scales_empty + S::kScaleStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* early = acc_empty + 2;  // what the next accumulator overlaps has been read
    uint32_t* slot = reinterpret_cast<uint32_t*>(early + 2);
    uint32_t* failed = slot + 1;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = PAIR ? cluster_rank() : 0, blocks = PAIR ? 2 : 1;
    const uint32_t first_tile = blockIdx.x / blocks, tile_step = gridDim.x / blocks;
    if (threadIdx.x == 32) {
        tma_prefetch(&map_a);
        tma_prefetch(&map_b);
        for (int s = 0; s < S::kStages; ++s) {
            bar_init(full + s, 1);   // the leader's: one arrival with the bytes of both blocks
            bar_init(empty + s, 1);  // each block's own
        }
        for (int s = 0; s < S::kScaleStages; ++s) {
            bar_init(scales_full + s, blocks);  // the leader's
            bar_init(scales_empty + s, 1);      // each block's own
        }
        for (int s = 0; s < 2; ++s) {
            bar_init(acc_full + s, 1);           // each block's own
            bar_init(acc_empty + s, S::kReaders);   // the leader's
            bar_init(early + s, S::kReaders);       // the leader's
        }
        bar_init_fence();
        *failed = 0;
    }
    if (warp == 2) tmem_alloc<PAIR>(slot, 512);
    tc_fence_before();
    // (the barrier inside make() orders all of the above)
    const Groups g = Groups::make(slot + 4, p.offsets, p.experts, p.rows, S::kRows, true);
    if constexpr (PAIR) cluster_sync();  // the other block's barriers are ready too
    tc_fence_after();
    const uint32_t tmem = *slot;
    const uint32_t across = (p.cols + BN - 1) / BN, tiles = g.tiles() * across;
    const uint32_t slices = (p.reduce + kF8Depth - 1) / kF8Depth;
    auto tile_at = [&](uint32_t tile) {
        TcTile t;
        const uint32_t down = tile / across;
        t.j0 = (tile - down * across) * BN;
        t.e = g.find(down);
        t.i0 = g.off[t.e] + (down - g.tile[t.e]) * S::kRows;
        t.i_end = g.off[t.e + 1];
        t.k0 = 0;
        t.k_end = t.e < p.experts ? p.reduce : 0;  // 0: the unused rows
        return t;
    };

    uint32_t issued = 0;  // stages filled so far (the copying warp)
    if (warp == 0) {
        uint32_t s = 0, round = 0;
        bool ok = true;
        for (uint32_t tile = first_tile; ok && tile < tiles; tile += tile_step) {
            const TcTile t = tile_at(tile);
            if (tile + 1 == p.stall) break;
            const int i0 = (int)(t.i0 + rank * kTcRows), w0 = (int)(t.e * p.cols + t.j0 + rank * 128);
            // Rows past the expert's end are not stored, so whole boxes of them are
            // not copied: what the stage held before stands in for them.
            const uint32_t rows = t.i_end - t.i0;  // of the tile, and more
            const uint32_t a_boxes = PAIR ? 1 : min((rows + 15) / 16, kTcRows / 16u);
            const bool second = PAIR && rows > kTcRows;  // the pair's second block has rows
            const uint32_t bytes = PAIR ? 2 * S::kB + (second ? 2 : 1) * S::kA : S::kB + a_boxes * 2048;
            for (uint32_t k = 0; k < t.k_end; k += kF8Depth, ++issued) {
                ok = bar_wait_warp(empty + s, (round & 1) ^ 1);
                if (!ok) break;
                unsigned char* a = ring + s * S::kStage;
                if (elect_one()) {
                    const uint32_t bar = PAIR ? cluster_addr(full + s, 0) : smem_addr(full + s);
                    if (rank == 0) bar_expect(full + s, bytes);
                    tma_load_2d<PAIR>(a + S::kA, &map_b, (int)k, w0, bar);
                    if constexpr (!PAIR) {
                        for (uint32_t i = 0; i < a_boxes; ++i)
                            tma_load_2d<PAIR>(a + i * 2048, &map_a, (int)k, i0 + (int)i * 16, bar);
                    } else if (rank == 0 || second) {
                        tma_load_2d<PAIR>(a, &map_a, (int)k, i0, bar);
                    }
                }
                __syncwarp();
                if (++s == S::kStages) s = 0, ++round;
            }
        }
        if (!ok) *failed = 1;
    } else if (warp == 3) {
        const uint32_t down = (p.cols + RS_QUANT_BLOCK - 1) / RS_QUANT_BLOCK;
        const uint8_t* a_end = p.a_scales + (p.rows - 1) * p.a_scales_i + slices;
        const uint8_t* b_end = p.b_scales + (size_t)p.experts * down * slices;
        uint32_t s = 0, round = 0;
        bool ok = true;
        for (uint32_t tile = first_tile; ok && tile < tiles; tile += tile_step) {
            const TcTile t = tile_at(tile);
            if (tile + 1 == p.stall) break;
            if (t.k_end == 0) continue;
            const uint8_t* a[4];
            const uint8_t* b[BN / 128];
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c)
                a[c] = p.a_scales + min(t.i0 + rank * kTcRows + c * 32 + lane, p.rows - 1) * p.a_scales_i;
#pragma unroll
            for (uint32_t h = 0; h < BN / 128; ++h)
                b[h] = p.b_scales + ((size_t)t.e * down + min(t.j0 / RS_QUANT_BLOCK + h, down - 1)) * slices;
            // The fences of a step wait for all that the warp has in flight, so loads for a
            // later step would only hold them up; the ring is two steps deep.
            for (uint32_t k = 0; k < slices; k += 8) {
                Scales8 ra[4], rb[BN / 128];
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) ra[c].load(a[c] + k, p.a_scales, a_end);
#pragma unroll
                for (uint32_t h = 0; h < BN / 128; ++h) rb[h].load(b[h] + k, p.b_scales, b_end);
                uint32_t wa[4][2], wb[BN / 128][2];
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) ra[c].get(wa[c], a[c] + k, p.a_scales, a_end);
#pragma unroll
                for (uint32_t h = 0; h < BN / 128; ++h) rb[h].get(wb[h], b[h] + k, p.b_scales, b_end);
                ok = bar_wait_warp(scales_empty + s, (round & 1) ^ 1);
                if (!ok) break;
                uint4* to = reinterpret_cast<uint4*>(scales + s * S::kScaleStage) + lane;
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i, to += S::kScales / 16) {
                    to[0] = make_uint4(wa[0][i], wa[1][i], wa[2][i], wa[3][i]);
#pragma unroll
                    for (uint32_t h = 0; h < BN / 128; ++h)
                        to[32 + 32 * h] = make_uint4(wb[h][i], wb[h][i], wb[h][i], wb[h][i]);
                }
                fence_async_shared();
                __syncwarp();
                if (elect_one()) {
                    if constexpr (PAIR) bar_arrive_cluster<true>(cluster_addr(scales_full + s, 0));
                    else bar_arrive(scales_full + s);
                }
                __syncwarp();
                if (++s == S::kScaleStages) s = 0, ++round;
            }
        }
        if (!ok) *failed = 1;
    } else if (warp == 1 && rank == 0) {
        // One thread alone: what a slice takes besides its matrix instructions has to
        // fit in their time (with votes and elections of the whole warp 630 cycles
        // per slice, whose instructions take 512).
        if (elect_one()) {
            constexpr uint32_t kDesc = mma_scaled_desc(S::kRows, BN);
            const uint64_t desc_a = smem_desc(smem_addr(ring), 16), desc_b = smem_desc(smem_addr(ring) + S::kA, 16);
            const uint64_t desc_s = scales_desc(smem_addr(scales));
            uint32_t s = 0, round = 0, n = 0, ss = 0, scale_round = 0, set = 0;
            bool ok = true;
            auto wait_for = [](uint64_t* bar, uint32_t parity) {
                return PAIR ? bar_wait_cluster(bar, parity) : bar_wait(bar, parity);
            };
            for (uint32_t tile = first_tile; ok && tile < tiles; tile += tile_step) {
                const TcTile t = tile_at(tile);
                if (t.k_end == 0) continue;
                const uint32_t h = n & 1, acc = tmem + h * S::kAccStep;
                for (uint32_t i = 0; i < slices; ++i) {
                    if (i % 8 == 0) {
                        ok = wait_for(scales_full + ss, scale_round & 1);
                        if (!ok) break;
                    }
                    if (i % 4 == 0) {
                        set ^= 1;
                        tc_fence_after();
#pragma unroll
                        for (uint32_t c = 0; c <= BN / 128; ++c)
                            tmem_copy_scales<PAIR>(tmem + S::kScaleCols + set * S::kScaleStep + c * 4,
                                                   desc_s + ((ss * S::kScaleStage + i / 4 % 2 * S::kScales + c * 512) >> 4));
                        if (i % 8 == 4 || i + 4 >= slices) {  // the last of this stage
                            mma_commit<PAIR>(scales_empty + ss);
                            if (++ss == S::kScaleStages) ss = 0, ++scale_round;
                        }
                    }
                    ok = bar_wait(full + s, round & 1);
                    if (!ok) break;
                    if (i == 0) {  // only now: all but the accumulator is there
                        ok = wait_for(acc_empty + h, ((n >> 1) & 1) ^ 1);
                        if (PAIR && ok && n) ok = wait_for(early + (h ^ 1), ((n - 1) >> 1) & 1);
                        if (!ok) break;
                        ++n;
                    }
                    const uint32_t steps = min((p.reduce - i * kF8Depth + 31) / 32, kF8Depth / 32u);
                    const uint32_t sa = tmem + S::kScaleCols + set * S::kScaleStep, desc = kDesc | mma_scale_byte(i % 4);
                    const uint64_t da = desc_a + s * (S::kStage >> 4), db = desc_b + s * (S::kStage >> 4);
                    tc_fence_after();
#pragma unroll
                    for (uint32_t k = 0; k < kF8Depth / 32; ++k)
                        if (k < steps) mma_e4m3_scaled<PAIR>(acc, da + k * 2, db + k * 2, desc, sa, sa + 4, i | k);
                    mma_commit<PAIR>(empty + s);
                    if (++s == S::kStages) s = 0, ++round;
                }
                if (ok) mma_commit<PAIR>(acc_full + h);
            }
            // What was issued is done before anything it uses is given up, also when
            // the epilogue's wait for it has run out.
            if (s || round) ok &= bar_wait(empty + (s ? s : S::kStages) - 1, (s ? round : round - 1) & 1);
            if (ss || scale_round)
                ok &= bar_wait(scales_empty + (ss ? ss : S::kScaleStages) - 1, (ss ? scale_round : scale_round - 1) & 1);
            if (!ok) *failed = 1;
        }
        __syncwarp();
    } else if (warp >= kTcFirstEpilogueWarp) {
        const uint32_t w = warp - kTcFirstEpilogueWarp, group = w / 4;
        const uint32_t quarter = warp % 4;  // the 32 tensor-memory lanes this warp can read
        uint4* stage = reinterpret_cast<uint4*>(staging + w * S::kStaging);
        const Rows<T> d(p.d, p.d_i, 0);
        const Rows<T> pre(p.pre, p.pre_i, 0);
        const Rows<const T> residual(p.residual, p.residual_i, 0);
        const bool vec_bias = ((uintptr_t)p.bias | p.bias_e * sizeof(T)) % 16 == 0;
        const bool q_sectors = ((uintptr_t)p.q | p.q_i) % 32 == 0;
        uint32_t n = 0, seen = 0;
        for (uint32_t tile = first_tile; tile < tiles; tile += tile_step, ++seen) {
            const TcTile t = tile_at(tile);
            const bool some = t.k_end != 0;
            const uint32_t h = n & 1, phase = (n >> 1) & 1;
            n += some;
            const uint32_t turn = some ? h : seen & 1;
            constexpr uint32_t W = S::kWarpCols, kOfTile = BN / W;  // groups that a tile takes
            if (S::kTurns && turn != group / kOfTile) continue;
            const uint32_t i0 = t.i0 + rank * kTcRows + quarter * 32, i = i0 + lane, c_first = group % kOfTile * W;
            const uint32_t j_first = t.j0 + c_first;
            const uint32_t acc = tmem + h * S::kAccStep + c_first + (quarter << 21);
            const uint32_t cols = j_first >= p.cols || i0 >= t.i_end ? 0 : min(W, p.cols - j_first);  // to be stored
            // this warp's part of the accumulator, or of what the next one overlaps, has been read
            auto release = [&](uint64_t* bar) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) bar_arrive_cluster<false>(cluster_addr(bar + h, 0));
                    else bar_arrive(bar + h);
                }
            };
            if constexpr (QUANT) {
                // A scale block's two warps go through every tile together.  The values
                // are gone through twice, first for the largest: two of a warp's four
                // pieces (those that a pair's next accumulator overlaps) wait in registers
                // and two in tensor memory.  With all four in registers some went to
                // local memory, whose path the operands of the matrix instructions fill:
                // 4000 cycles for the largest of 64 values.
                const uint32_t id = 1 + quarter + 4 * (group / 2);
                uint32_t* mine = reinterpret_cast<uint32_t*>(stage);
                const uint32_t* other = reinterpret_cast<const uint32_t*>(staging + (w ^ 4) * S::kStaging);
                const bool down = PAIR && h == 0;
                auto col = [&](uint32_t c) { return (down ? 3 - c : c) * 16; };
                uint32_t kept[2][16], z[16];
                if (some) {
                    if (!meet_two_warps(id, bar_wait_warp(acc_full + h, phase, 2 * slices))) {
                        *failed = 1;
                        break;
                    }
                    tc_fence_after();
                    if (cols) {
                        tmem_load16(kept[0], acc + col(0));
                        tmem_load16(kept[1], acc + col(1));
                        tmem_load_wait(kept[0]);
                        tmem_load_wait(kept[1]);
                    }
                    if constexpr (PAIR) release(early);
                }
                if (i0 >= t.i_end || j_first / RS_QUANT_BLOCK * RS_QUANT_BLOCK >= p.cols) {  // nothing for either warp
                    if (some) release(acc_empty);
                    continue;
                }
                // the epilogue of a piece; columns past the matrix count as zero
                auto finish = [&](uint32_t c, uint32_t (&v)[16]) {
                    if (col(c) >= cols || !some) {
#pragma unroll
                        for (uint32_t k = 0; k < 16; ++k) v[k] = 0;
                        if (col(c) >= cols) return;
                    }
                    const uint32_t j = j_first + col(c), left = cols - col(c);
                    if (p.bias && some) {
                        uint32_t bias[8];
                        load_bias<T>(bias, p.bias + t.e * p.bias_e + j, left, vec_bias);
                        add_pairs<T>(v, bias);
                    }
                    if (p.pre) {
                        uint32_t out[8];
                        round_all<T>(out, v);
                        store_piece<T>(stage, out, pre, i0, t.i_end, j, p.cols);
                    }
                    // (an activation of zero is zero)
                    activate_float32(v, p.act);
                    if (left < 16)
#pragma unroll
                        for (uint32_t k = 0; k < 16; ++k)
                            if (k >= left) v[k] = 0;
                };
                uint32_t most = 0;
#pragma unroll 1
                for (uint32_t c = 2; c < 4; ++c) {
                    if (some && cols) {
                        tmem_load16(z, acc + col(c));
                        tmem_load_wait(z);
                    }
                    finish(c, z);
                    most = max(most, largest16(z));
                    if (some && cols) tmem_store16(acc + col(c), z);
                }
#pragma unroll
                for (uint32_t c = 0; c < 2; ++c) {
                    finish(c, kept[c]);
                    most = max(most, largest16(kept[c]));
                }
                tmem_store_wait();
                most = max_of_both(most, mine, other, id);
                const bool all_finite = !__any_sync(0xFFFFFFFFu, most >= kNotFinite);
                auto again = [&](uint32_t c) {  // a piece from tensor memory
                    if (some && cols) {
                        tmem_load16(z, acc + col(c));
                        tmem_load_wait(z);
                    }
                };
                if (!all_finite) {
                    most = max(largest_finite16(kept[0]), largest_finite16(kept[1]));
#pragma unroll 1
                    for (uint32_t c = 2; c < 4; ++c) {
                        again(c);
                        most = max(most, largest_finite16(z));
                    }
                    most = max_of_both(most, mine, other, id);
                }
                const uint32_t byte = scale_byte(most);
                const float inverse = scale_inverse(byte);
                const bool live = i < t.i_end;
                // Two pieces are 32 adjacent bytes: one store where those are aligned.
                auto put = [&](const uint32_t (&v)[16], const uint4& before, uint32_t c) {
                    const uint4 q = quantized16(v, inverse, all_finite);
                    if (c % 2 == 0) return q;
                    uint8_t* to = p.q + i * p.q_i + j_first;
                    const uint4 lo = down ? q : before, hi = down ? before : q;
                    const uint32_t at = min(col(c), col(c - 1));
                    if (live && q_sectors && at + 16 < cols) {
                        const uint32_t both[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                        store_sector(to + at, both);
                    } else if (live) {
                        if (at < cols) *reinterpret_cast<uint4*>(to + at) = lo;
                        if (at + 16 < cols) *reinterpret_cast<uint4*>(to + at + 16) = hi;
                    }
                    return q;
                };
                uint4 q{};
#pragma unroll 1
                for (uint32_t c = 2; c < 4; ++c) {
                    again(c);
                    if (c == 3 && some) release(acc_empty);
                    q = put(z, q, c);
                }
                q = put(kept[0], q, 0);
                put(kept[1], q, 1);
                if (live && j_first % RS_QUANT_BLOCK == 0) p.q_scales[i * p.q_scales_i + j_first / RS_QUANT_BLOCK] = (uint8_t)byte;
            } else if (some) {
                // Two pieces of 16 columns at a time: one is on its way while the other is
                // finished.  A pair's first accumulator is read from its end, which the
                // second overlaps; both of its pieces there are loaded before anything
                // else is done, as the tensor pipe waits for them.
                const bool down = PAIR && h == 0;
                uint32_t z[2][16], add[2][8], bias[8];
                auto col = [&](uint32_t c) { return (down ? W / 16 - 1 - c : c) * 16; };
                auto fetch_residual = [&](uint32_t c, uint32_t (&r)[8]) {
                    if (RESIDUAL && c < W / 16 && col(c) < cols)
                        fetch_piece<T>(r, residual, i0, t.i_end, j_first + col(c), p.cols);
                };
                auto fetch_bias = [&](uint32_t c) {
                    if (p.bias && c < W / 16 && col(c) < cols)
                        load_bias<T>(bias, p.bias + t.e * p.bias_e + j_first + col(c), cols - col(c), vec_bias);
                };
                auto fetch_acc = [&](uint32_t c, uint32_t (&zz)[16]) {
                    if (c < W / 16 && col(c) < cols) tmem_load16(zz, acc + col(c));
                };
                static_assert(S::kOverlap <= 32, "two pieces");
                fetch_residual(0, add[0]);
                fetch_bias(0);
                if (!bar_wait_warp(acc_full + h, phase, 2 * slices)) {
                    *failed = 1;
                    break;
                }
                tc_fence_after();
                fetch_acc(0, z[0]);
                fetch_acc(1, z[1]);
                if constexpr (PAIR) {
                    tmem_load_wait(z[0]);
                    tmem_load_wait(z[1]);
                    release(early);
                }
#pragma unroll 1
                for (uint32_t c2 = 0; c2 < W / 16; c2 += 2)
#pragma unroll
                    for (uint32_t o = 0; o < 2; ++o) {
                        const uint32_t c = c2 + o, j = j_first + col(c);
                        uint32_t(&zz)[16] = z[o];
                        tmem_load_wait(zz);
                        if (c == W / 16 - 1) release(acc_empty);
                        if (p.bias && col(c) < cols) add_pairs<T>(zz, bias);
                        fetch_bias(c + 1);
                        fetch_residual(c + 1, add[o ^ 1]);
                        uint32_t out[8];
                        if (p.pre && col(c) < cols) {
                            round_all<T>(out, zz);
                            store_piece<T>(stage, out, pre, i0, t.i_end, j, p.cols);
                        }
                        activate_pairs(zz, p.act);
                        if (RESIDUAL && col(c) < cols) {
                            spread_piece<T>(stage, add[o], residual, j, p.cols);
                            add_pairs<T>(zz, add[o]);
                        }
                        round_all<T>(out, zz);
                        fetch_acc(c + 2, zz);
                        if (col(c) < cols) store_piece<T>(stage, out, d, i0, t.i_end, j, p.cols);
                    }
            } else {  // unused rows
                const uint32_t out[8] = {};
                for (uint32_t c = 0; c < cols; c += 16) {
                    if (p.pre) store_piece<T>(stage, out, pre, i0, t.i_end, j_first + c, p.cols);
                    store_piece<T>(stage, out, d, i0, t.i_end, j_first + c, p.cols);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();  // neither block's memory goes while the other's work may reach it
    tc_fence_after();
    if (threadIdx.x == 0) {
        if (*failed && rank == 0)  // a copy must not land in shared memory that its block no longer owns
            for (uint32_t s = 0; s < S::kStages && s < issued; ++s) {
                const uint32_t last = (issued - 1 - s) / S::kStages;
                bar_wait(full + s, last & 1);
            }
        p.status[blockIdx.x] = *failed;
    }
    if (blockIdx.x == 0)
        for (uint32_t i = gridDim.x + threadIdx.x; i < p.status_words; i += S::kThreads) p.status[i] = 0;
    __syncthreads();
    if constexpr (PAIR) cluster_sync();
    if (warp == 2) tmem_free<PAIR>(tmem, 512);
}

// x: rows x reduce, w: (experts * cols) x reduce, bytes; strides in bytes,
// multiples of 16, as the bases are.
struct F8Operands {
    const void* x;
    size_t x_stride;
    const void* w;
    size_t w_stride;
};

// Launches a product (the kernel by its sizes); RS_ERR_CUDA if the driver makes no
// tensor map.  Instantiated in rs_expert_f8_<type>.cu.
template <typename T>
rs_status f8_product(const F8Operands& o, const F8Args<T>& args, cudaStream_t stream);

}  // namespace rsx
