/*
 * rs_expert_block.h -- C ABI of an expert block in 8 bits for NVIDIA GB300
 * (sm_103a): rows and weights quantised in blocks of 128, the experts'
 * products of them, and the norms around the block with their gradients.  It
 * goes with rs_experts.h, whose conventions hold here too (plans, strides in
 * elements, dropped slots and unused rows, aliasing, streams, capture).
 *
 * Quantised values.  A value is an 8-bit float (e4m3: 4 exponent bits, 3
 * mantissa bits, no infinities) times a scale shared by 128 values of a row,
 * or by 128 x 128 of a weight matrix (the last block of a row or matrix may
 * be smaller).  A scale is a power of two, held as its exponent in one byte
 * (e8m0: 2^(byte - 127)): the smallest from 2^-126 on with which no value of
 * the block passes 448; 1 for a block without a nonzero finite value.  So a
 * quantised value is q = round(x / scale), to nearest, ties to even; the
 * division is exact and the rounding the only one.  An infinity or NaN
 * becomes NaN and does not count for its block's scale.
 *
 *   rs_expert_quantize             rows x[r] -> q[r], scales[r][i / 128]
 *   rs_expert_dispatch_quantized   the same rows laid out by expert:
 *                                  q[position[s]], scales[position[s]] of x[t]
 *   rs_expert_quantize_weights     w[e] -> q[e], scales[e][n / 128][k / 128]
 *   rs_expert_matmul_quantized     y[r] = act(x[r] w[e]^T + bias[e]) + residual[r]
 *   rs_expert_norm                 h = rms(x) weight, or
 *                                  y = residual_scale x + gate (rms(block) block_weight),
 *                                  h = rms(y) weight
 *   rs_expert_norm_grad            its gradients
 * with rms(v) = v / sqrt(mean(v^2) + eps) over a row.
 */
#ifndef RS_EXPERT_BLOCK_H
#define RS_EXPERT_BLOCK_H

#include "rs_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Values of a row that share a scale. */
#define RS_QUANT_BLOCK 128

/*
 * The quantisers.  x, w: float32, binary16 or bfloat16.  Quantised rows start
 * on 16 bytes (base and q_stride multiples of 16): what lies between a row's
 * width and the next multiple of 16 is set to zero.  scales: one byte per
 * block, ceil(width / 128) per row, row stride scales_stride bytes (>= that).
 *
 * rs_expert_dispatch_quantized takes a plan as rs_expert_dispatch does; the
 * rows of dropped slots are zero with scales of one.
 *
 * rs_expert_quantize_weights: element (e, n, k) of w at e*w_expert_stride +
 * n*w_outer_stride + k*w_inner_stride; one of the last two is 1 (the other
 * side's stride at least the adjacent side's length) unless outer or inner is
 * 1.  Output row (e, n) at q + (e*outer + n)*q_stride; scales contiguous
 * [num_experts][ceil(outer / 128)][ceil(inner / 128)].  Quantising the same
 * memory with outer and inner exchanged gives the transposed weights, with
 * the transposed scales, that the gradient of x takes.
 *
 * Nothing to write (rows, tokens, width, outer or inner 0): RS_OK.  Sizes:
 * rows <= RS_EXPERT_SLOTS_MAX, width, outer, inner <= RS_EXPERT_WIDTH_MAX,
 * num_experts <= RS_EXPERTS_MAX, fewer than 2^32 blocks of rows (tokens, for
 * a dispatch) and 2^31 of weights.
 */
rs_status rs_expert_quantize(rs_float_type type, const void* x, size_t x_stride, size_t rows, size_t width, void* q,
                             size_t q_stride, void* scales, size_t scales_stride, void* stream);
rs_status rs_expert_dispatch_quantized(rs_float_type type, const void* x, size_t x_stride, const int32_t* position,
                                       const int32_t* routed, size_t tokens, int slots, size_t width, void* q,
                                       size_t q_stride, void* scales, size_t scales_stride, void* stream);
rs_status rs_expert_quantize_weights(rs_float_type type, const void* w, size_t w_expert_stride, size_t w_outer_stride,
                                     size_t w_inner_stride, int num_experts, size_t outer, size_t inner, void* q,
                                     size_t q_stride, void* scales, void* stream);

/*
 * The experts' products of quantised rows and weights, on the tensor cores
 * with float32 sums (which cut off below the last bit once for every 32
 * products).  x: rows x inner, 16-byte aligned rows (base and
 * x_stride); w: row (e, n) at w + (e*outer + n)*w_stride, 16-byte aligned;
 * scales as the quantisers write them, x's with a row stride.  bias,
 * residual, y and pre are of `type`, binary16 or bfloat16, with any stride >=
 * outer (bias and residual: or 0), as in rs_expert_matmul.
 *
 * Either y (outer values per row), or q and q_scales (y quantised, from its
 * float32 values; rows as rs_expert_quantize writes them; no residual) is
 * given, and pre if the values before the activation are wanted.  inner >= 1.
 * Activations of results in 16 bits are as in rs_expert_matmul; of quantised
 * ones they are off by a few units of float32's last place (silu 8 + 1.25 |z|,
 * gelu 16 + 1.25 z^2 times 2^-24 of the value, z being the sum plus bias).
 * The exponents of two blocks that meet in a product may add up to anything a
 * float32 holds; a scale byte of 255 is NaN.
 *
 * temp: 256-byte aligned, rs_expert_matmul_quantized_temp_bytes bytes;
 * rs_expert_matmul_status reads it.
 */
typedef struct rs_expert_matmul_quantized_desc {
    rs_float_type type; /* of y, bias, residual and pre */
    rs_activation activation;
    int num_experts;
    size_t rows;
    size_t inner;
    size_t outer;
    const int32_t* offsets; /* num_experts + 1, on the device */
    const void* x;
    size_t x_stride;
    const void* x_scales;
    size_t x_scales_stride;
    const void* w;
    size_t w_stride;
    const void* w_scales;
    const void* bias;
    size_t bias_stride;
    const void* residual;
    size_t residual_stride;
    void* y;
    size_t y_stride;
    void* q;
    size_t q_stride;
    void* q_scales;
    size_t q_scales_stride;
    void* pre;
    size_t pre_stride;
    void* temp;
    size_t temp_bytes;
    void* stream;
    /* Testing hook, 0 in normal use: t + 1 makes the kernel never copy the
     * operands of output tile t, so the waits for them run out. */
    int32_t stall_tile;
} rs_expert_matmul_quantized_desc;

size_t rs_expert_matmul_quantized_temp_bytes(const rs_expert_matmul_quantized_desc* desc);
rs_status rs_expert_matmul_quantized(const rs_expert_matmul_quantized_desc* desc);

/* Largest width of a normed row. */
#define RS_EXPERT_NORM_WIDTH_MAX 16384

/*
 * The norms around a block.  x, block, y, h and their gradients: rows x width
 * of `type`; weight, block_weight and gate: of param_type, which is `type` or
 * float32, width adjacent values each.  gate_rows: 0 no gate; 1 one gate row
 * for all; G one for each rows / G rows (rows a multiple of G), row g at gate +
 * g * width.
 *
 * Forward.  block == NULL: h = rms(x) weight (y, block_weight, gate unused).
 * Else y = residual_scale x + gate u, u = block_weight ? rms(block)
 * block_weight : block, and, if weight is not NULL, h = rms(y) weight, where y
 * is taken as it is held, after its rounding.  Sums are float32, so the squares
 * of a row have to add up inside its range (magnitudes of about 1e-18 to 1e17).
 *
 * Gradient.  Reads y (block == NULL: x itself, in `x`; else the forward's y,
 * in `x`), dh (NULL only if weight is) and dy, the gradient that reaches y by
 * another way (NULL: none), and writes the ones of dx, dweight, dblock,
 * dblock_weight, dgate that are not NULL; with d = dy + the gradient of the
 * second norm, dx = residual_scale d, dgate = the sum of d u over its rows, and
 * so on.  dweight, dblock_weight and dgate are of param_type, summed in
 * float32 in an order that the sizes alone decide.  A gradient whose forward
 * input is missing is refused.
 *
 * Errors: RS_ERR_INVALID_ARG (also width > RS_EXPERT_NORM_WIDTH_MAX, an eps
 * that is negative, an eps or residual_scale that is not finite, rows not a
 * multiple of gate_rows),
 * RS_ERR_TEMP_TOO_SMALL, RS_ERR_ALIAS, RS_ERR_CUDA.  rows == 0 writes zeros to
 * the summed gradients; width == 0 does nothing.  Row strides may be 0 for
 * inputs (one row for all).
 */
typedef struct rs_expert_norm_desc {
    rs_float_type type;
    rs_float_type param_type;
    size_t rows;
    size_t width;
    float eps;
    float residual_scale;
    size_t gate_rows;
    const void* x;
    size_t x_stride;
    const void* block;
    size_t block_stride;
    const void* weight;
    const void* block_weight;
    const void* gate;
    void* y; /* forward only, with h */
    size_t y_stride;
    void* h;
    size_t h_stride;
    const void* dh; /* gradient only from here */
    size_t dh_stride;
    const void* dy;
    size_t dy_stride;
    void* dx;
    size_t dx_stride;
    void* dblock;
    size_t dblock_stride;
    void* dweight;
    void* dblock_weight;
    void* dgate;
    void* temp;
    size_t temp_bytes;
    void* stream;
} rs_expert_norm_desc;

rs_status rs_expert_norm(const rs_expert_norm_desc* desc);
size_t rs_expert_norm_grad_temp_bytes(const rs_expert_norm_desc* desc);
rs_status rs_expert_norm_grad(const rs_expert_norm_desc* desc);

#ifdef __cplusplus
}
#endif

#endif /* RS_EXPERT_BLOCK_H */
