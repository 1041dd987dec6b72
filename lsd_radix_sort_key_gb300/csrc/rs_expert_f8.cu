// rs_expert_f8.cu -- rs_expert_matmul_quantized: its arguments.  The kernels are
// in rs_expert_f8.cuh.
#include "rs_expert_f8.cuh"

// Instantiated in rs_expert_f8_<type>.cu; not here.
namespace rsx {
extern template rs_status f8_product<__half>(const F8Operands&, const F8Args<__half>&, cudaStream_t);
extern template rs_status f8_product<__nv_bfloat16>(const F8Operands&, const F8Args<__nv_bfloat16>&, cudaStream_t);
}  // namespace rsx

namespace {

using namespace rsx;

constexpr size_t kStatusBytes = kStatusWords * 4;

rs_status check_sizes(const rs_expert_matmul_quantized_desc* d)
{
    if (!d || (d->type != RS_FLOAT16 && d->type != RS_BFLOAT16)) return RS_ERR_INVALID_ARG;
    if (d->activation < RS_ACT_NONE || d->activation > RS_ACT_SILU) return RS_ERR_INVALID_ARG;
    if (d->num_experts < 1 || d->num_experts > RS_EXPERTS_MAX || d->stall_tile < 0) return RS_ERR_INVALID_ARG;
    if (d->rows > RS_EXPERT_SLOTS_MAX || d->inner < 1 || d->inner > RS_EXPERT_WIDTH_MAX || d->outer > RS_EXPERT_WIDTH_MAX)
        return RS_ERR_INVALID_ARG;
    return RS_OK;
}

// Rows of bytes at 16-byte addresses (a tensor map's strides are below 2^40).
bool valid_bytes(const void* p, size_t stride, size_t width)
{
    return p && (uintptr_t)p % 16 == 0 && stride % 16 == 0 && stride >= width && stride <= ((size_t)1 << 32);
}

template <typename T>
rs_status product(const rs_expert_matmul_quantized_desc* d)
{
    F8Args<T> p{};
    p.offsets = d->offsets;
    p.experts = (uint32_t)d->num_experts;
    p.rows = (uint32_t)d->rows;
    p.cols = (uint32_t)d->outer;
    p.reduce = (uint32_t)d->inner;
    p.act = d->activation;
    p.a_scales = static_cast<const uint8_t*>(d->x_scales);
    p.a_scales_i = d->x_scales_stride;
    p.b_scales = static_cast<const uint8_t*>(d->w_scales);
    p.bias = static_cast<const T*>(d->bias);
    p.bias_e = d->bias_stride;
    p.residual = static_cast<const T*>(d->residual);
    p.residual_i = d->residual_stride;
    p.d = static_cast<T*>(d->y);
    p.d_i = d->y_stride;
    p.q = static_cast<uint8_t*>(d->q);
    p.q_i = d->q_stride;
    p.q_scales = static_cast<uint8_t*>(d->q_scales);
    p.q_scales_i = d->q_scales_stride;
    p.pre = static_cast<T*>(d->pre);
    p.pre_i = d->pre_stride;
    p.status = static_cast<uint32_t*>(d->temp);
    p.status_words = kStatusWords;
    p.stall = (uint32_t)d->stall_tile;
    return f8_product<T>({d->x, d->x_stride, d->w, d->w_stride}, p, static_cast<cudaStream_t>(d->stream));
}

}  // namespace

extern "C" {

size_t rs_expert_matmul_quantized_temp_bytes(const rs_expert_matmul_quantized_desc* d)
{
    return check_sizes(d) == RS_OK ? kStatusBytes : (size_t)-1;
}

rs_status rs_expert_matmul_quantized(const rs_expert_matmul_quantized_desc* d)
{
    const rs_status st = check_sizes(d);
    if (st != RS_OK) return st;
    if (d->rows == 0 || d->outer == 0) return RS_OK;
    const size_t n = d->rows, e = (size_t)d->num_experts, xw = d->inner, yw = d->outer;
    const size_t across = ceil_div(xw, RS_QUANT_BLOCK), down = ceil_div(yw, RS_QUANT_BLOCK);
    if (!d->offsets || (uintptr_t)d->offsets % 4) return RS_ERR_INVALID_ARG;
    if (!valid_bytes(d->x, d->x_stride, xw) || !valid_bytes(d->w, d->w_stride, xw)) return RS_ERR_INVALID_ARG;
    if (!d->x_scales || d->x_scales_stride < across || d->x_scales_stride > ((size_t)1 << 32) || !d->w_scales)
        return RS_ERR_INVALID_ARG;
    if (d->bias && !valid_rows(d->bias, 2, yw, d->bias_stride, true)) return RS_ERR_INVALID_ARG;
    if (d->residual && !valid_rows(d->residual, 2, yw, d->residual_stride, true)) return RS_ERR_INVALID_ARG;
    if (d->pre && !valid_rows(d->pre, 2, yw, d->pre_stride, false)) return RS_ERR_INVALID_ARG;
    if (!d->y == !d->q) return RS_ERR_INVALID_ARG;
    if (d->y && !valid_rows(d->y, 2, yw, d->y_stride, false)) return RS_ERR_INVALID_ARG;
    if (d->q && (!valid_bytes(d->q, d->q_stride, yw) || !d->q_scales || d->q_scales_stride < down ||
                 d->q_scales_stride > ((size_t)1 << 32) || d->residual))
        return RS_ERR_INVALID_ARG;
    if (!d->temp || (uintptr_t)d->temp % 256) return RS_ERR_INVALID_ARG;
    if (d->temp_bytes < kStatusBytes) return RS_ERR_TEMP_TOO_SMALL;
    const Range r[] = {{d->y, span_bytes(n, yw, d->y_stride, 2)},
                       {d->q, span_bytes(n, align_up(yw, 16), d->q_stride, 1)},
                       {d->q ? d->q_scales : nullptr, span_bytes(n, down, d->q_scales_stride, 1)},
                       {d->pre, span_bytes(n, yw, d->pre_stride, 2)},
                       {d->temp, kStatusBytes},
                       {d->x, span_bytes(n, xw, d->x_stride, 1)},
                       {d->x_scales, span_bytes(n, across, d->x_scales_stride, 1)},
                       {d->w, span_bytes(e * yw, xw, d->w_stride, 1)},
                       {d->w_scales, e * down * across},
                       {d->bias, span_bytes(e, yw, d->bias_stride, 2)},
                       {d->residual, span_bytes(n, yw, d->residual_stride, 2)},
                       {d->offsets, (e + 1) * 4}};
    if (any_alias(r, 5, 12)) return RS_ERR_ALIAS;
    return d->type == RS_FLOAT16 ? product<__half>(d) : product<__nv_bfloat16>(d);
}

}  // extern "C"
