// rs_expert_norm.cu -- rs_expert_norm and rs_expert_norm_grad: their arguments.
// The kernels are in rs_expert_norm.cuh.
#include "rs_expert_norm.cuh"

// Instantiated in rs_expert_norm_<type>.cu; not here.
namespace rsx {
#define RS_EXTERN_NORM(T)                                                            \
    extern template rs_status norm_forward<T>(const NormArgs<T>&, bool, cudaStream_t); \
    extern template rs_status norm_gradient<T>(const NormArgs<T>&, bool, uint32_t, cudaStream_t);
RS_EXTERN_NORM(float)
RS_EXTERN_NORM(__half)
RS_EXTERN_NORM(__nv_bfloat16)
}  // namespace rsx

namespace {

using namespace rsx;

rs_status check_sizes(const rs_expert_norm_desc* d)
{
    if (!d || !valid_type(d->type) || (d->param_type != d->type && d->param_type != RS_FLOAT32)) return RS_ERR_INVALID_ARG;
    if (d->rows > RS_EXPERT_SLOTS_MAX || d->width > RS_EXPERT_NORM_WIDTH_MAX) return RS_ERR_INVALID_ARG;
    constexpr float most = 3.402823466e38f;
    if (!(d->eps >= 0.0f && d->eps <= most) || !(d->residual_scale >= -most && d->residual_scale <= most))
        return RS_ERR_INVALID_ARG;
    if (d->gate_rows > d->rows && d->rows) return RS_ERR_INVALID_ARG;
    if (d->gate_rows && d->rows % d->gate_rows) return RS_ERR_INVALID_ARG;
    return RS_OK;
}

// Whether the parts of the descriptor that both calls read go together.
bool valid_inputs(const rs_expert_norm_desc* d, bool reads_x)
{
    const size_t eb = type_bytes(d->type), pb = type_bytes(d->param_type);
    if (reads_x && !valid_rows(d->x, eb, d->width, d->x_stride, true)) return false;
    if (d->block && !valid_rows(d->block, eb, d->width, d->block_stride, true)) return false;
    if (!d->block && (d->block_weight || d->gate_rows)) return false;
    if (d->gate_rows && !d->gate) return false;
    for (const void* p : {d->weight, d->block_weight, d->gate})
        if ((uintptr_t)p % pb) return false;
    return true;
}

size_t param_bytes(const rs_expert_norm_desc* d) { return d->width * type_bytes(d->param_type); }

template <typename T>
NormArgs<T> norm_args(const rs_expert_norm_desc* d)
{
    NormArgs<T> p{};
    p.rows = (uint32_t)d->rows;
    p.width = (uint32_t)d->width;
    p.eps = d->eps;
    p.scale = d->block ? d->residual_scale : 1.0f;
    p.per_width = 1.0f / (float)d->width;
    p.wide_params = d->param_type == RS_FLOAT32;
    p.gate_rows = d->block ? (uint32_t)d->gate_rows : 0;
    p.x = static_cast<const T*>(d->x);
    p.x_i = d->x_stride;
    p.block = static_cast<const T*>(d->block);
    p.block_i = d->block_stride;
    p.weight = d->weight;
    p.block_weight = d->block_weight;
    p.gate = d->gate;
    return p;
}

// Whole 16-byte vectors at 16-byte addresses everywhere.
class Vectors {
public:
    explicit Vectors(const rs_expert_norm_desc* d)
        : rows_(d->rows), eb_(type_bytes(d->type)), ok_(d->width * eb_ % 16 == 0)
    {
        for (const void* p : {d->weight, d->block_weight, d->gate}) ok_ &= (uintptr_t)p % 16 == 0;
    }
    Vectors& matrix(const void* p, size_t stride)
    {
        ok_ &= !p || aligned16(p, rows_ > 1 ? stride : 0, eb_);
        return *this;
    }
    bool ok() const { return ok_; }

private:
    size_t rows_, eb_;
    bool ok_;
};

size_t grad_temp(const rs_expert_norm_desc* d)
{
    const size_t blocks = norm_grad_blocks(d->rows, d->width, type_bytes(d->type), d->block != nullptr);
    return align_up(kParts * blocks * d->width * 4, 256);
}

}  // namespace

extern "C" {

rs_status rs_expert_norm(const rs_expert_norm_desc* d)
{
    const rs_status st = check_sizes(d);
    if (st != RS_OK) return st;
    if (d->rows == 0 || d->width == 0) return RS_OK;
    const size_t eb = type_bytes(d->type), pb = param_bytes(d), n = d->rows, w = d->width;
    if (!valid_inputs(d, true) || (!d->block && !d->weight)) return RS_ERR_INVALID_ARG;
    if (d->weight && !valid_rows(d->h, eb, w, d->h_stride, false)) return RS_ERR_INVALID_ARG;
    if (d->block && !valid_rows(d->y, eb, w, d->y_stride, false)) return RS_ERR_INVALID_ARG;
    const Range r[] = {{d->weight ? d->h : nullptr, span_bytes(n, w, d->h_stride, eb)},
                       {d->block ? d->y : nullptr, span_bytes(n, w, d->y_stride, eb)},
                       {d->x, span_bytes(n, w, d->x_stride, eb)},
                       {d->block, span_bytes(n, w, d->block_stride, eb)},
                       {d->weight, pb},
                       {d->block_weight, pb},
                       {d->gate_rows ? d->gate : nullptr, d->gate_rows * pb}};
    if (any_alias(r, 2, 7)) return RS_ERR_ALIAS;
    const bool vectors = Vectors(d).matrix(d->x, d->x_stride).matrix(d->block, d->block_stride)
                             .matrix(d->block ? d->y : nullptr, d->y_stride).matrix(d->weight ? d->h : nullptr, d->h_stride).ok();
    return by_type(d->type, [&](auto t) {
        using T = decltype(t);
        NormArgs<T> p = norm_args<T>(d);
        p.y = static_cast<T*>(d->y);
        p.y_i = d->y_stride;
        p.h = static_cast<T*>(d->h);
        p.h_i = d->h_stride;
        return norm_forward<T>(p, vectors, static_cast<cudaStream_t>(d->stream));
    });
}

size_t rs_expert_norm_grad_temp_bytes(const rs_expert_norm_desc* d)
{
    return check_sizes(d) == RS_OK ? grad_temp(d) : (size_t)-1;
}

rs_status rs_expert_norm_grad(const rs_expert_norm_desc* d)
{
    const rs_status st = check_sizes(d);
    if (st != RS_OK) return st;
    const size_t eb = type_bytes(d->type), pe = type_bytes(d->param_type), pb = param_bytes(d), n = d->rows, w = d->width;
    if (w == 0 || (!d->dx && !d->dweight && !d->dblock && !d->dblock_weight && !d->dgate)) return RS_OK;
    for (const void* p : {d->dweight, d->dblock_weight, d->dgate})
        if ((uintptr_t)p % pe) return RS_ERR_INVALID_ARG;
    if (!d->weight != !d->dh && n) return RS_ERR_INVALID_ARG;  // the second norm and its gradient
    cudaStream_t s = static_cast<cudaStream_t>(d->stream);
    if (n == 0) {
        const struct {
            void* p;
            size_t bytes;
        } sums[] = {{d->dweight, pb}, {d->dblock_weight, pb}, {d->dgate, d->gate_rows * pb}};
        for (const auto& z : sums)
            if (z.p && z.bytes && cudaMemsetAsync(z.p, 0, z.bytes, s) != cudaSuccess) return RS_ERR_CUDA;
        return RS_OK;
    }
    if (!valid_inputs(d, d->dh != nullptr) || (!d->dh && !d->dy)) return RS_ERR_INVALID_ARG;
    if (d->dh && !valid_rows(d->dh, eb, w, d->dh_stride, true)) return RS_ERR_INVALID_ARG;
    if (d->dy && !valid_rows(d->dy, eb, w, d->dy_stride, true)) return RS_ERR_INVALID_ARG;
    if (d->dx && !valid_rows(d->dx, eb, w, d->dx_stride, false)) return RS_ERR_INVALID_ARG;
    if (d->dblock && !valid_rows(d->dblock, eb, w, d->dblock_stride, false)) return RS_ERR_INVALID_ARG;
    if ((d->dweight && !d->weight) || (d->dblock && !d->block) || (d->dblock_weight && !d->block_weight) ||
        (d->dgate && !d->gate_rows))
        return RS_ERR_INVALID_ARG;
    const size_t need = grad_temp(d);
    if (!d->temp || (uintptr_t)d->temp % 256) return RS_ERR_INVALID_ARG;
    if (d->temp_bytes < need) return RS_ERR_TEMP_TOO_SMALL;
    const Range r[] = {{d->dx, span_bytes(n, w, d->dx_stride, eb)},
                       {d->dblock, span_bytes(n, w, d->dblock_stride, eb)},
                       {d->dweight, pb},
                       {d->dblock_weight, pb},
                       {d->dgate, d->gate_rows * pb},
                       {d->temp, need},
                       {d->dh ? d->x : nullptr, span_bytes(n, w, d->x_stride, eb)},
                       {d->dh, span_bytes(n, w, d->dh_stride, eb)},
                       {d->dy, span_bytes(n, w, d->dy_stride, eb)},
                       {d->block, span_bytes(n, w, d->block_stride, eb)},
                       {d->weight, pb},
                       {d->block_weight, pb},
                       {d->gate_rows ? d->gate : nullptr, d->gate_rows * pb}};
    if (any_alias(r, 6, 13)) return RS_ERR_ALIAS;
    const bool vectors = Vectors(d).matrix(d->dh ? d->x : nullptr, d->x_stride).matrix(d->dh, d->dh_stride)
                             .matrix(d->dy, d->dy_stride).matrix(d->block, d->block_stride).matrix(d->dx, d->dx_stride)
                             .matrix(d->dblock, d->dblock_stride).ok();
    return by_type(d->type, [&](auto t) {
        using T = decltype(t);
        NormArgs<T> p = norm_args<T>(d);
        p.dh = static_cast<const T*>(d->dh);
        p.dh_i = d->dh_stride;
        p.dy = static_cast<const T*>(d->dy);
        p.dy_i = d->dy_stride;
        p.dx = static_cast<T*>(d->dx);
        p.dx_i = d->dx_stride;
        p.dblock = static_cast<T*>(d->dblock);
        p.dblock_i = d->dblock_stride;
        p.dweight = d->dweight;
        p.dblock_weight = d->dblock_weight;
        p.dgate = d->dgate;
        p.part = static_cast<float*>(d->temp);
        return norm_gradient<T>(p, vectors, norm_grad_blocks(n, w, eb, d->block != nullptr), s);
    });
}

}  // extern "C"
