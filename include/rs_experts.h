/*
 * rs_experts.h -- C ABI of the expert operators for NVIDIA GB300 (sm_103a):
 * tokens sorted by expert, their rows sent to the experts and back with
 * weights applied, the experts' matrix products, and the gradients.
 *
 * A mixture-of-experts layer gives each of T tokens K slots, each holding an
 * expert number.  Sorting the T*K slots by expert is a stable one-digit
 * counting sort (one pass of the sort in rs.h); every later step only needs
 * the permutation it leaves behind:
 *
 *   slot      s = t*K + k, the k-th choice of token t
 *   order[r]  the slot in sorted row r (ascending expert, ties in slot order;
 *             slots whose number is outside [0, num_experts) are DROPPED and
 *             come after every expert's, in slot order)
 *   position[s]  the sorted row of slot s (the inverse of order)
 *   offsets[e]   the first row of expert e, e = 0..num_experts: rows
 *             [offsets[e], offsets[e+1]) are expert e's, and rows from
 *             offsets[num_experts] on belong to dropped slots.
 *
 *   rs_expert_dispatch       out[position[s]] = x[t], dropped slots' rows zero
 *   rs_expert_combine        out[t] = sum_k weights[t,k] * y[position[t,k]]
 *   rs_expert_combine_grad   dy[position[t,k]] = weights[t,k] * dout[t],
 *                            dweights[t,k] = <dout[t], y[position[t,k]]>
 *   rs_expert_matmul         y[r] = act(x[r] w[e]^T + bias[e]) + residual[r]
 *   rs_expert_matmul_grad    its gradients for x, w and bias
 *
 * The gradient of rs_expert_dispatch is rs_expert_combine without weights; a
 * residual's gradient is dy itself.
 *
 * Conventions: as in rs.h (device pointers, caller-owned memory, calls only
 * enqueue work on `stream` and may be captured into a CUDA graph, arguments
 * are checked before anything is enqueued), and
 *   Types.    Rows and weights are float32, binary16 or bfloat16
 *     (rs_float_type).  Sums are held in float32 and rounded once, on the
 *     way out.  Positions, orders and offsets are int32.
 *   Layout.   A matrix of rows is given with its row stride in ELEMENTS; the
 *     elements of a row are adjacent.  Any stride >= the row's width and any
 *     element-aligned base are accepted; 16-byte-aligned rows are the fast
 *     ones (a product first copies 16-bit operands with other rows into
 *     temp).  An input's row stride may also be 0 (one row for all).
 *   Dropped slots and unused rows.  A dropped slot adds nothing to a
 *     combined row (its y row is not read, so NaN there does not spread), its
 *     dispatched row, its dy row and its dweights are zero.  Rows of a
 *     product's outputs from offsets[num_experts] on are zero, and the rows
 *     of its inputs there are not used.  A token whose slots are all dropped
 *     gets a zero row.  An expert without rows has zero dw and dbias.
 *   Bad plans.  Offsets are clamped to ascending values in [0, rows] and
 *     positions outside [0, T*K) are treated as dropped, so a wrong plan
 *     gives wrong rows but no access outside the arrays.
 *   Results do not depend on timing: no floating-point atomics are used.
 *   Aliasing.  Outputs must not overlap inputs, temp or each other
 *     (RS_ERR_ALIAS).
 */
#ifndef RS_EXPERTS_H
#define RS_EXPERTS_H

#include "rs.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest num_experts, slots (T*K) and row width any call below accepts. */
#define RS_EXPERTS_MAX 1024
#define RS_EXPERT_SLOTS_MAX 1073741824u
#define RS_EXPERT_WIDTH_MAX 1048576u

typedef enum rs_float_type { RS_FLOAT32 = 0, RS_FLOAT16 = 1, RS_BFLOAT16 = 2 } rs_float_type;

typedef enum rs_activation {
    RS_ACT_NONE = 0,
    RS_ACT_RELU = 1, /* max(z, 0); gradient 0 at z = 0       */
    RS_ACT_GELU = 2, /* z * Phi(z), Phi the normal cdf (erf) */
    RS_ACT_SILU = 3  /* z / (1 + exp(-z))                    */
} rs_activation;

/* Bytes of scratch rs_expert_sort needs for n slots (0 for small n),
 * (size_t)-1 for arguments it would reject. */
size_t rs_expert_sort_temp_bytes(size_t n, int num_experts);

/*
 * ids: n expert numbers, int32 or int64 (id_bytes 4 or 8); any value is
 * allowed, one outside [0, num_experts) marks a dropped slot.  order and
 * position: n int32 each; offsets: num_experts + 1 int32.  temp: 256-byte
 * aligned, NULL if it needs none.  n == 0 writes zero offsets.  Errors: RS_ERR_INVALID_ARG (a NULL or
 * misaligned pointer, n > RS_EXPERT_SLOTS_MAX, num_experts outside
 * [1, RS_EXPERTS_MAX], id_bytes), RS_ERR_TEMP_TOO_SMALL, RS_ERR_ALIAS,
 * RS_ERR_CUDA.
 */
rs_status rs_expert_sort(const void* ids, int id_bytes, size_t n, int num_experts, int32_t* order,
                         int32_t* position, int32_t* offsets, void* temp, size_t temp_bytes, void* stream);

/*
 * The row movers.  tokens = T, slots = K >= 1 per token, tokens*slots <=
 * RS_EXPERT_SLOTS_MAX; position: T*K; routed: one int32 on the device, the
 * number of rows that belong to experts (offsets + num_experts).
 * weights: T*K, row t at weights + t*slots, float32 or the rows' own type
 * (weight_type); NULL in rs_expert_combine means all ones.
 * tokens == 0 or width == 0: RS_OK, nothing enqueued (a zero width still
 * writes dweights = 0).  Errors: RS_ERR_INVALID_ARG, RS_ERR_ALIAS,
 * RS_ERR_CUDA.
 */
rs_status rs_expert_dispatch(rs_float_type type, const void* x, size_t x_stride, const int32_t* position,
                             const int32_t* routed, size_t tokens, int slots, size_t width, void* out,
                             size_t out_stride, void* stream);
rs_status rs_expert_combine(rs_float_type type, const void* y, size_t y_stride, const void* weights,
                            rs_float_type weight_type, const int32_t* position, const int32_t* routed,
                            size_t tokens, int slots, size_t width, void* out, size_t out_stride, void* stream);
rs_status rs_expert_combine_grad(rs_float_type type, const void* dout, size_t dout_stride, const void* y,
                                 size_t y_stride, const void* weights, rs_float_type weight_type,
                                 const int32_t* position, const int32_t* routed, size_t tokens, int slots,
                                 size_t width, void* dy, size_t dy_stride, void* dweights, void* stream);

/*
 * The experts' products.  x: rows x inner; w: one outer x inner matrix per
 * expert, element (e, n, k) at w[e*w_expert_stride + n*w_outer_stride +
 * k*w_inner_stride]; one of the last two strides is 1 (either layout of the
 * matrix runs at full speed) unless inner or outer is 1, and all are below
 * 2^40 bytes (the stride of a single expert, row or column is not used).
 * Row strides are at most 2^32 elements everywhere.  bias: outer
 * values per expert, row stride bias_stride (0: one bias for every expert), or
 * NULL.  residual: rows x outer, or NULL.  num_experts == 1 with offsets
 * {0, rows} is the plain dense product.
 *
 * rs_expert_matmul writes y and, if pre is not NULL, the values before the
 * activation (x w^T + bias, rounded), which the gradient needs.
 *
 * rs_expert_matmul_grad reads dy (in `y`, rows x outer, y_stride), x, w and,
 * for an activation other than NONE, pre; it writes the ones of dx (rows x
 * inner), dw (contiguous num_experts x outer x inner) and dbias (contiguous
 * num_experts x outer) that are not NULL, each in `type`.  dz = dy * act'(pre)
 * is formed in float32 and rounded to `type` as the products' operand, as x
 * and w are (so in binary16 a dz up to 2^-25 counts as 0 and one of 65520 or
 * more as infinite); dbias sums the unrounded values.
 *
 * temp: 256-byte aligned scratch of at least rs_expert_matmul_temp_bytes /
 * rs_expert_matmul_grad_temp_bytes bytes, computed from the same descriptor;
 * (size_t)-1 for one the call would reject.  rs_expert_matmul_status waits for
 * `stream` and says whether the last call with this temp ran to its end:
 * RS_OK, RS_ERR_DEVICE_TIMEOUT (a wait inside a tensor-core kernel ran out
 * after about two seconds, and 4 us more per 64 rows of a gradient's longest
 * expert; its outputs are then not complete), RS_ERR_CUDA.
 * Meaningful after a call that enqueued work.
 * rows == 0: dw and dbias are still written (zero).  Sizes: rows <=
 * RS_EXPERT_SLOTS_MAX, inner and outer <= RS_EXPERT_WIDTH_MAX; inner == 0 is
 * allowed (a product of nothing), outer == 0 is a no-op.
 */
typedef struct rs_expert_matmul_desc {
    rs_float_type type;
    rs_activation activation;
    int num_experts;
    size_t rows;
    size_t inner;
    size_t outer;
    const int32_t* offsets; /* num_experts + 1, on the device */
    const void* x;
    size_t x_stride;
    const void* w;
    size_t w_expert_stride;
    size_t w_outer_stride;
    size_t w_inner_stride;
    const void* bias;
    size_t bias_stride;
    const void* residual;
    size_t residual_stride;
    void* y; /* rs_expert_matmul: the output; _grad: dy, read only */
    size_t y_stride;
    void* pre;
    size_t pre_stride;
    void* dx; /* _grad only from here */
    size_t dx_stride;
    void* dw;
    void* dbias;
    void* temp;
    size_t temp_bytes;
    void* stream;
    /* Testing hook, 0 in normal use: t + 1 makes the tensor-core kernels never
     * copy the operands of output tile t, so the waits for them run out. */
    int32_t stall_tile;
} rs_expert_matmul_desc;

size_t rs_expert_matmul_temp_bytes(const rs_expert_matmul_desc* desc);
rs_status rs_expert_matmul(const rs_expert_matmul_desc* desc);
size_t rs_expert_matmul_grad_temp_bytes(const rs_expert_matmul_desc* desc);
rs_status rs_expert_matmul_grad(const rs_expert_matmul_desc* desc);
rs_status rs_expert_matmul_status(const void* temp, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RS_EXPERTS_H */
