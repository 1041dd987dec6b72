// rs_torch.cpp -- the expert operators' Python calls in their ordinary form, as
// a CPython extension over torch's tensors.
//
// The calls in experts.py cost 10 to 15 us each on the host, most of it in the
// interpreter and in torch.empty, which is more than the kernels of a decoding
// step take.  Each function here does what its namesake there does when
// nothing is out of the ordinary (plain tensors of the right types and shapes
// on the current device, the current stream) and returns its outputs; anything
// else, an error included, returns None, and the caller goes on in Python,
// which handles the rest and words the errors.  The kernels are reached through
// the C ABI of librs.so, whose entry points bind() takes by address, so that
// both ways use the one library that is loaded.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <utility>

#include "rs_expert_block.h"

namespace {

struct Entry {
    decltype(&rs_expert_sort_temp_bytes) sort_temp_bytes;
    decltype(&rs_expert_sort) sort;
    decltype(&rs_expert_dispatch) dispatch;
    decltype(&rs_expert_combine) combine;
    decltype(&rs_expert_combine_grad) combine_grad;
    decltype(&rs_expert_matmul_temp_bytes) matmul_temp_bytes;
    decltype(&rs_expert_matmul) matmul;
    decltype(&rs_expert_matmul_grad_temp_bytes) matmul_grad_temp_bytes;
    decltype(&rs_expert_matmul_grad) matmul_grad;
    decltype(&rs_expert_quantize) quantize;
    decltype(&rs_expert_dispatch_quantized) dispatch_quantized;
    decltype(&rs_expert_quantize_weights) quantize_weights;
    decltype(&rs_expert_matmul_quantized_temp_bytes) matmul_quantized_temp_bytes;
    decltype(&rs_expert_matmul_quantized) matmul_quantized;
    decltype(&rs_expert_norm) norm;
    decltype(&rs_expert_norm_grad_temp_bytes) norm_grad_temp_bytes;
    decltype(&rs_expert_norm_grad) norm_grad;
} g_rs;

PyObject* none() { Py_RETURN_NONE; }

// A flag is True or False; any other object's truth is Python's to find.
bool flag(PyObject* o, bool* value)
{
    *value = o == Py_True;
    return o == Py_True || o == Py_False;
}

// A plain tensor (not a subclass with ideas of its own), or nullptr.
const at::Tensor* tensor(PyObject* o)
{
    return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

bool on_current_device(const at::Tensor& t) { return t.is_cuda() && t.get_device() == c10::cuda::current_device(); }

int float_type(const at::Tensor& t)
{
    switch (t.scalar_type()) {
    case at::kFloat: return RS_FLOAT32;
    case at::kHalf: return RS_FLOAT16;
    case at::kBFloat16: return RS_BFLOAT16;
    default: return -1;
    }
}

// The row stride of a matrix whose rows' elements are adjacent and which the
// library takes as it is; false for any other tensor.
bool row_stride(const at::Tensor& t, size_t* stride)
{
    if (t.dim() != 2) return false;
    const int64_t rows = t.size(0), width = t.size(1);
    if (width > 1 && t.stride(1) != 1) return false;
    if (rows <= 1) {
        *stride = width ? (size_t)width : 1;
        return true;
    }
    if (t.stride(0) < width && t.stride(0) != 0) return false;
    *stride = (size_t)t.stride(0);
    return true;
}

bool is(const at::Tensor& t, const at::Tensor& like, int64_t rows, int64_t width)
{
    return t.dim() == 2 && t.size(0) == rows && t.size(1) == width && t.scalar_type() == like.scalar_type() &&
           t.device() == like.device();
}

struct Plan {
    const int32_t *position, *routed;
    int64_t tokens, slots;
};

bool plan(const at::Tensor& position, const at::Tensor& offsets, const at::Tensor& like, Plan* p)
{
    if (position.scalar_type() != at::kInt || offsets.scalar_type() != at::kInt || position.dim() != 2 ||
        offsets.dim() != 1 || position.device() != like.device() || offsets.device() != like.device() ||
        !position.is_contiguous() || !offsets.is_contiguous() || position.size(1) < 1 ||
        position.size(1) > RS_EXPERT_SLOTS_MAX || offsets.size(0) < 2)
        return false;
    *p = Plan{static_cast<const int32_t*>(position.const_data_ptr()),
              static_cast<const int32_t*>(offsets.const_data_ptr()) + offsets.size(0) - 1, position.size(0),
              position.size(1)};
    return true;
}

bool weights_ok(const at::Tensor& w, const at::Tensor& y, const Plan& p)
{
    return w.dim() == 2 && w.size(0) == p.tokens && w.size(1) == p.slots && w.device() == y.device() &&
           w.is_contiguous() && (w.scalar_type() == at::kFloat || w.scalar_type() == y.scalar_type());
}

void* current_stream(const at::Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }

at::Tensor like(const at::Tensor& t, at::IntArrayRef shape) { return at::empty(shape, t.options()); }
at::Tensor bytes(const at::Tensor& t, size_t n) { return at::empty({(int64_t)n}, t.options().dtype(at::kByte)); }

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

// A tuple of tensors; an undefined one becomes None.
template <size_t N>
PyObject* wrap_all(at::Tensor (&&t)[N])
{
    PyObject* r = PyTuple_New(N);
    if (!r) return nullptr;
    for (size_t i = 0; i < N; ++i) {
        PyObject* o = t[i].defined() ? wrap(std::move(t[i])) : Py_NewRef(Py_None);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, (Py_ssize_t)i, o);
    }
    return r;
}

// ---- the calls; arguments by position

// (ids, num_experts)
PyObject* sort(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const at::Tensor* ids = n == 2 ? tensor(a[0]) : nullptr;
    if (!ids || !PyLong_CheckExact(a[1])) return none();
    int over = 0;
    const long experts = PyLong_AsLongAndOverflow(a[1], &over);
    if (over || experts < 1 || experts > RS_EXPERTS_MAX || !on_current_device(*ids) || !ids->is_contiguous() ||
        (ids->scalar_type() != at::kLong && ids->scalar_type() != at::kInt))
        return none();
    const size_t count = (size_t)ids->numel(), tb = g_rs.sort_temp_bytes(count, (int)experts);
    if (tb == (size_t)-1) return none();
    const at::TensorOptions i32 = ids->options().dtype(at::kInt);
    at::Tensor order = at::empty({(int64_t)count}, i32), position = at::empty(ids->sizes(), i32);
    at::Tensor offsets = at::empty({experts + 1}, i32), temp;
    if (tb) temp = bytes(*ids, tb);
    if (g_rs.sort(ids->const_data_ptr(), (int)ids->element_size(), count, (int)experts,
                  static_cast<int32_t*>(order.mutable_data_ptr()), static_cast<int32_t*>(position.mutable_data_ptr()),
                  static_cast<int32_t*>(offsets.mutable_data_ptr()), tb ? temp.mutable_data_ptr() : nullptr, tb,
                  current_stream(*ids)) != RS_OK)
        return none();
    return wrap_all({std::move(order), std::move(position), std::move(offsets)});
    END_HANDLE_TH_ERRORS
}

// (x, position, offsets)
PyObject* dispatch(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 3) return none();
    const at::Tensor *x = tensor(a[0]), *position = tensor(a[1]), *offsets = tensor(a[2]);
    Plan p;
    size_t xs;
    if (!x || !position || !offsets || float_type(*x) < 0 || !on_current_device(*x) || !row_stride(*x, &xs) ||
        !plan(*position, *offsets, *x, &p) || x->size(0) != p.tokens)
        return none();
    const int64_t width = x->size(1);
    at::Tensor out = like(*x, {p.tokens * p.slots, width});
    if (g_rs.dispatch((rs_float_type)float_type(*x), x->const_data_ptr(), xs, p.position, p.routed, (size_t)p.tokens,
                      (int)p.slots, (size_t)width, out.mutable_data_ptr(), width ? (size_t)width : 1,
                      current_stream(*x)) != RS_OK)
        return none();
    return wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// (y, weights or None, position, offsets)
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 4) return none();
    const at::Tensor *y = tensor(a[0]), *w = a[1] == Py_None ? nullptr : tensor(a[1]);
    const at::Tensor *position = tensor(a[2]), *offsets = tensor(a[3]);
    Plan p;
    size_t ys;
    if (!y || (!w && a[1] != Py_None) || !position || !offsets || float_type(*y) < 0 || !on_current_device(*y) ||
        !row_stride(*y, &ys) || !plan(*position, *offsets, *y, &p) || y->size(0) != p.tokens * p.slots ||
        (w && !weights_ok(*w, *y, p)))
        return none();
    const int64_t width = y->size(1);
    at::Tensor out = like(*y, {p.tokens, width});
    if (g_rs.combine((rs_float_type)float_type(*y), y->const_data_ptr(), ys, w ? w->const_data_ptr() : nullptr,
                     w ? (rs_float_type)float_type(*w) : RS_FLOAT32, p.position, p.routed, (size_t)p.tokens,
                     (int)p.slots, (size_t)width, out.mutable_data_ptr(), width ? (size_t)width : 1,
                     current_stream(*y)) != RS_OK)
        return none();
    return wrap(std::move(out));
    END_HANDLE_TH_ERRORS
}

// (dout, y, weights, position, offsets)
PyObject* combine_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 5) return none();
    const at::Tensor *dout = tensor(a[0]), *y = tensor(a[1]), *w = tensor(a[2]), *position = tensor(a[3]),
                     *offsets = tensor(a[4]);
    Plan p;
    size_t ys, ds;
    if (!dout || !y || !w || !position || !offsets || float_type(*y) < 0 || !on_current_device(*y) ||
        !row_stride(*y, &ys) || !plan(*position, *offsets, *y, &p) || y->size(0) != p.tokens * p.slots ||
        !is(*dout, *y, p.tokens, y->size(1)) || !row_stride(*dout, &ds) || !weights_ok(*w, *y, p))
        return none();
    const int64_t width = y->size(1);
    at::Tensor dy = like(*y, {y->size(0), width}), dw = like(*w, {p.tokens, p.slots});
    if (g_rs.combine_grad((rs_float_type)float_type(*y), dout->const_data_ptr(), ds, y->const_data_ptr(), ys,
                          w->const_data_ptr(), (rs_float_type)float_type(*w), p.position, p.routed, (size_t)p.tokens,
                          (int)p.slots, (size_t)width, dy.mutable_data_ptr(), width ? (size_t)width : 1,
                          dw.mutable_data_ptr(), current_stream(*y)) != RS_OK)
        return none();
    return wrap_all({std::move(dy), std::move(dw)});
    END_HANDLE_TH_ERRORS
}

// What both products check, and the descriptor's head.
bool products(const at::Tensor& x, const at::Tensor& w, const at::Tensor& offsets, long act, rs_expert_matmul_desc* d)
{
    const int type = float_type(x);
    if (type < 0 || act < RS_ACT_NONE || act > RS_ACT_SILU || !on_current_device(x) || w.dim() != 3 ||
        w.scalar_type() != x.scalar_type() || w.device() != x.device() || !row_stride(x, &d->x_stride) ||
        w.size(2) != x.size(1) || offsets.scalar_type() != at::kInt || offsets.device() != x.device() ||
        offsets.dim() != 1 || offsets.size(0) != w.size(0) + 1 || !offsets.is_contiguous() || w.size(0) < 1 ||
        w.size(0) > RS_EXPERTS_MAX || w.size(1) < 2 || w.size(2) < 2 || (w.stride(1) != 1 && w.stride(2) != 1))
        return false;
    d->type = (rs_float_type)type;
    d->activation = (rs_activation)act;
    d->num_experts = (int)w.size(0);
    d->rows = (size_t)x.size(0);
    d->inner = (size_t)x.size(1);
    d->outer = (size_t)w.size(1);
    d->offsets = static_cast<const int32_t*>(offsets.const_data_ptr());
    d->x = x.const_data_ptr();
    d->w = w.const_data_ptr();
    d->w_expert_stride = w.size(0) > 1 ? (size_t)w.stride(0) : 0;
    d->w_outer_stride = (size_t)w.stride(1);
    d->w_inner_stride = (size_t)w.stride(2);
    d->stream = current_stream(x);
    return true;
}

// (x, w, offsets, bias or None, activation number, residual or None, return_pre)
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 7) return none();
    const at::Tensor *x = tensor(a[0]), *w = tensor(a[1]), *offsets = tensor(a[2]);
    const at::Tensor *bias = a[3] == Py_None ? nullptr : tensor(a[3]), *res = a[5] == Py_None ? nullptr : tensor(a[5]);
    bool want_pre;
    if (!x || !w || !offsets || (!bias && a[3] != Py_None) || (!res && a[5] != Py_None) || !PyLong_CheckExact(a[4]) ||
        !flag(a[6], &want_pre))
        return none();
    rs_expert_matmul_desc d{};
    if (!products(*x, *w, *offsets, PyLong_AsLong(a[4]), &d)) return none();
    const int64_t rows = x->size(0), outer = w->size(1);
    if (bias) {
        if (!is(*bias, *x, w->size(0), outer) || !row_stride(*bias, &d.bias_stride)) return none();
        d.bias = bias->const_data_ptr();
    }
    if (res) {
        if (!is(*res, *x, rows, outer) || !row_stride(*res, &d.residual_stride)) return none();
        d.residual = res->const_data_ptr();
    }
    at::Tensor y = like(*x, {rows, outer}), pre;
    d.y = y.mutable_data_ptr();
    d.y_stride = d.pre_stride = (size_t)outer;
    if (want_pre) {
        pre = like(*x, {rows, outer});
        d.pre = pre.mutable_data_ptr();
    }
    const size_t tb = g_rs.matmul_temp_bytes(&d);
    if (tb == (size_t)-1) return none();
    const at::Tensor temp = bytes(*x, tb);
    d.temp = temp.mutable_data_ptr();
    d.temp_bytes = tb;
    if (g_rs.matmul(&d) != RS_OK) return none();
    if (want_pre) return wrap_all({std::move(y), std::move(pre)});
    return wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

// (dy, x, w, offsets, pre or None, activation number, bias, need_dx, need_dw)
PyObject* matmul_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 9) return none();
    const at::Tensor *dy = tensor(a[0]), *x = tensor(a[1]), *w = tensor(a[2]), *offsets = tensor(a[3]);
    const at::Tensor* pre = a[4] == Py_None ? nullptr : tensor(a[4]);
    bool want_bias, want_dx, want_dw;
    if (!dy || !x || !w || !offsets || (!pre && a[4] != Py_None) || !PyLong_CheckExact(a[5]) ||
        !flag(a[6], &want_bias) || !flag(a[7], &want_dx) || !flag(a[8], &want_dw))
        return none();
    rs_expert_matmul_desc d{};
    const long act = PyLong_AsLong(a[5]);
    if (!products(*x, *w, *offsets, act, &d)) return none();
    const int64_t rows = x->size(0), inner = x->size(1), outer = w->size(1);
    if (!is(*dy, *x, rows, outer) || !row_stride(*dy, &d.y_stride)) return none();
    d.y = const_cast<void*>(dy->const_data_ptr());
    if (act != RS_ACT_NONE) {
        if (!pre || !is(*pre, *x, rows, outer) || !row_stride(*pre, &d.pre_stride)) return none();
        d.pre = const_cast<void*>(pre->const_data_ptr());
    }
    at::Tensor dx, dw, dbias;
    if (want_dx) {
        dx = like(*x, {rows, inner});
        d.dx = dx.mutable_data_ptr();
        d.dx_stride = (size_t)inner;
    }
    if (want_dw) {
        dw = like(*x, {w->size(0), outer, inner});
        d.dw = dw.mutable_data_ptr();
    }
    if (want_bias) {
        dbias = like(*x, {w->size(0), outer});
        d.dbias = dbias.mutable_data_ptr();
    }
    const size_t tb = g_rs.matmul_grad_temp_bytes(&d);
    if (tb == (size_t)-1) return none();
    const at::Tensor temp = bytes(*x, tb);
    d.temp = temp.mutable_data_ptr();
    d.temp_bytes = tb;
    if (g_rs.matmul_grad(&d) != RS_OK) return none();
    return wrap_all({std::move(dx), std::move(dw), std::move(dbias)});
    END_HANDLE_TH_ERRORS
}

// ---- an expert block in 8 bits, and the norms around it

constexpr int64_t kBlock = RS_QUANT_BLOCK;
int64_t blocks_of(int64_t width) { return (width + kBlock - 1) / kBlock; }
int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Quantised rows on 16 bytes and their scales on 4.
struct Quantized {
    at::Tensor q, scales;  // as the caller sees them
    void *q_at, *scales_at;
    size_t q_stride, scales_stride;

    Quantized(const at::Tensor& like, int64_t rows, int64_t width)
    {
        const int64_t n = blocks_of(width), qs = std::max<int64_t>(16, up(width, 16)), ss = std::max<int64_t>(4, up(n, 4));
        q = at::empty({rows, qs}, like.options().dtype(at::kFloat8_e4m3fn));
        scales = at::empty({rows, ss}, like.options().dtype(at::kFloat8_e8m0fnu));
        q_at = q.mutable_data_ptr();
        scales_at = scales.mutable_data_ptr();
        q_stride = (size_t)qs;
        scales_stride = (size_t)ss;
        seen(q, {rows, width}, {qs, 1});
        seen(scales, {rows, n}, {ss, 1});
    }

    // A new tensor that shows part of its memory (a view takes the host 2 us longer).
    static void seen(const at::Tensor& t, at::IntArrayRef sizes, at::IntArrayRef strides)
    {
        if (t.sizes() != sizes) t.unsafeGetTensorImpl()->set_sizes_and_strides(sizes, strides);
    }
};

// (x)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const at::Tensor* x = n == 1 ? tensor(a[0]) : nullptr;
    size_t xs;
    if (!x || float_type(*x) < 0 || !on_current_device(*x) || !row_stride(*x, &xs)) return none();
    Quantized out(*x, x->size(0), x->size(1));
    if (g_rs.quantize((rs_float_type)float_type(*x), x->const_data_ptr(), xs, (size_t)x->size(0), (size_t)x->size(1), out.q_at,
                      out.q_stride, out.scales_at, out.scales_stride, current_stream(*x)) != RS_OK)
        return none();
    return wrap_all({std::move(out.q), std::move(out.scales)});
    END_HANDLE_TH_ERRORS
}

// (x, position, offsets)
PyObject* dispatch_quantized(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 3) return none();
    const at::Tensor *x = tensor(a[0]), *position = tensor(a[1]), *offsets = tensor(a[2]);
    Plan p;
    size_t xs;
    if (!x || !position || !offsets || float_type(*x) < 0 || !on_current_device(*x) || !row_stride(*x, &xs) ||
        !plan(*position, *offsets, *x, &p) || x->size(0) != p.tokens)
        return none();
    Quantized out(*x, p.tokens * p.slots, x->size(1));
    if (g_rs.dispatch_quantized((rs_float_type)float_type(*x), x->const_data_ptr(), xs, p.position, p.routed, (size_t)p.tokens,
                                (int)p.slots, (size_t)x->size(1), out.q_at, out.q_stride, out.scales_at,
                                out.scales_stride, current_stream(*x)) != RS_OK)
        return none();
    return wrap_all({std::move(out.q), std::move(out.scales)});
    END_HANDLE_TH_ERRORS
}

// (w)
PyObject* quantize_weights(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const at::Tensor* w = n == 1 ? tensor(a[0]) : nullptr;
    if (!w || float_type(*w) < 0 || !on_current_device(*w) || w->dim() != 3 || w->size(0) < 1 ||
        w->size(0) > RS_EXPERTS_MAX || (w->stride(1) != 1 && w->stride(2) != 1))
        return none();
    const int64_t experts = w->size(0), outer = w->size(1), inner = w->size(2), qs = std::max<int64_t>(16, up(inner, 16));
    at::Tensor q = at::empty({experts, outer, qs}, w->options().dtype(at::kFloat8_e4m3fn));
    at::Tensor scales = at::empty({experts, blocks_of(outer), blocks_of(inner)}, w->options().dtype(at::kFloat8_e8m0fnu));
    if (g_rs.quantize_weights((rs_float_type)float_type(*w), w->const_data_ptr(), (size_t)w->stride(0), (size_t)w->stride(1),
                              (size_t)w->stride(2), (int)experts, (size_t)outer, (size_t)inner, q.mutable_data_ptr(),
                              (size_t)qs, scales.mutable_data_ptr(), current_stream(*w)) != RS_OK)
        return none();
    Quantized::seen(q, {experts, outer, inner}, {outer * qs, qs, 1});
    return wrap_all({std::move(q), std::move(scales)});
    END_HANDLE_TH_ERRORS
}

// (x, x_scales, w, w_scales, offsets, bias or None, activation number, residual
// or None, float type, return_pre, quantize)
PyObject* matmul_quantized(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 11) return none();
    const at::Tensor *x = tensor(a[0]), *xs = tensor(a[1]), *w = tensor(a[2]), *ws = tensor(a[3]), *offsets = tensor(a[4]);
    const at::Tensor *bias = a[5] == Py_None ? nullptr : tensor(a[5]), *res = a[7] == Py_None ? nullptr : tensor(a[7]);
    bool want_pre, want_q;
    if (!x || !xs || !w || !ws || !offsets || (!bias && a[5] != Py_None) || (!res && a[7] != Py_None) ||
        !PyLong_CheckExact(a[6]) || !PyLong_CheckExact(a[8]) || !flag(a[9], &want_pre) || !flag(a[10], &want_q))
        return none();
    const long act = PyLong_AsLong(a[6]), type = PyLong_AsLong(a[8]);
    rs_expert_matmul_quantized_desc d{};
    if (act < RS_ACT_NONE || act > RS_ACT_SILU || (type != RS_FLOAT16 && type != RS_BFLOAT16) || !on_current_device(*x) ||
        x->scalar_type() != at::kFloat8_e4m3fn || w->scalar_type() != at::kFloat8_e4m3fn ||
        xs->scalar_type() != at::kFloat8_e8m0fnu || ws->scalar_type() != at::kFloat8_e8m0fnu ||
        offsets->scalar_type() != at::kInt || w->dim() != 3 || ws->dim() != 3 || offsets->dim() != 1 ||
        !row_stride(*x, &d.x_stride) || !row_stride(*xs, &d.x_scales_stride))
        return none();
    const int64_t rows = x->size(0), inner = x->size(1), experts = w->size(0), outer = w->size(1);
    for (const at::Tensor* t : {xs, w, ws, offsets})
        if (t->device() != x->device()) return none();
    if (rows == 1) d.x_stride = (size_t)up(inner, 16);  // a single row's stride is not used
    // (experts and columns enough that every other stride says something)
    if (rows < 1 || experts < 1 || experts > RS_EXPERTS_MAX || outer < 2 || inner < 2 || w->size(2) != inner ||
        w->stride(2) != 1 || (experts > 1 && w->stride(0) != outer * w->stride(1)) || xs->size(0) != rows ||
        xs->size(1) != blocks_of(inner) || ws->size(0) != experts || ws->size(1) != blocks_of(outer) ||
        ws->size(2) != blocks_of(inner) || !ws->is_contiguous() || offsets->size(0) != experts + 1 ||
        !offsets->is_contiguous())
        return none();
    const at::ScalarType out_type = type == RS_FLOAT16 ? at::kHalf : at::kBFloat16;
    auto given = [&](const at::Tensor& t, int64_t r, size_t* stride) {
        return t.dim() == 2 && t.size(0) == r && t.size(1) == outer && t.scalar_type() == out_type &&
               t.device() == x->device() && row_stride(t, stride);
    };
    if (bias) {
        if (!given(*bias, experts, &d.bias_stride)) return none();
        d.bias = bias->const_data_ptr();
    }
    if (res) {
        if (want_q || !given(*res, rows, &d.residual_stride)) return none();
        d.residual = res->const_data_ptr();
    }
    d.type = (rs_float_type)type;
    d.activation = (rs_activation)act;
    d.num_experts = (int)experts;
    d.rows = (size_t)rows;
    d.inner = (size_t)inner;
    d.outer = (size_t)outer;
    d.offsets = static_cast<const int32_t*>(offsets->const_data_ptr());
    d.x = x->const_data_ptr();
    d.x_scales = xs->const_data_ptr();
    d.w = w->const_data_ptr();
    d.w_stride = (size_t)w->stride(1);
    d.w_scales = ws->const_data_ptr();
    d.stream = current_stream(*x);
    const at::TensorOptions options = x->options().dtype(out_type);
    at::Tensor y, scales, pre;
    if (want_q) {
        Quantized out(*x, rows, outer);
        d.q = out.q_at;
        d.q_stride = out.q_stride;
        d.q_scales = out.scales_at;
        d.q_scales_stride = out.scales_stride;
        y = std::move(out.q);
        scales = std::move(out.scales);
    } else {
        y = at::empty({rows, outer}, options);
        d.y = y.mutable_data_ptr();
        d.y_stride = (size_t)outer;
    }
    if (want_pre) {
        pre = at::empty({rows, outer}, options);
        d.pre = pre.mutable_data_ptr();
        d.pre_stride = (size_t)outer;
    }
    const size_t tb = g_rs.matmul_quantized_temp_bytes(&d);
    if (tb == (size_t)-1) return none();
    const at::Tensor temp = bytes(*x, tb);
    d.temp = temp.mutable_data_ptr();
    d.temp_bytes = tb;
    if (g_rs.matmul_quantized(&d) != RS_OK) return none();
    if (want_q && want_pre) return wrap_all({std::move(y), std::move(scales), std::move(pre)});
    if (want_q) return wrap_all({std::move(y), std::move(scales)});
    if (want_pre) return wrap_all({std::move(y), std::move(pre)});
    return wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

// A number that is exactly what it seems; false for anything else.
bool number(PyObject* o, float* value)
{
    if (PyFloat_CheckExact(o)) *value = (float)PyFloat_AS_DOUBLE(o);
    else if (PyLong_CheckExact(o)) *value = (float)PyLong_AsDouble(o);
    else return false;
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return true;
}

// What a norm and its gradient share: x, weight, block, block_weight, gate,
// residual_scale, eps; absent tensors are None.
struct NormInputs {
    const at::Tensor *x, *weight, *block, *block_weight, *gate;
    rs_expert_norm_desc d{};

    bool take(PyObject* const* a)
    {
        PyObject* const objects[] = {a[0], a[1], a[2], a[3], a[4]};
        const at::Tensor** const to[] = {&x, &weight, &block, &block_weight, &gate};
        for (int i = 0; i < 5; ++i) {
            *to[i] = objects[i] == Py_None ? nullptr : tensor(objects[i]);
            if (!*to[i] && objects[i] != Py_None) return false;
        }
        if (!x || float_type(*x) < 0 || !on_current_device(*x) || !row_stride(*x, &d.x_stride) ||
            !number(a[5], &d.residual_scale) || !number(a[6], &d.eps))
            return false;
        const int64_t rows = x->size(0), width = x->size(1);
        if (block ? !is(*block, *x, rows, width) || !row_stride(*block, &d.block_stride)
                  : !weight || block_weight || gate)
            return false;
        int type = -1;
        for (const at::Tensor* t : {weight, block_weight, gate}) {
            if (!t) continue;
            const bool by_row = t == gate && t->dim() == 2;
            if (t->dim() != (by_row ? 2 : 1) || t->size(by_row ? 1 : 0) != width || t->device() != x->device() ||
                !t->is_contiguous() || (t->scalar_type() != x->scalar_type() && t->scalar_type() != at::kFloat) ||
                (type >= 0 && type != float_type(*t)))
                return false;
            type = float_type(*t);
        }
        d.type = (rs_float_type)float_type(*x);
        d.param_type = type < 0 ? d.type : (rs_float_type)type;
        d.rows = (size_t)rows;
        d.width = (size_t)width;
        d.x = x->const_data_ptr();
        if (block) d.block = block->const_data_ptr();
        if (weight) d.weight = weight->const_data_ptr();
        if (block_weight) d.block_weight = block_weight->const_data_ptr();
        if (gate) {
            d.gate = gate->const_data_ptr();
            d.gate_rows = gate->dim() == 2 ? (size_t)gate->size(0) : 1;
            if (d.gate_rows < 1) return false;
        }
        d.stream = current_stream(*x);
        return true;
    }
};

// (x, weight, block, block_weight, gate, residual_scale, eps)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    NormInputs in;
    if (n != 7 || !in.take(a)) return none();
    const int64_t rows = in.x->size(0), width = in.x->size(1);
    at::Tensor y, h;
    in.d.y_stride = in.d.h_stride = width ? (size_t)width : 1;
    if (in.block) {
        y = like(*in.x, {rows, width});
        in.d.y = y.mutable_data_ptr();
    }
    if (in.weight) {
        h = like(*in.x, {rows, width});
        in.d.h = h.mutable_data_ptr();
    }
    if (g_rs.norm(&in.d) != RS_OK) return none();
    if (in.block) return wrap_all({std::move(y), std::move(h)});
    return wrap(std::move(h));
    END_HANDLE_TH_ERRORS
}

// (dh, y, weight, dy, block, block_weight, gate, residual_scale, eps)
PyObject* norm_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 9) return none();
    PyObject* const inputs[] = {a[1], a[2], a[4], a[5], a[6], a[7], a[8]};
    NormInputs in;
    if (!in.take(inputs)) return none();
    rs_expert_norm_desc& d = in.d;
    const at::Tensor *dh = a[0] == Py_None ? nullptr : tensor(a[0]), *dy = a[3] == Py_None ? nullptr : tensor(a[3]);
    const int64_t rows = in.x->size(0), width = in.x->size(1);
    if ((!dh && a[0] != Py_None) || (!dy && a[3] != Py_None) || !dh != !in.weight || (!dh && !dy) ||
        (dh && (!is(*dh, *in.x, rows, width) || !row_stride(*dh, &d.dh_stride))) ||
        (dy && (!is(*dy, *in.x, rows, width) || !row_stride(*dy, &d.dy_stride))))
        return none();
    if (dh) d.dh = dh->const_data_ptr();
    if (dy) d.dy = dy->const_data_ptr();
    at::Tensor dx = like(*in.x, {rows, width}), dblock, dweight, dblock_weight, dgate;
    d.dx = dx.mutable_data_ptr();
    d.dx_stride = d.dblock_stride = width ? (size_t)width : 1;
    if (in.block) {
        dblock = like(*in.x, {rows, width});
        d.dblock = dblock.mutable_data_ptr();
    }
    auto sum = [](const at::Tensor* of, at::Tensor* to, void** at) {
        if (!of) return;
        *to = like(*of, of->sizes());
        *at = to->mutable_data_ptr();
    };
    sum(in.weight, &dweight, &d.dweight);
    sum(in.block_weight, &dblock_weight, &d.dblock_weight);
    sum(in.gate, &dgate, &d.dgate);
    const size_t tb = g_rs.norm_grad_temp_bytes(&d);
    if (tb == (size_t)-1) return none();
    const at::Tensor temp = bytes(*in.x, tb);
    d.temp = temp.mutable_data_ptr();
    d.temp_bytes = tb;
    if (g_rs.norm_grad(&d) != RS_OK) return none();
    return wrap_all({std::move(dx), std::move(dweight), std::move(dblock), std::move(dblock_weight), std::move(dgate)});
    END_HANDLE_TH_ERRORS
}

// bind(addresses): the C entry points in the order of Entry.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    constexpr Py_ssize_t kEntries = sizeof(Entry) / sizeof(void*);
    if (n != kEntries) {
        PyErr_Format(PyExc_TypeError, "%zd addresses are wanted", kEntries);
        return nullptr;
    }
    void* p[kEntries];
    for (Py_ssize_t i = 0; i < n; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    static_assert(sizeof(p) == sizeof(g_rs), "one address per entry");
    memcpy(&g_rs, p, sizeof p);
    Py_RETURN_NONE;
}

#define RS_METHOD(f, doc) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, doc}
PyMethodDef methods[] = {RS_METHOD(bind, "bind(addresses of librs entry points)"),
                         RS_METHOD(sort, "expert_sort or None"),
                         RS_METHOD(dispatch, "expert_dispatch or None"),
                         RS_METHOD(combine, "expert_combine or None"),
                         RS_METHOD(combine_grad, "expert_combine_grad or None"),
                         RS_METHOD(matmul, "expert_matmul or None"),
                         RS_METHOD(matmul_grad, "expert_matmul_grad or None"),
                         RS_METHOD(quantize, "expert_quantize or None"),
                         RS_METHOD(dispatch_quantized, "expert_dispatch_quantized or None"),
                         RS_METHOD(quantize_weights, "expert_quantize_weights or None"),
                         RS_METHOD(matmul_quantized, "expert_matmul_quantized or None"),
                         RS_METHOD(norm, "expert_norm or None"),
                         RS_METHOD(norm_grad, "expert_norm_grad or None"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "rs_torch", "the expert operators' ordinary calls", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_rs_torch() { return PyModule_Create(&module); }
