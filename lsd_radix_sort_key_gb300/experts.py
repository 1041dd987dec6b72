"""Python binding of the expert operators (C ABI in include/rs_experts.h).

A mixture-of-experts layer, between the router's choice and the layer's
output, is

    order, position, offsets = expert_sort(ids, E)               # ids [T, K]
    rows = expert_dispatch(x, position, offsets)                 # [T*K, H]
    mid  = expert_matmul(rows, w1, offsets, bias=b1, activation="silu")
    back = expert_matmul(mid, w2, offsets, bias=b2)
    out  = expert_combine(back, weights, position, offsets)      # [T, H]

and the ``_grad`` functions give its gradients.  Functions named as in C
(``rs_expert_*``) take torch tensors or raw addresses and return the status;
the others check their tensors, allocate outputs and scratch with torch,
enqueue on ``stream`` (default: the current stream), never synchronise, and
raise on a refused call.
"""
from __future__ import annotations

import contextlib
import ctypes

FLOAT_TYPES = {"float32": 0, "float16": 1, "bfloat16": 2}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
EXPERTS_MAX = 1024  # RS_EXPERTS_MAX

_SIZE_ERROR = ctypes.c_size_t(-1).value


class ExpertMatmulDesc(ctypes.Structure):
    """Mirror of rs_expert_matmul_desc."""
    _fields_ = [("type", ctypes.c_int), ("activation", ctypes.c_int), ("num_experts", ctypes.c_int),
                ("rows", ctypes.c_size_t), ("inner", ctypes.c_size_t), ("outer", ctypes.c_size_t),
                ("offsets", ctypes.c_void_p), ("x", ctypes.c_void_p), ("x_stride", ctypes.c_size_t),
                ("w", ctypes.c_void_p), ("w_expert_stride", ctypes.c_size_t),
                ("w_outer_stride", ctypes.c_size_t), ("w_inner_stride", ctypes.c_size_t),
                ("bias", ctypes.c_void_p), ("bias_stride", ctypes.c_size_t),
                ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_size_t),
                ("y", ctypes.c_void_p), ("y_stride", ctypes.c_size_t),
                ("pre", ctypes.c_void_p), ("pre_stride", ctypes.c_size_t),
                ("dx", ctypes.c_void_p), ("dx_stride", ctypes.c_size_t),
                ("dw", ctypes.c_void_p), ("dbias", ctypes.c_void_p),
                ("temp", ctypes.c_void_p), ("temp_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p),
                ("stall_tile", ctypes.c_int32)]


def _rs():
    from . import lib
    return lib()


def _addr(x):
    return x if x is None or isinstance(x, int) else x.data_ptr()


def _raw_stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


# ---------------------------------------------------------- C-named wrappers

def rs_expert_sort_temp_bytes(n: int, num_experts: int) -> int:
    return _rs().rs_expert_sort_temp_bytes(n, num_experts)


def rs_expert_sort(ids, id_bytes, n, num_experts, order, position, offsets, temp, temp_bytes, stream=None) -> int:
    return _rs().rs_expert_sort(_addr(ids), id_bytes, n, num_experts, _addr(order), _addr(position),
                                _addr(offsets), _addr(temp), temp_bytes, _raw_stream(stream))


def rs_expert_dispatch(ftype, x, x_stride, position, routed, tokens, slots, width, out, out_stride,
                       stream=None) -> int:
    return _rs().rs_expert_dispatch(FLOAT_TYPES[ftype], _addr(x), x_stride, _addr(position), _addr(routed), tokens,
                                    slots, width, _addr(out), out_stride, _raw_stream(stream))


def rs_expert_combine(ftype, y, y_stride, weights, weight_type, position, routed, tokens, slots, width, out,
                      out_stride, stream=None) -> int:
    return _rs().rs_expert_combine(FLOAT_TYPES[ftype], _addr(y), y_stride, _addr(weights), FLOAT_TYPES[weight_type],
                                   _addr(position), _addr(routed), tokens, slots, width, _addr(out), out_stride,
                                   _raw_stream(stream))


def rs_expert_combine_grad(ftype, dout, dout_stride, y, y_stride, weights, weight_type, position, routed, tokens,
                           slots, width, dy, dy_stride, dweights, stream=None) -> int:
    return _rs().rs_expert_combine_grad(FLOAT_TYPES[ftype], _addr(dout), dout_stride, _addr(y), y_stride,
                                        _addr(weights), FLOAT_TYPES[weight_type], _addr(position), _addr(routed),
                                        tokens, slots, width, _addr(dy), dy_stride, _addr(dweights),
                                        _raw_stream(stream))


def rs_expert_matmul_temp_bytes(desc: ExpertMatmulDesc) -> int:
    return _rs().rs_expert_matmul_temp_bytes(ctypes.byref(desc))


def rs_expert_matmul(desc: ExpertMatmulDesc) -> int:
    return _rs().rs_expert_matmul(ctypes.byref(desc))


def rs_expert_matmul_grad_temp_bytes(desc: ExpertMatmulDesc) -> int:
    return _rs().rs_expert_matmul_grad_temp_bytes(ctypes.byref(desc))


def rs_expert_matmul_grad(desc: ExpertMatmulDesc) -> int:
    return _rs().rs_expert_matmul_grad(ctypes.byref(desc))


def rs_expert_matmul_status(temp, stream=None) -> int:
    """Waits for the stream; whether the last product with this temp ran to its end."""
    return _rs().rs_expert_matmul_status(_addr(temp), _raw_stream(stream))


# --------------------------------------------------------------- convenience

def _ftype(t, what):
    name = str(t.dtype)[6:]  # torch.xxx
    if name not in FLOAT_TYPES:
        raise TypeError(f"{what}: float32, float16 or bfloat16 wanted, got {t.dtype}")
    return FLOAT_TYPES[name]


def _cuda(what, t, dtype, shape, device):
    """t is a CUDA tensor of this type and shape (None: any) on this device (None: any)."""
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{what}: a tensor on {device or 'a CUDA device'} is wanted, got one on {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: {dtype} wanted, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(shape)} wanted, got {tuple(t.shape)}")


def _row_stride(what, t, out=False):
    """The row stride of a matrix whose rows' elements are adjacent."""
    rows, width = t.shape
    if width > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the elements of a row must be adjacent")
    stride = t.stride(0)
    if rows <= 1:
        return max(width, 1)
    if stride < width and (out or stride != 0):
        raise ValueError(f"{what}: rows must not overlap")
    return stride


def _plan(position, offsets, device):
    import torch
    _cuda("position", position, torch.int32, None, device)
    _cuda("offsets", offsets, torch.int32, None, device)
    if position.dim() != 2 or position.shape[1] < 1:
        raise ValueError("position: shape [tokens, slots] wanted")
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets: shape [num_experts + 1] wanted")
    if not position.is_contiguous() or not offsets.is_contiguous():
        raise ValueError("position and offsets must be contiguous")
    return position.shape[0], position.shape[1], offsets.data_ptr() + 4 * (offsets.shape[0] - 1)


def _weights(weights, y, shape):
    import torch
    if weights.dtype != torch.float32 and weights.dtype != y.dtype:
        raise TypeError(f"weights: float32 or {y.dtype} wanted, got {weights.dtype}")
    _cuda("weights", weights, None, shape, y.device)
    return weights.contiguous()


@contextlib.contextmanager
def _other(device, stream, inputs):
    """Allocate on, and launch into, `stream` of `device`; the inputs' memory
    is then not handed out again before `stream` has passed."""
    import torch
    s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
    with torch.cuda.device(device):
        if s is None:
            yield torch.cuda.current_stream().cuda_stream
            return
        with torch.cuda.stream(s):
            for t in inputs:
                if t is not None:
                    t.record_stream(s)
            yield s.cuda_stream


class _On:
    """The usual case of _other, without its cost: the tensors' device is the
    current one and the call goes to its current stream."""
    __slots__ = ("raw",)

    def __init__(self, raw):
        self.raw = raw

    def __enter__(self):
        return self.raw

    def __exit__(self, *a):
        return False


def _on(device, stream, *inputs):
    import torch
    if stream is None and device.index == torch.cuda.current_device():
        return _On(torch.cuda.current_stream().cuda_stream)
    return _other(device, stream, inputs)


def _check(code, where):
    if code != 0:
        from . import RadixSortError
        raise RadixSortError(code, where)


def expert_sort(ids, num_experts: int, *, stream=None):
    """The slots of `ids` (int32 or int64, any shape, contiguous) in stable
    order of their expert.

    Returns int32 tensors (order [n], position [ids.shape], offsets
    [num_experts + 1]): sorted row r holds slot order[r], slot s is in row
    position[s], expert e has rows offsets[e]..offsets[e+1].  A slot whose
    number lies outside [0, num_experts) is dropped: such slots come last, in
    rows offsets[num_experts] and on.
    """
    import torch
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids: int32 or int64 wanted, got {ids.dtype}")
    if not ids.is_cuda or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous CUDA tensor")
    n, dev = ids.numel(), ids.device
    h = _rs()
    tb = h.rs_expert_sort_temp_bytes(n, num_experts)
    if tb == _SIZE_ERROR:
        _check(1, "rs_expert_sort")
    with _on(dev, stream, ids) as s:
        order = torch.empty(n, dtype=torch.int32, device=dev)
        position = torch.empty(ids.shape, dtype=torch.int32, device=dev)
        offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
        temp = torch.empty(tb, dtype=torch.uint8, device=dev)
        _check(h.rs_expert_sort(ids.data_ptr(), ids.element_size(), n, num_experts, order.data_ptr(),
                                position.data_ptr(), offsets.data_ptr(), temp.data_ptr(), tb, s), "rs_expert_sort")
    return order, position, offsets


def expert_dispatch(x, position, offsets, *, stream=None):
    """x [T, H] laid out by expert: [T*K, H], row position[t, k] = x[t];
    the rows of dropped slots are zero."""
    import torch
    ft = _ftype(x, "x")
    t, k, routed = _plan(position, offsets, x.device)
    if x.dim() != 2 or x.shape[0] != t:
        raise ValueError(f"x: shape [{t}, width] wanted, got {tuple(x.shape)}")
    width, xs = x.shape[1], _row_stride("x", x)
    with _on(x.device, stream, x, position, offsets) as s:
        out = torch.empty((t * k, width), dtype=x.dtype, device=x.device)
        _check(_rs().rs_expert_dispatch(ft, x.data_ptr(), xs, position.data_ptr(), routed, t, k, width,
                                        out.data_ptr(), max(width, 1), s), "rs_expert_dispatch")
    return out


def _combine(y, weights, position, offsets, stream):
    import torch
    ft = _ftype(y, "y")
    t, k, routed = _plan(position, offsets, y.device)
    if y.dim() != 2 or y.shape[0] != t * k:
        raise ValueError(f"y: shape [{t * k}, width] wanted, got {tuple(y.shape)}")
    width, ys = y.shape[1], _row_stride("y", y)
    with _on(y.device, stream, y, weights, position, offsets) as s:
        w, wt = None, 0
        if weights is not None:
            w = _weights(weights, y, (t, k))
            wt = _ftype(w, "weights")
        out = torch.empty((t, width), dtype=y.dtype, device=y.device)
        _check(_rs().rs_expert_combine(ft, y.data_ptr(), ys, None if w is None else w.data_ptr(), wt,
                                       position.data_ptr(), routed, t, k, width, out.data_ptr(), max(width, 1), s),
               "rs_expert_combine")
    return out


def expert_dispatch_grad(dout, position, offsets, *, stream=None):
    """The gradient of expert_dispatch: each token's sum over its slots' rows
    of dout [T*K, H]; dropped slots add nothing."""
    return _combine(dout, None, position, offsets, stream)


def expert_combine(y, weights, position, offsets, *, stream=None):
    """out[t] = sum over k of weights[t, k] * y[position[t, k]]: y [T*K, H],
    weights [T, K] (float32 or y's type), out [T, H]; dropped slots add nothing."""
    if weights is None:
        raise TypeError("weights: a tensor is wanted")
    return _combine(y, weights, position, offsets, stream)


def expert_combine_grad(dout, y, weights, position, offsets, *, stream=None):
    """The gradient of expert_combine for dout [T, H]: (dy [T*K, H] like y,
    dweights [T, K] like weights); zero for dropped slots."""
    import torch
    ft = _ftype(y, "y")
    t, k, routed = _plan(position, offsets, y.device)
    if y.dim() != 2 or y.shape[0] != t * k:
        raise ValueError(f"y: shape [{t * k}, width] wanted, got {tuple(y.shape)}")
    width, ys = y.shape[1], _row_stride("y", y)
    _cuda("dout", dout, y.dtype, (t, width), y.device)
    ds = _row_stride("dout", dout)
    with _on(y.device, stream, dout, y, weights, position, offsets) as s:
        w = _weights(weights, y, (t, k))
        dy = torch.empty((t * k, width), dtype=y.dtype, device=y.device)
        dweights = torch.empty((t, k), dtype=w.dtype, device=y.device)
        _check(_rs().rs_expert_combine_grad(ft, dout.data_ptr(), ds, y.data_ptr(), ys, w.data_ptr(),
                                            _ftype(w, "weights"), position.data_ptr(), routed, t, k, width,
                                            dy.data_ptr(), max(width, 1), dweights.data_ptr(), s),
               "rs_expert_combine_grad")
    return dy, dweights


def _matmul_desc(x, w, offsets, activation):
    import torch
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation: one of {', '.join(ACTIVATIONS)} wanted, got {activation!r}")
    ft = _ftype(x, "x")
    if x.dim() != 2 or w.dim() != 3:
        raise ValueError("x: [rows, inner] and w: [experts, outer, inner] wanted")
    (rows, inner), (experts, outer, wi) = x.shape, w.shape
    _cuda("x", x, None, None, None)
    _cuda("w", w, x.dtype, (experts, outer, inner), x.device)
    _cuda("offsets", offsets, torch.int32, (experts + 1,), x.device)
    if not offsets.is_contiguous():
        raise ValueError("offsets must be contiguous")
    so, si = w.stride(1), w.stride(2)
    if inner <= 1:  # a single column's stride says nothing
        si = 1
    elif outer <= 1 and si == 1:
        so = inner
    d = ExpertMatmulDesc(ft, ACTIVATIONS[activation], experts, rows, inner, outer, offsets.data_ptr(),
                         x.data_ptr(), _row_stride("x", x), w.data_ptr(), w.stride(0) if experts > 1 else 0, so, si)
    if min(inner, outer) > 1 and so != 1 and si != 1:
        raise ValueError("w: each expert's matrix must have adjacent elements along one side")
    return d


def expert_matmul(x, w, offsets, *, bias=None, activation="none", residual=None, return_pre=False, temp=None,
                  stream=None):
    """Each expert's rows times its matrix: y[r] = act(x[r] w[e]^T + bias[e]) +
    residual[r] for rows offsets[e] <= r < offsets[e+1]; rows from
    offsets[experts] on are zero.

    x [rows, inner]; w [experts, outer, inner], either of its last two sides
    adjacent in memory; bias [experts, outer]; residual [rows, outer]; all of
    x's type.  activation: none, relu, gelu (erf) or silu.  Returns y [rows,
    outer], or (y, pre) with the values before the activation, which
    expert_matmul_grad needs.  temp: scratch of the caller's (uint8, at least
    rs_expert_matmul_temp_bytes), for rs_expert_matmul_status.
    """
    import torch
    d = _matmul_desc(x, w, offsets, activation)
    rows, outer = d.rows, d.outer
    if bias is not None:
        _cuda("bias", bias, x.dtype, (d.num_experts, outer), x.device)
        d.bias, d.bias_stride = bias.data_ptr(), _row_stride("bias", bias)
    if residual is not None:
        _cuda("residual", residual, x.dtype, (rows, outer), x.device)
        d.residual, d.residual_stride = residual.data_ptr(), _row_stride("residual", residual)
    h = _rs()
    with _on(x.device, stream, x, w, offsets, bias, residual) as s:
        y = torch.empty((rows, outer), dtype=x.dtype, device=x.device)
        d.y, d.y_stride, d.stream = y.data_ptr(), max(outer, 1), s
        pre = None
        if return_pre:
            pre = torch.empty((rows, outer), dtype=x.dtype, device=x.device)
            d.pre, d.pre_stride = pre.data_ptr(), max(outer, 1)
        ref = ctypes.byref(d)
        tb = h.rs_expert_matmul_temp_bytes(ref)
        if tb == _SIZE_ERROR:
            _check(1, "rs_expert_matmul")
        if temp is None:
            temp = torch.empty(tb, dtype=torch.uint8, device=x.device)
        d.temp, d.temp_bytes = temp.data_ptr(), temp.numel()
        _check(h.rs_expert_matmul(ref), "rs_expert_matmul")
    return (y, pre) if return_pre else y


def expert_matmul_grad(dy, x, w, offsets, *, pre=None, activation="none", bias=True, need_dx=True, need_dw=True,
                       temp=None, stream=None):
    """The gradient of expert_matmul for dy [rows, outer]: (dx like x, dw
    [experts, outer, inner], dbias [experts, outer]); None for the ones not
    wanted (need_dx, need_dw, bias).  `pre` is what return_pre gave; not
    needed for activation "none".  The residual's gradient is dy.
    """
    import torch
    d = _matmul_desc(x, w, offsets, activation)
    rows, inner, outer, experts = d.rows, d.inner, d.outer, d.num_experts
    _cuda("dy", dy, x.dtype, (rows, outer), x.device)
    d.y, d.y_stride = dy.data_ptr(), _row_stride("dy", dy)
    if activation != "none":
        if pre is None:
            raise TypeError(f"pre: needed for activation {activation!r}")
        _cuda("pre", pre, x.dtype, (rows, outer), x.device)
        d.pre, d.pre_stride = pre.data_ptr(), _row_stride("pre", pre)
    h = _rs()
    with _on(x.device, stream, dy, x, w, offsets, pre) as s:
        dx = dw = dbias = None
        if need_dx:
            dx = torch.empty((rows, inner), dtype=x.dtype, device=x.device)
            d.dx, d.dx_stride = dx.data_ptr() or None, max(inner, 1)
        if need_dw:
            dw = torch.empty((experts, outer, inner), dtype=x.dtype, device=x.device)
            d.dw = dw.data_ptr() or None
        if bias:
            dbias = torch.empty((experts, outer), dtype=x.dtype, device=x.device)
            d.dbias = dbias.data_ptr() or None
        ref = ctypes.byref(d)
        tb = h.rs_expert_matmul_grad_temp_bytes(ref)
        if tb == _SIZE_ERROR:
            _check(1, "rs_expert_matmul_grad")
        d.stream = s
        if temp is None:
            temp = torch.empty(tb, dtype=torch.uint8, device=x.device)
        d.temp, d.temp_bytes = temp.data_ptr(), temp.numel()
        _check(h.rs_expert_matmul_grad(ref), "rs_expert_matmul_grad")
    return dx, dw, dbias
