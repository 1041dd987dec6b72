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
raise on a refused call.  They compute values only: what they return is not
part of autograd's graph, whatever their inputs require
(``examples/expert_layer.py`` has autograd Functions made of them).
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os
import struct
import sys

_pkg = sys.modules[__package__]
torch = None  # imported by the first call that needs it (importing the package does not)


# The calls below in their ordinary form, as a CPython extension (csrc/rs_torch.cpp):
# each gives its outputs, or None for a call that is out of the ordinary or
# refused, which then goes the way written here.  None where it is not built
# for the installed torch.
_fast = None


def _torch():
    global torch, _fast
    if torch is not None:
        return
    import torch as module
    FTYPES.update({getattr(module, name): code for name, code in FLOAT_TYPES.items()})
    path = _pkg._build.torch_ext()
    if path and os.path.exists(path):
        loader = importlib.machinery.ExtensionFileLoader("rs_torch", path)
        ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("rs_torch", loader))
        loader.exec_module(ext)
        names = ("sort_temp_bytes", "sort", "dispatch", "combine", "combine_grad", "matmul_temp_bytes", "matmul",
                 "matmul_grad_temp_bytes", "matmul_grad", "quantize", "dispatch_quantized", "quantize_weights",
                 "matmul_quantized_temp_bytes", "matmul_quantized", "norm", "norm_grad_temp_bytes",
                 "norm_grad")  # the order of Entry there
        ext.bind(*(ctypes.cast(getattr(_rs(), "rs_expert_" + n), ctypes.c_void_p).value for n in names))
        _fast = ext
    torch = module


FLOAT_TYPES = {"float32": 0, "float16": 1, "bfloat16": 2}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
EXPERTS_MAX = 1024  # RS_EXPERTS_MAX
SLOTS_MAX = 1 << 30  # RS_EXPERT_SLOTS_MAX

FTYPES = {}  # torch dtype -> rs_float_type
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


# The same structure as bytes: packing is several times cheaper than a
# ctypes.Structure's fields one by one.
_DESC = struct.Struct("@3i4x 3N 2PN P3N PN PN PN PN PN PP PN P i4x")


def _rs():
    return _pkg._lib or _pkg.lib()


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
    return _rs().rs_expert_matmul_temp_bytes(ctypes.addressof(desc))


def rs_expert_matmul(desc: ExpertMatmulDesc) -> int:
    return _rs().rs_expert_matmul(ctypes.addressof(desc))


def rs_expert_matmul_grad_temp_bytes(desc: ExpertMatmulDesc) -> int:
    return _rs().rs_expert_matmul_grad_temp_bytes(ctypes.addressof(desc))


def rs_expert_matmul_grad(desc: ExpertMatmulDesc) -> int:
    return _rs().rs_expert_matmul_grad(ctypes.addressof(desc))


def rs_expert_matmul_status(temp, stream=None) -> int:
    """Waits for the stream; whether the last product with this temp ran to its end."""
    return _rs().rs_expert_matmul_status(_addr(temp), _raw_stream(stream))


# --------------------------------------------------------------- convenience

def _ftype(t, what):
    code = FTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: float32, float16 or bfloat16 wanted, got {t.dtype}")
    return code


def _like(what, t, x, shape):
    """t has x's device and type and this shape."""
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(shape)} wanted, got {tuple(t.shape)}")
    if t.dtype != x.dtype:
        raise TypeError(f"{what}: {x.dtype} wanted, got {t.dtype}")
    if t.device != x.device:
        raise ValueError(f"{what}: a tensor on {x.device} is wanted, got one on {t.device}")


def _rows(what, t):
    """(rows, width, row stride) of a CUDA matrix whose rows' elements are adjacent."""
    if not t.is_cuda:
        raise ValueError(f"{what}: a CUDA tensor is wanted, got one on {t.device}")
    if t.dim() != 2:
        raise ValueError(f"{what}: a matrix of rows is wanted, got shape {tuple(t.shape)}")
    rows, width = t.shape
    stride, inner = t.stride()
    if inner != 1 and width > 1:
        raise ValueError(f"{what}: the elements of a row must be adjacent")
    if rows <= 1:
        stride = width or 1
    elif stride < width and stride != 0:
        raise ValueError(f"{what}: rows must not overlap")
    return rows, width, stride


def _plan(position, offsets, device):
    """(tokens, slots, address of the number of rows in use) of a sort's result."""
    for what, t, dims in (("position", position, 2), ("offsets", offsets, 1)):
        if t.dtype != torch.int32:
            raise TypeError(f"{what}: torch.int32 wanted, got {t.dtype}")
        if t.device != device:
            raise ValueError(f"{what}: a tensor on {device} is wanted, got one on {t.device}")
        if t.dim() != dims or not t.is_contiguous():
            raise ValueError(f"{what}: a contiguous tensor of {dims} dimension(s) is wanted")
    tokens, slots = position.shape
    if slots < 1:
        raise ValueError("position: shape [tokens, slots] wanted")
    if slots > SLOTS_MAX:  # C's int would hold its low 32 bits
        _check(1, "position")
    edges = offsets.shape[0]
    if edges < 2:
        raise ValueError("offsets: shape [num_experts + 1] wanted")
    return tokens, slots, offsets.data_ptr() + 4 * (edges - 1)


def _weights(weights, y, shape):
    if weights.dtype != torch.float32 and weights.dtype != y.dtype:
        raise TypeError(f"weights: float32 or {y.dtype} wanted, got {weights.dtype}")
    if weights.shape != shape:
        raise ValueError(f"weights: shape {shape} wanted, got {tuple(weights.shape)}")
    if weights.device != y.device:
        raise ValueError(f"weights: a tensor on {y.device} is wanted, got one on {weights.device}")


def _scratch(temp, x):
    """The caller's scratch is memory that x's device can be handed: all of its
    bytes are its own."""
    if not isinstance(temp, torch.Tensor) or temp.dtype != torch.uint8:
        raise TypeError(f"temp: a torch.uint8 tensor is wanted, got {getattr(temp, 'dtype', type(temp).__name__)}")
    if temp.device != x.device:
        raise ValueError(f"temp: a tensor on {x.device} is wanted, got one on {temp.device}")
    if not temp.is_contiguous():
        raise ValueError("temp: a contiguous tensor is wanted")


def _current(device, stream):
    """The current stream's handle in the usual case: no stream is asked for
    and the tensors are on the current device; else None."""
    i = device.index
    if stream is None and i == torch._C._cuda_getDevice():
        return torch._C._cuda_getCurrentRawStream(i)
    return None


@contextlib.contextmanager
def _other(device, stream, inputs):
    """Allocate on, and launch into, `stream` (None: the current one) of
    `device`; the memory of the caller's tensors (inputs, scratch) is then not
    handed out again before `stream` has passed."""
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


def _check(code, where):
    if code != 0:
        raise _pkg.RadixSortError(code, where)


def expert_sort(ids, num_experts: int, *, stream=None):
    """The slots of `ids` (int32 or int64, any shape, contiguous) in stable
    order of their expert.

    Returns int32 tensors (order [n], position [ids.shape], offsets
    [num_experts + 1]): sorted row r holds slot order[r], slot s is in row
    position[s], expert e has rows offsets[e]..offsets[e+1].  A slot whose
    number lies outside [0, num_experts) is dropped: such slots come last, in
    rows offsets[num_experts] and on.
    """
    if torch is None:
        _torch()
    if stream is None and _fast is not None:
        out = _fast.sort(ids, num_experts)
        if out is not None:
            return out
    if ids.dtype != torch.int64 and ids.dtype != torch.int32:
        raise TypeError(f"ids: int32 or int64 wanted, got {ids.dtype}")
    if not ids.is_cuda or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous CUDA tensor")
    dev = ids.device
    s = _current(dev, stream)
    if s is None:
        with _other(dev, stream, (ids,)) as s:
            return _sort(ids, num_experts, dev, s)
    return _sort(ids, num_experts, dev, s)


def _sort(ids, num_experts, dev, s):
    n, i32, h = ids.numel(), torch.int32, _rs()
    if not 1 <= num_experts <= EXPERTS_MAX:  # here, as C's int would hold its low 32 bits
        _check(1, "rs_expert_sort")
    tb = h.rs_expert_sort_temp_bytes(n, num_experts)
    if tb == _SIZE_ERROR:
        _check(1, "rs_expert_sort")
    order = torch.empty(n, dtype=i32, device=dev)
    position = torch.empty(ids.shape, dtype=i32, device=dev)
    offsets = torch.empty(num_experts + 1, dtype=i32, device=dev)
    temp = torch.empty(tb, dtype=torch.uint8, device=dev).data_ptr() if tb else None
    _check(h.rs_expert_sort(ids.data_ptr(), ids.element_size(), n, num_experts, order.data_ptr(),
                            position.data_ptr(), offsets.data_ptr(), temp, tb, s), "rs_expert_sort")
    return order, position, offsets


def expert_dispatch(x, position, offsets, *, stream=None):
    """x [T, H] laid out by expert: [T*K, H], row position[t, k] = x[t];
    the rows of dropped slots are zero."""
    if torch is None:
        _torch()
    if stream is None and _fast is not None:
        out = _fast.dispatch(x, position, offsets)
        if out is not None:
            return out
    ft, dev = _ftype(x, "x"), x.device
    rows, width, xs = _rows("x", x)
    t, k, routed = _plan(position, offsets, dev)
    if rows != t:
        raise ValueError(f"x: shape [{t}, width] wanted, got {tuple(x.shape)}")
    args = (ft, x, xs, position, routed, t, k, width)
    s = _current(dev, stream)
    if s is None:
        with _other(dev, stream, (x, position, offsets)) as s:
            return _dispatch(*args, s)
    return _dispatch(*args, s)


def _dispatch(ft, x, xs, position, routed, t, k, width, s):
    out = torch.empty((t * k, width), dtype=x.dtype, device=x.device)
    _check(_rs().rs_expert_dispatch(ft, x.data_ptr(), xs, position.data_ptr(), routed, t, k, width, out.data_ptr(),
                                    width or 1, s), "rs_expert_dispatch")
    return out


def _combine(y, weights, position, offsets, stream):
    if torch is None:
        _torch()
    if stream is None and _fast is not None:
        out = _fast.combine(y, weights, position, offsets)
        if out is not None:
            return out
    ft, dev = _ftype(y, "y"), y.device
    rows, width, ys = _rows("y", y)
    t, k, routed = _plan(position, offsets, dev)
    if rows != t * k:
        raise ValueError(f"y: shape [{t * k}, width] wanted, got {tuple(y.shape)}")
    if weights is not None:
        _weights(weights, y, (t, k))
    args = (ft, y, ys, weights, position, routed, t, k, width)
    s = _current(dev, stream)
    if s is None:
        with _other(dev, stream, (y, weights, position, offsets)) as s:
            return _combine_on(*args, s)
    return _combine_on(*args, s)


def _combine_on(ft, y, ys, weights, position, routed, t, k, width, s):
    w, wt = None, 0
    if weights is not None:
        weights = weights.contiguous()
        w, wt = weights.data_ptr(), FTYPES[weights.dtype]
    out = torch.empty((t, width), dtype=y.dtype, device=y.device)
    _check(_rs().rs_expert_combine(ft, y.data_ptr(), ys, w, wt, position.data_ptr(), routed, t, k, width,
                                   out.data_ptr(), width or 1, s), "rs_expert_combine")
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
    if torch is None:
        _torch()
    if stream is None and _fast is not None:
        out = _fast.combine_grad(dout, y, weights, position, offsets)
        if out is not None:
            return out
    ft, dev = _ftype(y, "y"), y.device
    rows, width, ys = _rows("y", y)
    t, k, routed = _plan(position, offsets, dev)
    if rows != t * k:
        raise ValueError(f"y: shape [{t * k}, width] wanted, got {tuple(y.shape)}")
    _like("dout", dout, y, (t, width))
    ds = _rows("dout", dout)[2]
    _weights(weights, y, (t, k))
    args = (ft, dout, ds, y, ys, weights, position, routed, t, k, width)
    s = _current(dev, stream)
    if s is None:
        with _other(dev, stream, (dout, y, weights, position, offsets)) as s:
            return _combine_grad(*args, s)
    return _combine_grad(*args, s)


def _combine_grad(ft, dout, ds, y, ys, weights, position, routed, t, k, width, s):
    w = weights.contiguous()
    dy = torch.empty((t * k, width), dtype=y.dtype, device=y.device)
    dweights = torch.empty((t, k), dtype=w.dtype, device=y.device)
    _check(_rs().rs_expert_combine_grad(ft, dout.data_ptr(), ds, y.data_ptr(), ys, w.data_ptr(), FTYPES[w.dtype],
                                        position.data_ptr(), routed, t, k, width, dy.data_ptr(), width or 1,
                                        dweights.data_ptr(), s), "rs_expert_combine_grad")
    return dy, dweights


def _products(x, w, offsets, activation):
    """The head of the descriptor (up to w's strides) after the checks that
    both products share, and (rows, inner, outer, experts)."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation: one of {', '.join(ACTIVATIONS)} wanted, got {activation!r}")
    ft = _ftype(x, "x")
    rows, inner, xs = _rows("x", x)
    if w.dim() != 3:
        raise ValueError("w: [experts, outer, inner] wanted")
    experts, outer, _ = w.shape
    _like("w", w, x, (experts, outer, inner))
    if offsets.dtype != torch.int32:
        raise TypeError(f"offsets: torch.int32 wanted, got {offsets.dtype}")
    if offsets.shape != (experts + 1,) or offsets.device != x.device or not offsets.is_contiguous():
        raise ValueError(f"offsets: a contiguous tensor of shape ({experts + 1},) on {x.device} is wanted")
    se, so, si = w.stride()
    if inner <= 1:  # the stride of a single column or row says nothing
        si = 1
    elif outer <= 1 and si == 1:
        so = inner
    if so != 1 and si != 1 and inner > 1 and outer > 1:
        raise ValueError("w: each expert's matrix must have adjacent elements along one side")
    head = (ft, act, experts, rows, inner, outer, offsets.data_ptr(), x.data_ptr(), xs, w.data_ptr(),
            se if experts > 1 else 0, so, si)
    return head, rows, inner, outer, experts


def expert_matmul(x, w, offsets, *, bias=None, activation="none", residual=None, return_pre=False, temp=None,
                  stream=None):
    """Each expert's rows times its matrix: y[r] = act(x[r] w[e]^T + bias[e]) +
    residual[r] for rows offsets[e] <= r < offsets[e+1]; rows from
    offsets[experts] on are zero.

    x [rows, inner]; w [experts, outer, inner], either of its last two sides
    adjacent in memory; bias [experts, outer]; residual [rows, outer]; all of
    x's type.  activation: none, relu, gelu (erf) or silu.  Returns y [rows,
    outer], or (y, pre) with the values before the activation, which
    expert_matmul_grad needs.  temp: scratch of the caller's (uint8 on x's
    device, contiguous, 256-byte aligned, at least rs_expert_matmul_temp_bytes),
    for rs_expert_matmul_status.
    """
    if torch is None:
        _torch()
    if stream is None and temp is None and _fast is not None:
        out = _fast.matmul(x, w, offsets, bias, ACTIVATIONS.get(activation), residual, return_pre)
        if out is not None:
            return out
    head, rows, inner, outer, experts = _products(x, w, offsets, activation)
    extra = [None, 0, None, 0]
    if bias is not None:
        _like("bias", bias, x, (experts, outer))
        extra[0:2] = bias.data_ptr(), _rows("bias", bias)[2]
    if residual is not None:
        _like("residual", residual, x, (rows, outer))
        extra[2:4] = residual.data_ptr(), _rows("residual", residual)[2]
    if temp is not None:
        _scratch(temp, x)
    args = (head, extra, x, rows, outer, return_pre, temp)
    s = _current(x.device, stream)
    if s is None:
        with _other(x.device, stream, (x, w, offsets, bias, residual, temp)) as s:
            return _matmul(*args, s)
    return _matmul(*args, s)


def _matmul(head, extra, x, rows, outer, return_pre, temp, s):
    y = torch.empty((rows, outer), dtype=x.dtype, device=x.device)
    pre = torch.empty((rows, outer), dtype=x.dtype, device=x.device) if return_pre else None
    h = _rs()
    body = (*head, *[v or 0 for v in extra], y.data_ptr(), outer or 1, pre.data_ptr() if return_pre else 0, outer or 1,
            0, 0, 0, 0)
    if temp is None:
        tb = h.rs_expert_matmul_temp_bytes(_DESC.pack(*body, 0, 0, 0, 0))
        if tb == _SIZE_ERROR:
            _check(1, "rs_expert_matmul")
        temp = torch.empty(tb, dtype=torch.uint8, device=x.device)
    _check(h.rs_expert_matmul(_DESC.pack(*body, temp.data_ptr(), temp.numel(), s, 0)), "rs_expert_matmul")
    return (y, pre) if return_pre else y


def expert_matmul_grad(dy, x, w, offsets, *, pre=None, activation="none", bias=True, need_dx=True, need_dw=True,
                       temp=None, stream=None):
    """The gradient of expert_matmul for dy [rows, outer]: (dx like x, dw
    [experts, outer, inner], dbias [experts, outer]); None for the ones not
    wanted (need_dx, need_dw, bias).  `pre` is what return_pre gave; not
    needed for activation "none".  The residual's gradient is dy.
    """
    if torch is None:
        _torch()
    if stream is None and temp is None and _fast is not None:
        out = _fast.matmul_grad(dy, x, w, offsets, pre, ACTIVATIONS.get(activation), bias, need_dx, need_dw)
        if out is not None:
            return out
    head, rows, inner, outer, experts = _products(x, w, offsets, activation)
    _like("dy", dy, x, (rows, outer))
    grads = [dy.data_ptr(), _rows("dy", dy)[2], 0, 0]
    if activation != "none":
        if pre is None:
            raise TypeError(f"pre: needed for activation {activation!r}")
        _like("pre", pre, x, (rows, outer))
        grads[2:4] = pre.data_ptr(), _rows("pre", pre)[2]
    if temp is not None:
        _scratch(temp, x)
    args = (head, grads, x, rows, inner, outer, experts, need_dx, need_dw, bias, temp)
    s = _current(x.device, stream)
    if s is None:
        with _other(x.device, stream, (dy, x, w, offsets, pre, temp)) as s:
            return _matmul_grad(*args, s)
    return _matmul_grad(*args, s)


def _matmul_grad(head, grads, x, rows, inner, outer, experts, need_dx, need_dw, bias, temp, s):
    dt, dev, h = x.dtype, x.device, _rs()
    dx = torch.empty((rows, inner), dtype=dt, device=dev) if need_dx else None
    dw = torch.empty((experts, outer, inner), dtype=dt, device=dev) if need_dw else None
    dbias = torch.empty((experts, outer), dtype=dt, device=dev) if bias else None
    outs = [0 if t is None else t.data_ptr() for t in (dx, dw, dbias)]
    tail = (*head, 0, 0, 0, 0, *grads, outs[0], inner or 1, outs[1], outs[2])
    if temp is None:
        tb = h.rs_expert_matmul_grad_temp_bytes(_DESC.pack(*tail, 0, 0, 0, 0))
        if tb == _SIZE_ERROR:
            _check(1, "rs_expert_matmul_grad")
        temp = torch.empty(tb, dtype=torch.uint8, device=dev)
    _check(h.rs_expert_matmul_grad(_DESC.pack(*tail, temp.data_ptr(), temp.numel(), s, 0)), "rs_expert_matmul_grad")
    return dx, dw, dbias
