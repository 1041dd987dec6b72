"""Python binding of an expert block in 8 bits and the norms around it (C ABI
in include/rs_expert_block.h).

Between the residual stream and back, with the experts' weights quantised once
(w1, w1_scales = expert_quantize_weights(w)):

    h = expert_norm(x, weight)                                        # [T, H]
    order, position, offsets = expert_sort(ids, E)                    # ids [T, K]
    rows, scales = expert_dispatch_quantized(h, position, offsets)    # [T*K, H]
    mid, mid_scales = expert_matmul_quantized(rows, scales, w1, w1_scales, offsets, bias=b1, activation="silu",
                                              quantize=True)
    back = expert_matmul_quantized(mid, mid_scales, w2, w2_scales, offsets, bias=b2)
    out = expert_combine(back, weights, position, offsets)            # [T, H]
    x, h = expert_norm(x, next_weight, block=out, block_weight=after, gate=gate, residual_scale=0.7)

Quantised values are ``torch.float8_e4m3fn``, their scales (one for 128 values of
a row, or for 128 x 128 of a weight matrix) ``torch.float8_e8m0fnu``: powers of
two, so ``q.float() * scales.float().repeat_interleave(128, -1)[..., :width]`` is
exactly what quantised rows stand for.  Conventions are those of ``experts.py``.
"""
from __future__ import annotations

import ctypes
import struct

from . import experts as _x
from .experts import (ACTIVATIONS, FLOAT_TYPES, FTYPES, _SIZE_ERROR, _addr, _check, _current, _ftype, _like, _other, _plan,
                      _raw_stream, _rows, _rs, _scratch)

QUANT_BLOCK = 128  # RS_QUANT_BLOCK
NORM_WIDTH_MAX = 16384  # RS_EXPERT_NORM_WIDTH_MAX


class ExpertMatmulQuantizedDesc(ctypes.Structure):
    """Mirror of rs_expert_matmul_quantized_desc."""
    _fields_ = [("type", ctypes.c_int), ("activation", ctypes.c_int), ("num_experts", ctypes.c_int),
                ("rows", ctypes.c_size_t), ("inner", ctypes.c_size_t), ("outer", ctypes.c_size_t),
                ("offsets", ctypes.c_void_p), ("x", ctypes.c_void_p), ("x_stride", ctypes.c_size_t),
                ("x_scales", ctypes.c_void_p), ("x_scales_stride", ctypes.c_size_t),
                ("w", ctypes.c_void_p), ("w_stride", ctypes.c_size_t), ("w_scales", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("bias_stride", ctypes.c_size_t),
                ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_size_t),
                ("y", ctypes.c_void_p), ("y_stride", ctypes.c_size_t),
                ("q", ctypes.c_void_p), ("q_stride", ctypes.c_size_t),
                ("q_scales", ctypes.c_void_p), ("q_scales_stride", ctypes.c_size_t),
                ("pre", ctypes.c_void_p), ("pre_stride", ctypes.c_size_t),
                ("temp", ctypes.c_void_p), ("temp_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p),
                ("stall_tile", ctypes.c_int32)]


class ExpertNormDesc(ctypes.Structure):
    """Mirror of rs_expert_norm_desc."""
    _fields_ = [("type", ctypes.c_int), ("param_type", ctypes.c_int), ("rows", ctypes.c_size_t),
                ("width", ctypes.c_size_t), ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("gate_rows", ctypes.c_size_t), ("x", ctypes.c_void_p), ("x_stride", ctypes.c_size_t),
                ("block", ctypes.c_void_p), ("block_stride", ctypes.c_size_t), ("weight", ctypes.c_void_p),
                ("block_weight", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("y_stride", ctypes.c_size_t), ("h", ctypes.c_void_p), ("h_stride", ctypes.c_size_t),
                ("dh", ctypes.c_void_p), ("dh_stride", ctypes.c_size_t), ("dy", ctypes.c_void_p),
                ("dy_stride", ctypes.c_size_t), ("dx", ctypes.c_void_p), ("dx_stride", ctypes.c_size_t),
                ("dblock", ctypes.c_void_p), ("dblock_stride", ctypes.c_size_t), ("dweight", ctypes.c_void_p),
                ("dblock_weight", ctypes.c_void_p), ("dgate", ctypes.c_void_p), ("temp", ctypes.c_void_p),
                ("temp_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p)]


# The same structures as bytes (see experts.py).
_MATMUL = struct.Struct("@3i4x 3N 2PN PN PN P PN PN PN PN PN PN PN P i4x")
_NORM = struct.Struct("@2i 2N 2f N PN PN 3P PN PN PN PN PN PN 3P PN P")


# ---------------------------------------------------------- C-named wrappers

def rs_expert_quantize(ftype, x, x_stride, rows, width, q, q_stride, scales, scales_stride, stream=None) -> int:
    return _rs().rs_expert_quantize(FLOAT_TYPES[ftype], _addr(x), x_stride, rows, width, _addr(q), q_stride,
                                    _addr(scales), scales_stride, _raw_stream(stream))


def rs_expert_dispatch_quantized(ftype, x, x_stride, position, routed, tokens, slots, width, q, q_stride, scales,
                                 scales_stride, stream=None) -> int:
    return _rs().rs_expert_dispatch_quantized(FLOAT_TYPES[ftype], _addr(x), x_stride, _addr(position), _addr(routed),
                                              tokens, slots, width, _addr(q), q_stride, _addr(scales), scales_stride,
                                              _raw_stream(stream))


def rs_expert_quantize_weights(ftype, w, w_expert_stride, w_outer_stride, w_inner_stride, num_experts, outer, inner, q,
                               q_stride, scales, stream=None) -> int:
    return _rs().rs_expert_quantize_weights(FLOAT_TYPES[ftype], _addr(w), w_expert_stride, w_outer_stride,
                                            w_inner_stride, num_experts, outer, inner, _addr(q), q_stride,
                                            _addr(scales), _raw_stream(stream))


def rs_expert_matmul_quantized_temp_bytes(desc: ExpertMatmulQuantizedDesc) -> int:
    return _rs().rs_expert_matmul_quantized_temp_bytes(ctypes.addressof(desc))


def rs_expert_matmul_quantized(desc: ExpertMatmulQuantizedDesc) -> int:
    return _rs().rs_expert_matmul_quantized(ctypes.addressof(desc))


def rs_expert_norm(desc: ExpertNormDesc) -> int:
    return _rs().rs_expert_norm(ctypes.addressof(desc))


def rs_expert_norm_grad_temp_bytes(desc: ExpertNormDesc) -> int:
    return _rs().rs_expert_norm_grad_temp_bytes(ctypes.addressof(desc))


def rs_expert_norm_grad(desc: ExpertNormDesc) -> int:
    return _rs().rs_expert_norm_grad(ctypes.addressof(desc))


# --------------------------------------------------------------- convenience

def _blocks(width):
    return -(-width // QUANT_BLOCK)


def _quantized_rows(rows, width, device):
    """(values, scales, their strides): rows of values start on 16 bytes, rows of
    scales on 4, which a product reads fastest."""
    torch, n = _x.torch, _blocks(width)
    qs, ss = max(16, (width + 15) // 16 * 16), max(4, (n + 3) // 4 * 4)
    q = torch.empty((rows, qs), dtype=torch.float8_e4m3fn, device=device)
    s = torch.empty((rows, ss), dtype=torch.float8_e8m0fnu, device=device)
    return (q if qs == width else q[:, :width]), (s if ss == n else s[:, :n]), qs, ss


def expert_quantize(x, *, stream=None):
    """Rows x [R, W] (float32, float16 or bfloat16) in 8 bits: (values [R, W],
    scales [R, ceil(W / 128)]).  Rows of values start on 16 bytes, so they are
    contiguous only where W is a multiple of 16."""
    if _x.torch is None:
        _x._torch()
    if stream is None and _x._fast is not None:
        out = _x._fast.quantize(x)
        if out is not None:
            return out
    ft, dev = _ftype(x, "x"), x.device
    rows, width, xs = _rows("x", x)
    s = _current(dev, stream)
    if s is None:
        with _other(dev, stream, (x,)) as s:
            return _quantize(ft, x, xs, rows, width, s)
    return _quantize(ft, x, xs, rows, width, s)


def _quantize(ft, x, xs, rows, width, s):
    q, scales, qs, ss = _quantized_rows(rows, width, x.device)
    _check(_rs().rs_expert_quantize(ft, x.data_ptr(), xs, rows, width, q.data_ptr(), qs, scales.data_ptr(), ss, s),
           "rs_expert_quantize")
    return q, scales


def expert_dispatch_quantized(x, position, offsets, *, stream=None):
    """x [T, H] quantised and laid out by expert: (values [T*K, H], scales [T*K,
    ceil(H / 128)]), row position[t, k] being x[t]'s; the rows of dropped slots
    are zero, with scales of one."""
    if _x.torch is None:
        _x._torch()
    if stream is None and _x._fast is not None:
        out = _x._fast.dispatch_quantized(x, position, offsets)
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
            return _dispatch_quantized(*args, s)
    return _dispatch_quantized(*args, s)


def _dispatch_quantized(ft, x, xs, position, routed, t, k, width, s):
    q, scales, qs, ss = _quantized_rows(t * k, width, x.device)
    _check(_rs().rs_expert_dispatch_quantized(ft, x.data_ptr(), xs, position.data_ptr(), routed, t, k, width,
                                              q.data_ptr(), qs, scales.data_ptr(), ss, s), "rs_expert_dispatch_quantized")
    return q, scales


def expert_quantize_weights(w, *, stream=None):
    """Weights w [experts, outer, inner] (either of the last two sides adjacent in
    memory) in 8 bits: (values [experts, outer, inner], scales [experts,
    ceil(outer / 128), ceil(inner / 128)]).  Of ``w.transpose(1, 2)`` it gives the
    weights with which a product takes dy to dx."""
    if _x.torch is None:
        _x._torch()
    if stream is None and _x._fast is not None:
        out = _x._fast.quantize_weights(w)
        if out is not None:
            return out
    ft, dev = _ftype(w, "w"), w.device
    if not w.is_cuda:
        raise ValueError(f"w: a CUDA tensor is wanted, got one on {dev}")
    if w.dim() != 3:
        raise ValueError("w: [experts, outer, inner] wanted")
    experts, outer, inner = w.shape
    if experts > _x.EXPERTS_MAX:
        _check(1, "rs_expert_quantize_weights")
    se, so, si = w.stride()
    if outer > 1 and inner > 1 and so != 1 and si != 1:
        raise ValueError("w: each expert's matrix must have adjacent elements along one side")
    s = _current(dev, stream)
    if s is None:
        with _other(dev, stream, (w,)) as s:
            return _quantize_weights(ft, w, s)
    return _quantize_weights(ft, w, s)


def _quantize_weights(ft, w, s):
    torch, (experts, outer, inner) = _x.torch, w.shape
    qs = max(16, (inner + 15) // 16 * 16)
    q = torch.empty((experts, outer, qs), dtype=torch.float8_e4m3fn, device=w.device)
    scales = torch.empty((experts, _blocks(outer), _blocks(inner)), dtype=torch.float8_e8m0fnu, device=w.device)
    if experts:
        _check(_rs().rs_expert_quantize_weights(ft, w.data_ptr(), *w.stride(), experts, outer, inner, q.data_ptr(), qs,
                                                scales.data_ptr(), s), "rs_expert_quantize_weights")
    return (q if qs == inner else q[:, :, :inner]), scales


def _quantized(what, t, dims):
    if t.dtype != _x.torch.float8_e4m3fn:
        raise TypeError(f"{what}: torch.float8_e4m3fn wanted, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what}: a CUDA tensor is wanted, got one on {t.device}")
    if t.dim() != dims:
        raise ValueError(f"{what}: {dims} dimensions wanted, got shape {tuple(t.shape)}")


def _scales_of(what, t, shape, device):
    if t.dtype != _x.torch.float8_e8m0fnu:
        raise TypeError(f"{what}: torch.float8_e8m0fnu wanted, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{what}: shape {shape} wanted, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{what}: a tensor on {device} is wanted, got one on {t.device}")


def expert_matmul_quantized(x, x_scales, w, w_scales, offsets, *, bias=None, activation="none", residual=None, dtype=None,
                            return_pre=False, quantize=False, temp=None, stream=None):
    """expert_matmul of quantised rows and weights, with float32 sums: y[r] =
    act(x[r] w[e]^T + bias[e]) + residual[r] for rows offsets[e] <= r <
    offsets[e+1]; rows from offsets[experts] on are zero.

    x [rows, inner] and w [experts, outer, inner] (inner adjacent, rows on 16
    bytes) with their scales, as the quantisers give them; bias [experts,
    outer]; residual [rows, outer]; dtype: float16 or bfloat16 (the default), the
    type of bias, residual and results.  Returns y [rows, outer], or with
    quantize (y's values, scales) as expert_quantize gives them, from the float32
    y (without a residual); return_pre adds the values before the activation,
    which expert_matmul_grad needs, as the last result.  temp: as in
    expert_matmul.
    """
    if _x.torch is None:
        _x._torch()
    torch = _x.torch
    if dtype is None:
        dtype = torch.bfloat16
    if stream is None and temp is None and _x._fast is not None:
        out = _x._fast.matmul_quantized(x, x_scales, w, w_scales, offsets, bias, ACTIVATIONS.get(activation), residual,
                                        FTYPES.get(dtype, -1), return_pre, quantize)
        if out is not None:
            return out
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation: one of {', '.join(ACTIVATIONS)} wanted, got {activation!r}")
    if dtype != torch.float16 and dtype != torch.bfloat16:
        raise TypeError(f"dtype: float16 or bfloat16 wanted, got {dtype}")
    _quantized("x", x, 2)
    _quantized("w", w, 3)
    rows, inner, xs = _rows("x", x)
    experts, outer, _ = w.shape
    _like("w", w, x, (experts, outer, inner))
    _scales_of("x_scales", x_scales, (rows, _blocks(inner)), x.device)
    _scales_of("w_scales", w_scales, (experts, _blocks(outer), _blocks(inner)), x.device)
    if rows <= 1:
        xs = (inner + 15) // 16 * 16
    ws = w.stride(1) if outer > 1 else w.stride(0) if experts > 1 else (inner + 15) // 16 * 16
    if inner > 1 and w.stride(2) != 1 or experts > 1 and outer > 1 and w.stride(0) != outer * ws:
        raise ValueError("w: the elements of a row must be adjacent, and the experts' rows at one distance")
    scale_rows, blocks, ss = _rows("x_scales", x_scales)
    if not w_scales.is_contiguous():
        raise ValueError("w_scales: a contiguous tensor is wanted")
    for what, t, stride in (("x", x, xs), ("w", w, ws)):
        if t.data_ptr() % 16 or stride % 16 or stride < inner:
            raise ValueError(f"{what}: rows on 16 bytes are wanted, as expert_quantize and expert_quantize_weights lay them out")
    if offsets.dtype != torch.int32:
        raise TypeError(f"offsets: torch.int32 wanted, got {offsets.dtype}")
    if offsets.shape != (experts + 1,) or offsets.device != x.device or not offsets.is_contiguous():
        raise ValueError(f"offsets: a contiguous tensor of shape ({experts + 1},) on {x.device} is wanted")
    extra = [0, 0, 0, 0]
    for i, (what, t, shape) in enumerate((("bias", bias, (experts, outer)), ("residual", residual, (rows, outer)))):
        if t is None:
            continue
        if t.dtype != dtype:
            raise TypeError(f"{what}: {dtype} wanted, got {t.dtype}")
        _like(what, t, t if t.device == x.device else x, shape)
        extra[2 * i:2 * i + 2] = t.data_ptr(), _rows(what, t)[2]
    if quantize and residual is not None:
        raise ValueError("residual: a product whose result is quantised takes none")
    if temp is not None:
        _scratch(temp, x)
    head = (FTYPES[dtype], act, experts, rows, inner, outer, offsets.data_ptr(), x.data_ptr(), xs, x_scales.data_ptr(), ss,
            w.data_ptr(), ws, w_scales.data_ptr(), *extra)
    args = (head, x, rows, outer, dtype, return_pre, quantize, temp)
    s = _current(x.device, stream)
    if s is None:
        with _other(x.device, stream, (x, x_scales, w, w_scales, offsets, bias, residual, temp)) as s:
            return _matmul_quantized(*args, s)
    return _matmul_quantized(*args, s)


def _matmul_quantized(head, x, rows, outer, dtype, return_pre, quantize, temp, s):
    torch, h, dev = _x.torch, _rs(), x.device
    pre = torch.empty((rows, outer), dtype=dtype, device=dev) if return_pre else None
    if quantize:
        q, scales, qs, ss = _quantized_rows(rows, outer, dev)
        out, where = (q, scales), (0, 0, q.data_ptr(), qs, scales.data_ptr(), ss)
    else:
        y = torch.empty((rows, outer), dtype=dtype, device=dev)
        out, where = (y,), (y.data_ptr(), outer or 1, 0, 0, 0, 0)
    body = (*head, *where, pre.data_ptr() if return_pre else 0, outer or 1)
    if temp is None:
        tb = h.rs_expert_matmul_quantized_temp_bytes(_MATMUL.pack(*body, 0, 0, 0, 0))
        if tb == _SIZE_ERROR:
            _check(1, "rs_expert_matmul_quantized")
        temp = torch.empty(tb, dtype=torch.uint8, device=dev)
    _check(h.rs_expert_matmul_quantized(_MATMUL.pack(*body, temp.data_ptr(), temp.numel(), s, 0)),
           "rs_expert_matmul_quantized")
    if return_pre:
        out += (pre,)
    return out if len(out) > 1 else out[0]


def _params(what, t, x, width, rows=None):
    """1 if t is float32, else 0, of parameters of x's type or float32."""
    if t.dtype != x.dtype and t.dtype != _x.torch.float32:
        raise TypeError(f"{what}: {x.dtype} or float32 wanted, got {t.dtype}")
    shape = (width,) if rows is None else (rows, width)
    if tuple(t.shape) != shape:
        raise ValueError(f"{what}: shape {shape} wanted, got {tuple(t.shape)}")
    if t.device != x.device:
        raise ValueError(f"{what}: a tensor on {x.device} is wanted, got one on {t.device}")


def _norm_inputs(x, weight, block, block_weight, gate, residual_scale, eps):
    """The checks that a norm and its gradient share: (the head of the descriptor
    up to the parameters, these)."""
    for what, v in (("residual_scale", residual_scale), ("eps", eps)):
        if isinstance(v, _x.torch.Tensor):  # its value would have to be waited for
            raise TypeError(f"{what}: a number is wanted, got a tensor")
    ft = _ftype(x, "x")
    if block is None and weight is None:
        raise TypeError("weight: a tensor is wanted (or a block)")
    rows, width, xs = _rows("x", x)
    if block is None:
        if block_weight is not None or gate is not None:
            raise ValueError("block_weight and gate go with a block")
        bs = 0
    else:
        _like("block", block, x, (rows, width))
        bs = _rows("block", block)[2]
    gate_rows = 0 if gate is None else gate.shape[0] if gate.dim() == 2 else 1
    params = [("weight", weight, None), ("block_weight", block_weight, None),
              ("gate", gate, gate_rows if gate is not None and gate.dim() == 2 else None)]
    kind = None
    for what, t, g in params:
        if t is None:
            continue
        _params(what, t, x, width, g)
        if kind is not None and t.dtype != kind:
            raise TypeError(f"{what}: {kind} wanted, as the other parameters are, got {t.dtype}")
        kind = t.dtype
    if gate is not None and rows and (gate_rows < 1 or rows % gate_rows):
        raise ValueError(f"gate: a number of rows that divides {rows} is wanted, got {gate_rows}")
    head = (ft, ft if kind is None else FTYPES[kind], rows, width, eps, residual_scale, gate_rows, x.data_ptr(), xs,
            0 if block is None else block.data_ptr(), bs)
    return head, (weight, block_weight, gate)


def _contiguous(params):
    """The parameters, copied where they are not contiguous (on the stream that
    reads them), and their addresses."""
    flat = [None if t is None else t.contiguous() for t in params]
    return flat, [0 if t is None else t.data_ptr() for t in flat]


def expert_norm(x, weight, *, block=None, block_weight=None, gate=None, residual_scale=1.0, eps=1e-6, stream=None):
    """The norm before a block, h = rms(x) * weight with rms(v) = v / sqrt(mean(v^2)
    + eps) over a row; or, given a block's output, the way out of it and into
    the next block in one:

        u = rms(block) * block_weight     (block itself without block_weight)
        y = residual_scale * x + gate * u
        h = rms(y) * weight               (of y as it is returned)

    x, block [rows, width] (width at most 16384); weight, block_weight [width];
    gate None, [width], or [sequences, width] with a row for each rows /
    sequences adjacent rows.  The parameters are of x's type or all float32;
    residual_scale and eps are numbers.  Returns h, or (y, h) with a block, h being
    None where weight is.
    """
    if _x.torch is None:
        _x._torch()
    if stream is None and _x._fast is not None:
        out = _x._fast.norm(x, weight, block, block_weight, gate, residual_scale, eps)
        if out is not None:
            return out
    head, params = _norm_inputs(x, weight, block, block_weight, gate, residual_scale, eps)
    s = _current(x.device, stream)
    if s is None:
        with _other(x.device, stream, (x, block, *params)) as s:
            return _norm(head, x, block, params, s)
    return _norm(head, x, block, params, s)


def _norm(head, x, block, params, s):
    torch, width = _x.torch, x.shape[1]
    flat, at = _contiguous(params)
    y = None if block is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    h = None if flat[0] is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _check(_rs().rs_expert_norm(_NORM.pack(*head, *at, 0 if y is None else y.data_ptr(), width or 1,
                                           0 if h is None else h.data_ptr(), width or 1, *([0] * 13), s)), "rs_expert_norm")
    return h if block is None else (y, h)


def expert_norm_grad(dh, y, weight, *, dy=None, block=None, block_weight=None, gate=None, residual_scale=1.0, eps=1e-6,
                     stream=None):
    """The gradients of expert_norm: (dx, dweight, dblock, dblock_weight, dgate),
    None for what the forward call did not have.

    y is what the norm read: x without a block, else the y that expert_norm
    returned.  dh is h's gradient (None if weight is), dy the gradient that
    reaches y by another way, the residual path (None: none; without a block it
    is simply added to dx).  The parameters' gradients have their types and are
    summed in float32.
    """
    if _x.torch is None:
        _x._torch()
    if stream is None and _x._fast is not None:
        out = _x._fast.norm_grad(dh, y, weight, dy, block, block_weight, gate, residual_scale, eps)
        if out is not None:
            return out
    if (dh is None) != (weight is None):
        raise TypeError("dh and weight go together")
    if dh is None and dy is None:
        raise TypeError("dh or dy: a tensor is wanted")
    head, params = _norm_inputs(y, weight, block, block_weight, gate, residual_scale, eps)
    grads = []
    for what, t in (("dh", dh), ("dy", dy)):
        if t is not None:
            _like(what, t, y, tuple(y.shape))
        grads += (0, 0) if t is None else (t.data_ptr(), _rows(what, t)[2])
    s = _current(y.device, stream)
    if s is None:
        with _other(y.device, stream, (dh, y, dy, block, *params)) as s:
            return _norm_grad(head, grads, y, block, params, s)
    return _norm_grad(head, grads, y, block, params, s)


def _norm_grad(head, grads, y, block, params, s):
    torch, h, width = _x.torch, _rs(), y.shape[1]
    flat, at = _contiguous(params)
    dx = torch.empty(y.shape, dtype=y.dtype, device=y.device)
    dblock = None if block is None else torch.empty(y.shape, dtype=y.dtype, device=y.device)
    sums = [None if t is None else torch.empty(t.shape, dtype=t.dtype, device=y.device) for t in flat]
    body = (*head, *at, 0, 0, 0, 0, *grads, dx.data_ptr(), width or 1, 0 if dblock is None else dblock.data_ptr(), width or 1,
            *(0 if t is None else t.data_ptr() for t in sums))
    tb = h.rs_expert_norm_grad_temp_bytes(_NORM.pack(*body, 0, 0, 0))
    if tb == _SIZE_ERROR:
        _check(1, "rs_expert_norm_grad")
    temp = torch.empty(tb, dtype=torch.uint8, device=y.device)
    _check(h.rs_expert_norm_grad(_NORM.pack(*body, temp.data_ptr(), tb, s)), "rs_expert_norm_grad")
    return dx, sums[0], dblock, sums[1], sums[2]
