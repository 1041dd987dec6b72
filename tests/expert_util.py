"""Plain 64-bit forms of the expert operators and the error bounds the GPU
tests hold them to.

Bounds.  u(T) is half the distance from 1 to the next value of type T (2^-24,
2^-11, 2^-8 for float32, binary16, bfloat16): rounding a result once costs at
most u(T) of it, or half the smallest step of T below its normal range
(2^-25 for binary16).  A sum of n products held in float32 costs at most
(n + c) * 2^-23 times the sum of the products' magnitudes, whatever the order
and whether the adder rounds or cuts off; c = 8 covers the few operations
after it (bias, activation, residual), whose own error is a few float32 ulps
of values that the magnitudes bound.
"""
import math

import torch

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {torch.float32: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
TINY = {torch.float32: 2.0**-149, torch.float16: 2.0**-25, torch.bfloat16: 2.0**-134}
ADD = 2.0**-23


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def plain_order(ids, experts):
    """order, position, offsets by a stable sort, on the CPU."""
    flat = ids.flatten().cpu().long()
    key = torch.where((flat < 0) | (flat >= experts), experts, flat)
    _, order = torch.sort(key, stable=True)
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel())
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    return order.int(), position.int().view(ids.shape), offsets.int()


def make_plan(tokens, slots, experts, seed, drop=0.0):
    g = gen(seed)
    ids = torch.randint(0, experts, (tokens, slots), device=DEV, generator=g)
    if drop:
        ids[torch.rand(tokens, slots, device=DEV, generator=g) < drop] = -1
    _, position, offsets = plain_order(ids, experts)
    return position.to(DEV), offsets.to(DEV)


def held(got, want, bound):
    """got within the elementwise bound of want (64 bits); NaN where want has NaN."""
    assert got.shape == want.shape
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    off = (got - want).abs()
    bad = (off > bound) & ~torch.isnan(want) & (got != want)  # equal infinities differ by NaN
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, worst {float((off / bound)[bad].max()):.2f} bounds"


def rounded(want, dtype):
    """The cost of rounding `want` to dtype."""
    return want.abs() * UNIT[dtype] + TINY[dtype]


# ------------------------------------------------------------ row movers

def plain_dispatch(x, position, offsets):
    t, k = position.shape
    out = torch.zeros(t * k, x.shape[1], dtype=torch.float64, device=DEV)
    for j in range(k):
        at = position[:, j].long()
        kept = at < offsets[-1]
        out[at[kept]] = x.double()[kept]
    return out


def plain_combine(y, weights, position, offsets):
    """The sum and the sum of magnitudes."""
    t, k = position.shape
    out = torch.zeros(t, y.shape[1], dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(out)
    for j in range(k):
        at = position[:, j].long()
        tok = torch.nonzero(at < offsets[-1]).flatten()
        part = y[at[tok]].double()
        if weights is not None:
            part = part * weights[tok, j, None].double()
        out[tok] += part
        mag[tok] += part.abs()
    return out, mag


def plain_combine_grad(dout, y, weights, position, offsets):
    t, k = position.shape
    dy = torch.zeros(t * k, y.shape[1], dtype=torch.float64, device=DEV)
    dw = torch.zeros(t, k, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(dw)
    for j in range(k):
        at = position[:, j].long()
        tok = torch.nonzero(at < offsets[-1]).flatten()
        d, row = dout[tok].double(), y[at[tok]].double()
        dy[at[tok]] = weights[tok, j, None].double() * d
        dw[tok, j] = (d * row).sum(1)
        mag[tok, j] = (d * row).abs().sum(1)
    return dy, dw, mag


# -------------------------------------------------------------- products

def act64(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def act_grad64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def plain_matmul(x, w, offsets, bias=None, act="none", residual=None):
    """y, z and the magnitudes behind z, in 64 bits."""
    rows, n = x.shape[0], w.shape[1]
    y = torch.zeros(rows, n, dtype=torch.float64, device=x.device)
    z, mag = torch.zeros_like(y), torch.zeros_like(y)
    edge = offsets.tolist()
    for e, (a, b) in enumerate(zip(edge, edge[1:])):
        xe, we = x[a:b].double(), w[e].double()
        z[a:b] = xe @ we.T
        mag[a:b] = xe.abs() @ we.abs().T
        if bias is not None:
            z[a:b] += bias[e].double()
            mag[a:b] += bias[e].double().abs()
        y[a:b] = act64(z[a:b], act)
        if residual is not None:
            y[a:b] += residual[a:b].double()
    return y, z, mag


def matmul_bounds(y, z, mag, inner, dtype, residual=None):
    # |act'| <= 1.13 for every activation here
    sums = 1.13 * (inner + 8) * ADD * mag
    extra = 0 if residual is None else residual.double().abs() * 2 * ADD
    return sums + extra + rounded(y, dtype) + 1e-30, sums + rounded(z, dtype) + 1e-30


def plain_matmul_grad(dy, x, w, offsets, pre=None, act="none"):
    """dx, dw, dbias; for each, the magnitudes behind it, and what an error of
    dz comes to in it: dz is computed in float32 (16 ulps of values at most
    1.13 |dy|) and, for dx and dw, rounded to the type."""
    dx = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    dw = torch.zeros(w.shape, dtype=torch.float64, device=x.device)
    db = torch.zeros(w.shape[:2], dtype=torch.float64, device=x.device)
    mags = [torch.zeros_like(t) for t in (dx, dw, db)]
    errs = [torch.zeros_like(t) for t in (dx, dw, db)]
    edge = offsets.tolist()
    for e, (a, b) in enumerate(zip(edge, edge[1:])):
        dz = dy[a:b].double()
        xe, we = x[a:b].double(), w[e].double()
        if act != "none":
            formed = 16 * ADD * 1.13 * dz.abs()
            dz = dz * act_grad64(pre[a:b].double(), act)
            kept = formed + rounded(dz, x.dtype)
            errs[0][a:b], errs[1][e], errs[2][e] = kept @ we.abs(), kept.T @ xe.abs(), formed.sum(0)
        dx[a:b], dw[e], db[e] = dz @ we, dz.T @ xe, dz.sum(0)
        mags[0][a:b], mags[1][e], mags[2][e] = dz.abs() @ we.abs(), dz.abs().T @ xe.abs(), dz.abs().sum(0)
    return (dx, dw, db), mags, errs


def grad_bounds(values, mags, errs, lengths, dtype):
    """lengths: terms in each sum."""
    return [(n + 8) * ADD * m + e + rounded(v, dtype) + 1e-30 for v, m, e, n in zip(values, mags, errs, lengths)]
