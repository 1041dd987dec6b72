"""Plain 64-bit forms of the quantisers, the products of quantised rows and the
norms, and the error bounds the GPU tests hold them to.

Quantising is exact but for one rounding that is defined to the bit, so its
tests compare bits.  Products: see expert_util (the products of two e4m3
values and two powers of two are exact in float32, so only the additions
round).  Norms: with u = 2^-24, a row's sum of squares of W values held in
float32 is off by at most (W / 2 + 16) u of itself as the kernels add it (in
chains of at most 64, then in pairs: 64 + 10 additions and one rounding each,
taken as W / 2 + 80 below), so r = 1 / sqrt(...) by half of that and 3 u; the
products after it add a few u of values that the magnitudes bound.
"""
import torch

from expert_util import DEV, UNIT, rounded

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
U32 = UNIT[torch.float32]


def round_e4m3(v):
    """Values of magnitude at most 448 to the nearest e4m3 value, ties to even, in 64 bits."""
    _, e = torch.frexp(v.abs().clamp(min=2.0**-6))
    step = torch.exp2((e - 4).double())  # |v| in [2^(e-1), 2^e): eight steps
    return torch.round(v / step) * step


def scale_of(amax):
    """The smallest power of two from 2^-126 on with amax <= 448 scale; 1 for amax 0."""
    m, e = torch.frexp(amax.double())  # m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(amax > 0, torch.exp2(e.double()), torch.ones_like(amax, dtype=torch.float64))


def plain_quantize(x, down=1):
    """x [rows, width] with scales for each `down` x 128: (e4m3 values, scales), 64 bits."""
    r, w = x.shape
    m, n = -(-r // down), -(-w // 128)
    v = torch.zeros(m * down, n * 128, dtype=torch.float64, device=x.device)
    v[:r, :w] = x.double()
    v = torch.where(torch.isinf(v), torch.full_like(v, float("nan")), v)
    b = v.view(m, down, n, 128)
    scales = scale_of(torch.nan_to_num(b.abs(), nan=0.0).amax((1, 3)))
    q = torch.where(torch.isnan(b), b, round_e4m3(torch.nan_to_num(b) / scales[:, None, :, None]))
    return q.view(m * down, n * 128)[:r, :w], scales


def same(q, want):
    """e4m3 values equal to 64-bit ones, NaN for NaN (zeros of either sign are equal)."""
    q = q.double()
    return torch.equal(torch.isnan(q), torch.isnan(want)) and torch.equal(torch.nan_to_num(q), torch.nan_to_num(want))


def values(q, scales, down=1):
    """What quantised rows, or matrices of rows, stand for, in 64 bits."""
    s = scales.double().repeat_interleave(128, -1)[..., :q.shape[-1]]
    if down > 1:
        s = s.repeat_interleave(down, -2)[..., :q.shape[-2], :]
    return q.double() * s


def aligned(q):
    """The same values with rows that start on 16 bytes."""
    *lead, w = q.shape
    out = torch.zeros(*lead, max(16, (w + 15) // 16 * 16), dtype=torch.uint8, device=q.device)
    out[..., :w] = q.view(torch.uint8)
    return out.view(E4M3)[..., :w]


def random_quantized(g, *shape, down=1, spread=6):
    """Random e4m3 values and scales of rows (or of [experts, outer, inner] weights), as the products take them."""
    q = (torch.randn(*shape, device=DEV, generator=g) * 60).clamp(-448, 448).to(E4M3)
    blocks = (*shape[:-2], -(-shape[-2] // down), -(-shape[-1] // 128))
    scales = torch.randint(127 - spread, 127 + spread, blocks, dtype=torch.uint8, device=DEV, generator=g).view(E8M0)
    return aligned(q), scales


# ------------------------------------------------------------------ norms

def off_root(width):
    """Relative error of r: half of the sum's, and the division's and root's."""
    return ((width / 2 + 80) / 2 + 3) * U32


def root(v, eps):
    return torch.rsqrt(v.square().mean(1, keepdim=True) + eps)


def gates(gate, rows):
    if gate is None:
        return torch.ones(1, 1, dtype=torch.float64, device=DEV)
    g = gate.double()
    return g[None] if g.dim() == 1 else g.repeat_interleave(rows // g.shape[0], 0)


def plain_norm(x, weight, block, after, gate, scale, eps, held_y=None):
    """(y, its bound, h, its bound); h is of held_y, the y that was returned."""
    dt, w = x.dtype, x.shape[1]
    y = y_bound = None
    v = x.double()
    if block is not None:
        b = block.double()
        u = b if after is None else b * root(b, eps) * after.double()
        part = gates(gate, x.shape[0]) * u
        y = scale * v + part
        off = (off_root(w) + 4 * U32) * part.abs() + 3 * U32 * (scale * v).abs() + 2 * U32 * y.abs()
        y_bound = off + rounded(y, dt) + 1e-30
        v = held_y.double()
    if weight is None:
        return y, y_bound, None, None
    h = v * root(v, eps) * weight.double()
    return y, y_bound, h, (off_root(w) + 3 * U32) * h.abs() + rounded(h, dt) + 1e-30


def plain_norm_grad(dh, y, weight, dy, block, after, gate, scale, eps):
    """{name: (value, bound)} in 64 bits."""
    rows, w = y.shape
    dt = y.dtype
    d, d_off = torch.zeros(y.shape, dtype=torch.float64, device=y.device), 0.0
    out = {}

    def back(g, g_off, v, wt):
        """The gradients of v r wt for v and wt, and their errors, g being off by g_off."""
        r, f = root(v, eps), off_root(w)
        gw, gw_off = g * wt, g_off * wt.abs()
        dot, mag, dot_off = (gw * v).mean(1, keepdim=True), (gw * v).abs().mean(1, keepdim=True), \
            (gw_off * v.abs()).mean(1, keepdim=True)
        k = r**3 * v
        value = r * gw - k * dot
        off = r * gw_off + k.abs() * dot_off + (f + 4 * U32) * r * gw.abs() + 3 * (f + 4 * U32) * (k * dot).abs()
        off = off + k.abs() * mag * (w / 2 + 84) * U32
        n = v * r
        return value, off, (g * n).sum(0), (g_off * n.abs() + (f + 4 * U32) * (g * n).abs()).sum(0), (g * n).abs().sum(0)

    adds = (rows + 40) * U32  # a column's sum over the rows, whatever the order

    def summed(name, value, off, mag, like):
        out[name] = value, off + adds * mag + rounded(value, like.dtype) + 1e-30

    if dh is not None:
        g = dh.double()
        d, d_off, dw, dw_off, mag = back(g, torch.zeros_like(g), y.double(), weight.double())
        summed("dweight", dw, dw_off, mag, weight)
    if dy is not None:
        d = d + dy.double()
        d_off = d_off + U32 * d.abs()
    dx = scale * d if block is not None else d
    out["dx"] = dx, abs(scale) * d_off + 2 * U32 * dx.abs() + rounded(dx, dt) + 1e-30
    if block is None:
        return out
    d_off = d_off if torch.is_tensor(d_off) else torch.zeros_like(d)
    b = block.double()
    rb = root(b, eps) if after is not None else torch.ones(1, 1, dtype=torch.float64, device=y.device)
    wa = torch.ones(w, dtype=torch.float64, device=y.device) if after is None else after.double()
    u = b * rb * wa
    if gate is not None:
        per = rows // (1 if gate.dim() == 1 else gate.shape[0])
        sums = [t.view(-1, per, w).sum(1).view(gate.shape) for t in
                (d * u, d_off * u.abs() + (off_root(w) + 4 * U32) * (d * u).abs(), (d * u).abs())]
        summed("dgate", *sums, gate)
    gt = gates(gate, rows)
    du, du_off = d * gt, d_off * gt.abs() + U32 * (d * gt).abs()
    if after is None:
        db, db_off = du, du_off
    else:
        db, db_off, da, da_off, mag = back(du, du_off, b, wa)
        summed("dblock_weight", da, da_off, mag, after)
    out["dblock"] = db, db_off + 2 * U32 * db.abs() + rounded(db, dt) + 1e-30
    return out
