"""The sums of the norms' rows, to within what their order costs whatever the width,
so that a row which lost one ordinary element is seen.

With u = 2^-24.  A thread adds at most 8 pairs, then its two halves (1), then come
5 exchanges in the warp and at most 32 warps' sums, four at a time (2 + 8): a
term goes through at most 24 roundings.  So a sum of squares is off by 24 u of
itself, the mean plus eps by 26 u (the factor 1 / W and a rounding), and r = 1 /
sqrt by half of that and the root's documented 2 ulps, 4 u: 17 u, taken as 18.  A
lost element of ordinary size is 1 / (2 W) of r, 512 u at the greatest width.
<g, v> is off by 25 u of its terms' magnitudes, g = d w having one rounding.
"""
import pytest

import lsd_radix_sort_key_gb300 as rs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from expert_util import DEV, TYPES, gen, held, rounded  # noqa: E402

U = 2.0**-24
R = 18 * U
EPS = 1e-6
WIDTHS = [1, 7, 64, 129, 256, 513, 1037, 2047, 2048, 4096, 4097, 8184, 8191, 8192, 12001, 16383, 16384]


@pytest.fixture(scope="module", autouse=True)
def built():
    rs.build()
    rs.lib()


def inverse_root(v):
    return torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)


def normal(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def back(g, g_off, v):
    """The gradient of rms(v) for v, given g, and its error, g being off by g_off of itself."""
    r = inverse_root(v)
    n, dot, mag = v * r, (g * v).mean(1, keepdim=True), (g * v).abs().mean(1, keepdim=True)
    c = r * dot
    value = r * (g - n * c)
    off = r * (g.abs() * g_off + (n * c).abs() * (2 * R + 4 * U) + (n * r).abs() * mag * (24 * U + g_off))
    return value, off + (R + 2 * U) * r * (g.abs() + (n * c).abs())


@pytest.mark.parametrize("width", WIDTHS)
def test_norms_in_32_bits(width):
    g = gen(width)
    x, b = normal(g, 37, width), normal(g, 37, width)
    w, after, gate = (1 + 0.3 * normal(g, width) for _ in range(3))
    want = x.double() * inverse_root(x.double()) * w.double()
    held(rs.expert_norm(x, w), want, (R + 3 * U) * want.abs() + 1e-30)
    y, h = rs.expert_norm(x, w, block=b, block_weight=after, gate=gate, residual_scale=0.75)
    part = gate.double() * b.double() * inverse_root(b.double()) * after.double()
    want = 0.75 * x.double() + part
    held(y, want, (R + 4 * U) * part.abs() + 2 * U * want.abs() + 1e-30)
    want = y.double() * inverse_root(y.double()) * w.double()
    held(h, want, (R + 3 * U) * want.abs() + 1e-30)


@pytest.mark.parametrize("width", WIDTHS)
def test_gradients_in_32_bits(width):
    g = gen(width + 1)
    y, b, dh, dy = (normal(g, 37, width) for _ in range(4))
    w, after, gate = (1 + 0.3 * normal(g, width) for _ in range(3))
    # without a block, and the block's own norm alone
    want, off = back(dh.double() * w.double(), U, y.double())
    want = want + dy.double()
    held(rs.expert_norm_grad(dh, y, w, dy=dy)[0], want, off + 2 * U * want.abs() + 1e-30)
    want, off = back(dy.double() * gate.double() * after.double(), 2 * U, b.double())
    got = rs.expert_norm_grad(None, y, None, dy=dy, block=b, block_weight=after, gate=gate)[2]
    held(got, want, off + 2 * U * want.abs() + 1e-30)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("width", [129, 264, 1037, 2048, 4104, 8191, 8192, 12001, 16384])
def test_every_column_counts(dt, width):
    # nearly all of a row is one element, another in each row: lost, it would be seen in any type
    dtype, g = TYPES[dt], gen(width)
    at = torch.arange(width, device=DEV) if width <= 2048 else torch.cat(
        [torch.arange(64, device=DEV), torch.arange(64, width - 64, 13, device=DEV), torch.arange(width - 64, width, device=DEV)])
    rows = torch.arange(at.numel(), device=DEV)
    x = (0.1 * normal(g, at.numel(), width)).to(dtype)
    x[rows, at] = 30.0
    w, after = (1 + 0.3 * normal(g, width) for _ in range(2))
    want = x.double() * inverse_root(x.double()) * w.double()
    bound = (R + 3 * U) * want.abs() + rounded(want, dtype) + 1e-30
    held(rs.expert_norm(x, w), want, bound)
    y, _ = rs.expert_norm(torch.zeros_like(x), w, block=x, block_weight=after)
    want = x.double() * inverse_root(x.double()) * after.double()
    held(y, want, (R + 4 * U) * want.abs() + rounded(want, dtype) + 1e-30)
    # the gradients: dh is one element too, at the same place, so that <g, v> is it
    dh = torch.zeros_like(x)
    dh[rows, at] = 2.0
    want, off = back(dh.double() * w.double(), U, x.double())
    held(rs.expert_norm_grad(dh, x, w)[0], want, off + 2 * U * want.abs() + rounded(want, dtype) + 1e-30)
    want, off = back(dh.double() * after.double(), 2 * U, x.double())
    got = rs.expert_norm_grad(None, x, None, dy=dh, block=x, block_weight=after)[2]
    held(got, want, off + 2 * U * want.abs() + rounded(want, dtype) + 1e-30)
