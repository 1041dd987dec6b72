"""Activations of products whose results are quantised: the definition's values
but for what float32 costs, not for what 16 bits would hide.

The sums are zero, so that the values before the activation are the biases and
every error is the activation's.  Bounds, with u = 2^-24 (half a step of
float32 is u of a value): the hardware's power of two is documented to 2^-22 =
4 u and its reciprocal to one ulp, 2 u.

  silu  z / (1 + exp(-z)): the exponential 4 u, its argument a product and a constant
        that is off by less than u / 4, 1.25 u of z, which the quotient does not
        magnify; a sum u, the reciprocal 2 u, a product u.  8 u + 1.25 |z| u.
  gelu  the tail Phi(-|z|) = t P(t) exp(-z^2 / 2): t P(t) with t as rounded 6.5 u (measured
        on the CPU over the whole range, in float32 steps), the reciprocal in t 2 u, the
        exponential 4 u, its argument two products and that constant, 2.5 u of z^2 / 2;
        two products and max(z, 0) - |z| Phi are 3 u, and |z| Phi at most the result.  16 u + 1.25 z^2 u.
Below float32's normal range the exponential and the tail are off by up to
4 of its smallest steps, 2^-149, which |z| multiplies.
"""
import pytest

import lsd_radix_sort_key_gb300 as rs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from block_util import E4M3, E8M0, round_e4m3, scale_of, values  # noqa: E402
from expert_util import DEV, TYPES, act64, gen  # noqa: E402

U = 2.0**-24


@pytest.fixture(scope="module", autouse=True)
def built():
    rs.build()
    rs.lib()


def bound(z, y, act):
    if act == "silu":
        return (8 + 1.25 * z.abs()) * U * y.abs() + 4 * 2.0**-149 * z.abs()
    if act == "gelu":
        return (16 + 1.25 * z * z) * U * y.abs() + 4 * 2.0**-149 * z.abs()
    return torch.zeros_like(y)


def zeros(rows, inner, experts, outer):
    """Operands whose products are zero, with scales of one."""
    def ones(*shape):
        return torch.full(shape, 127, dtype=torch.uint8, device=DEV).view(E8M0)

    def none(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device=DEV).view(E4M3)

    n, m = -(-inner // 128), -(-outer // 128)
    return none(rows, inner), ones(rows, n), none(experts, outer, inner), ones(experts, m, n)


# What a block of 128 values may hold; a block far below zero has a scale of its own.
RANGES = {"none": [(-3, 3), (-1000, 1000), (1e-6, 1e-3)], "relu": [(-3, 3), (-1000, 1000), (1e-6, 1e-3)],
          "gelu": [(-3, 3), (-0.01, 0.01), (-4, -2), (-6, -4), (-9, -6), (-12.5, -9), (-13.5, -13), (3, 20)],
          "silu": [(-3, 3), (-0.01, 0.01), (-9, -5), (-30, -9), (-80, -30), (-87, -80), (-91, -88), (3, 200)]}


@pytest.mark.parametrize("rows", [40, 4096])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", RANGES)
def test_values_before_the_rounding_are_float32(act, dt, rows):
    experts, ranges, g = 4, RANGES[act], gen(rows)
    outer = 128 * 2 * len(ranges) + 72
    span = torch.tensor([ranges[i // 128 % len(ranges)] for i in range(outer)], dtype=torch.float64, device=DEV)
    z = span[:, 0] + (span[:, 1] - span[:, 0]) * torch.rand(experts, outer, device=DEV, generator=g, dtype=torch.float64)
    z = z.to(TYPES[dt])
    x, xs, w, ws = zeros(rows, 256, experts, outer)
    offsets = torch.arange(experts + 1, dtype=torch.int32, device=DEV) * (rows // experts)
    q, scales = rs.expert_matmul_quantized(x, xs, w, ws, offsets, bias=z, activation=act, dtype=TYPES[dt], quantize=True)
    # every row of an expert is the same
    every = rows // experts
    for t in (q, scales):
        t = t.view(torch.uint8).view(experts, every, -1)
        assert torch.equal(t, t[:, :1].expand_as(t))
    q, scales = q[::every].double(), scales[::every].double()
    y = act64(z.double(), act)
    off = bound(z.double(), y, act)
    pad = -outer % 128

    def largest(t):
        return torch.nn.functional.pad(t.clamp(min=0), (0, pad)).view(experts, -1, 128).amax(2)

    low, high = scale_of(largest(y.abs() - off)), scale_of(largest(y.abs() + off))
    assert bool(((scales == low) | (scales == high)).all())
    s = scales.repeat_interleave(128, 1)[:, :outer]
    a, b = round_e4m3((y - off) / s), round_e4m3((y + off) / s)
    assert bool(((a <= q) & (q <= b)).all())
    assert bool((values(q, scales).abs().amax() > 0))


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_infinities_and_nan_before_the_rounding(act):
    # infinity becomes NaN; far below zero nothing is left, and the scale is the finite values'
    z = torch.zeros(1, 256, dtype=torch.bfloat16, device=DEV)
    z[0, :4] = torch.tensor([float("inf"), float("nan"), -3e38, -1e20])
    z[0, 4] = 3.0
    x, xs, w, ws = zeros(300, 128, 1, 256)
    q, scales = rs.expert_matmul_quantized(x, xs, w, ws, torch.tensor([0, 300], dtype=torch.int32, device=DEV), bias=z,
                                           activation=act, quantize=True)
    q = q.double()
    assert bool(torch.isnan(q[:, :2]).all()) and bool((q[:, 2:4] == 0).all()) and bool((q[:, 5:] == 0).all())
    want = act64(torch.tensor([3.0], dtype=torch.float64, device=DEV), act)
    assert bool((scales[:, 0].double() == scale_of(want)).all()) and bool((scales[:, 1].double() == 1).all())
    assert bool((q[:, 4] == round_e4m3(want / scale_of(want))).all())


@pytest.mark.parametrize("rows", [40, 4096])
@pytest.mark.parametrize("outer", [520, 1000, 72])
def test_blocks_of_zeros_have_a_scale_of_one(rows, outer):
    # rows of an expert, not unused ones: zero sums, and sums that relu makes zero
    x, xs, w, ws = zeros(rows, 256, 2, outer)
    offsets = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device=DEV)
    for act in ("none", "relu", "gelu", "silu"):
        q, scales = rs.expert_matmul_quantized(x, xs, w, ws, offsets, activation=act, quantize=True)
        assert bool((q.double() == 0).all()) and bool((scales.view(torch.uint8) == 127).all())
    g = gen(outer)
    x = (torch.randn(rows, 256, device=DEV, generator=g) * 60).to(E4M3)
    w = (torch.randn(2, outer, 256, device=DEV, generator=g) * 60).to(E4M3)
    # sums of at most 256 * 448 * 448 < 2^26 with a bias far below them in every other block
    blocks = torch.arange(outer, device=DEV) // 128
    for gone in (0, 1):
        bias = torch.where(blocks % 2 == gone, -2.0**30, 0.0).expand(2, outer).bfloat16()
        q, scales = rs.expert_matmul_quantized(x, xs, w, ws, offsets, bias=bias, activation="relu", quantize=True)
        live = torch.arange(scales.shape[1], device=DEV) % 2 != gone
        assert bool((scales.view(torch.uint8)[:, ~live] == 127).all()) and bool((q.double()[:, blocks % 2 == gone] == 0).all())
        # the other blocks hold something, but where every sum of a few columns is negative
        held = torch.nn.functional.pad(q.double(), (0, -outer % 128)).view(rows, -1, 128).amax(2) > 0
        assert bool((scales.view(torch.uint8)[~held] == 127).all())
        assert int(held[:, live].sum()) >= 0.9 * held[:, live].numel()


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_values_do_not_depend_on_their_neighbours(act):
    # values far below zero take a longer way, and leave those beside them as they are
    g = gen(8)
    z = torch.randn(1, 512, device=DEV, generator=g).bfloat16()
    x, xs, w, ws = zeros(300, 128, 1, 512)
    offsets = torch.tensor([0, 300], dtype=torch.int32, device=DEV)
    want = rs.expert_matmul_quantized(x, xs, w, ws, offsets, bias=z, activation=act, quantize=True)[0]
    deep = z.clone()
    deep[0, 5::16] = -95.0 if act == "silu" else -13.5
    got = rs.expert_matmul_quantized(x, xs, w, ws, offsets, bias=deep, activation=act, quantize=True)[0]
    same = torch.ones(512, dtype=torch.bool, device=DEV)
    same[5::16] = False
    assert torch.equal(got.view(torch.uint8)[:, same], want.view(torch.uint8)[:, same])
