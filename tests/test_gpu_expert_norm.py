"""The norms around an expert block and their gradients against 64 bits."""
import pytest

import lsd_radix_sort_key_gb300 as rs
from lsd_radix_sort_key_gb300 import experts

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from block_util import plain_norm, plain_norm_grad  # noqa: E402
from expert_util import DEV, TYPES, gen, held  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    rs.build()
    rs.lib()


@pytest.fixture(params=["extension", "python"])
def way(request, monkeypatch):
    """Both forms of a call."""
    experts._torch()
    assert experts._fast is not None
    if request.param == "python":
        monkeypatch.setattr(experts, "_fast", None)


def inputs(rows, width, dt, params="f32", block=True, after=True, gate=1, weight=True, seed=1):
    """x, weight, block, after, gate; gate: -1 none, 0 one row without a dimension, else rows of gates."""
    g, dtype, pt = gen(seed + rows + width), TYPES[dt], TYPES[params]

    def normal(*shape, scale=1.0, to=dtype):
        return (torch.randn(*shape, device=DEV, generator=g) * scale).to(to)

    x = (normal(rows, width, to=torch.float32) * torch.exp(normal(rows, 1, to=torch.float32))).to(dtype)
    ws = [(1 + normal(width, scale=0.3, to=torch.float32)).to(pt) for _ in range(2)]
    gates = None if gate < 0 or not block else normal(*((width,) if gate == 0 else (gate, width)), to=pt)
    return (x, ws[0] if weight else None, normal(rows, width, scale=0.5) if block else None,
            ws[1] if block and after else None, gates)


def check(x, weight, block, after, gate, scale=0.7, eps=1e-6):
    if block is None:
        y, h = None, rs.expert_norm(x, weight, eps=eps)
    else:
        y, h = rs.expert_norm(x, weight, block=block, block_weight=after, gate=gate, residual_scale=scale, eps=eps)
    want_y, y_bound, want_h, h_bound = plain_norm(x, weight, block, after, gate, scale, eps, y)
    if block is not None:
        assert y.dtype == x.dtype
        held(y, want_y, y_bound)
    if weight is None:
        assert h is None
    else:
        assert h.dtype == x.dtype
        held(h, want_h, h_bound)


NAMES = ("dx", "dweight", "dblock", "dblock_weight", "dgate")


def check_grad(y, weight, block, after, gate, dh, dy, scale=0.7, eps=1e-6):
    got = rs.expert_norm_grad(dh, y, weight, dy=dy, block=block, block_weight=after, gate=gate, residual_scale=scale, eps=eps)
    want = plain_norm_grad(dh, y, weight, dy, block, after, gate, scale, eps)
    for name, t in zip(NAMES, got):
        if t is None:
            assert name not in want
            continue
        like = {"dweight": weight, "dblock_weight": after, "dgate": gate}.get(name, y)
        assert t.dtype == like.dtype and t.shape == like.shape
        held(t, *want[name])


SIZES = [(1, 1), (1, 8), (3, 7), (5, 64), (2, 129), (64, 4096), (33, 1032), (9, 1037), (700, 256), (4, 8192), (3, 8191), (2, 16384),
         (3, 12001), (1001, 520), (2500, 2048), (620, 513)]


@pytest.mark.parametrize("dt,params", [("f32", "f32"), ("f16", "f32"), ("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,width", SIZES)
def test_norms(way, dt, params, rows, width):
    check(*inputs(rows, width, dt, params, block=False))
    check(*inputs(rows, width, dt, params))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("after", [False, True])
@pytest.mark.parametrize("gate", [-1, 0, 1, 3, 12, 36])
@pytest.mark.parametrize("width", [72, 1037])
def test_every_part_may_be_absent(way, dt, after, gate, width):
    for weight in (True, False):
        x, w, b, a, g = inputs(36, width, dt, dt, after=after, gate=gate, weight=weight)
        check(x, w, b, a, g, scale=-1.25)
        dh = torch.randn(36, width, device=DEV, generator=gen(9)).to(x.dtype) if weight else None
        dy = torch.randn(36, width, device=DEV, generator=gen(10)).to(x.dtype)
        check_grad(x, w, b, a, g, dh, dy, scale=-1.25)
        if weight:
            check_grad(x, w, b, a, g, dh, None, scale=-1.25)
            check_grad(x, w, None, None, None, dh, dy)


@pytest.mark.parametrize("dt,params", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,width", SIZES)
def test_gradients(way, dt, params, rows, width):
    x, w, b, a, g = inputs(rows, width, dt, params)
    dh, dy = (torch.randn(rows, width, device=DEV, generator=gen(s)).to(x.dtype) for s in (5, 6))
    check_grad(x, w, b, a, g, dh, dy)
    check_grad(x, w, None, None, None, dh, None)


@pytest.mark.parametrize("rows,gate", [(4096, 1), (4096, 8), (4096, 256), (4096, 1024), (4096, 4096), (3000, 3), (3000, 750),
                                       (1217, 1217), (1300, 13), (40, 40), (9, 3)])
@pytest.mark.parametrize("width", [64, 1040])
def test_gates_of_many_sequences(rows, gate, width):
    # gate rows whole in a block, shared by two, and shared by many
    x, w, b, a, g = inputs(rows, width, "bf16", "f32", gate=gate)
    check(x, w, b, a, g)
    dh, dy = (torch.randn(rows, width, device=DEV, generator=gen(s)).bfloat16() for s in (5, 6))
    check_grad(x, w, b, a, g, dh, dy)


def test_gradients_against_differences():
    # of the formula in 64 bits, which the other tests hold the kernels to
    x, w, b, a, g = (t.cpu().double() for t in inputs(6, 24, "f32", gate=3))
    dh, dy = (torch.randn(6, 24, device=DEV, generator=gen(s)).cpu().double() for s in (5, 6))
    scale, eps, step = 0.7, 1e-3, 1e-6

    def loss(x, w, b, a, g):
        u = b / torch.sqrt(b.square().mean(1, keepdim=True) + eps) * a
        y = scale * x + g.repeat_interleave(2, 0) * u
        h = y / torch.sqrt(y.square().mean(1, keepdim=True) + eps) * w
        return (dh * h).sum() + (dy * y).sum(), y

    y = loss(x, w, b, a, g)[1].to(DEV)
    got = rs.expert_norm_grad(dh.to(DEV).float(), y.float(), w.to(DEV).float(), dy=dy.to(DEV).float(), block=b.to(DEV).float(),
                              block_weight=a.to(DEV).float(), gate=g.to(DEV).float(), residual_scale=scale, eps=eps)
    for i, (t, name) in enumerate(((x, "dx"), (w, "dweight"), (b, "dblock"), (a, "dblock_weight"), (g, "dgate"))):
        flat = t.view(-1)
        for j in range(0, flat.numel(), 5):
            kept = flat[j].item()
            flat[j] = kept + step
            up = loss(x, w, b, a, g)[0]
            flat[j] = kept - step
            low = loss(x, w, b, a, g)[0]
            flat[j] = kept
            diff = float(up - low) / (2 * step)
            # differences: 1e-6 squared and 1e-16 / 1e-6 of sums up to 1e3; float32: some hundred 2^-24
            assert abs(float(got[NAMES.index(name)].view(-1)[j]) - diff) < 2e-4 * max(1.0, abs(diff)), (name, j)


@pytest.mark.parametrize("dt", TYPES)
def test_strides_and_one_row_for_all(way, dt):
    dtype, g = TYPES[dt], gen(3)
    big = torch.randn(5, 60, 700, device=DEV, generator=g).to(dtype)
    _, w, _, a, _ = inputs(1, 264, dt, dt)
    gate = torch.randn(30, 264, device=DEV, generator=g).to(dtype)[::3]  # (made contiguous by the call)
    for cut in (lambda t: t[:50, 8:272], lambda t: t[:50, 1:265], lambda t: t[:50, 400:664], lambda t: t[3:4, 16:280].expand(50, 264)):
        x, b, dh, dy = (cut(big[i]) for i in range(4))
        check(x, w, b, a, gate)
        check_grad(x, w, b, a, gate, dh, dy)
    check(big[0, :50, 8:272], w, big[1, :50, 1:265], a, gate)  # one aligned, one not
    wide = torch.randn(300, device=DEV, generator=g).to(dtype)
    check(big[0, :50, 8:272], wide[3:267], big[1, :50, 8:272], wide[8:272], gate)


def test_a_zero_row_and_eps():
    x, w, b, a, g = inputs(6, 264, "bf16")
    x[2], b[3] = 0, 0
    for eps in (1e-6, 1e-2, 1.0):
        check(x, w, b, a, g, eps=eps)
        check(x, w, None, None, None, eps=eps)
    h = rs.expert_norm(x, w, eps=0.0)
    assert bool(torch.isnan(h[2]).all()) and not bool(torch.isnan(h[3]).any())  # 0 / 0, as the formula says


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("power", [-46, 46])
@pytest.mark.parametrize("width", [264, 1037])
def test_rows_of_extreme_magnitude(dt, power, width):
    # r^3 is 2^138 or 2^-138, outside float32's range; the squares and every result are inside
    x, w, b, a, g = inputs(24, width, dt)
    x, b = x * 2.0**power, b * 2.0**power
    check(x, w, b, a, g, scale=2.0**-power, eps=0.0)
    check(x, w, None, None, None, eps=0.0)
    dh, dy = (torch.randn(24, width, device=DEV, generator=gen(s)).to(x.dtype) for s in (5, 6))
    check_grad(x, w, b, a, g, dh, dy * 2.0**-power, eps=0.0)
    check_grad(x, w, None, None, None, dh, None, eps=0.0)


def test_nan_and_infinity_stay_in_their_rows():
    x, w, b, a, g = inputs(40, 1037, "f32")
    x[3, 5], b[7, 900], x[9, 0] = float("nan"), float("inf"), float("inf")
    y, h = rs.expert_norm(x, w, block=b, block_weight=a, gate=g)
    bad = torch.zeros(40, dtype=torch.bool, device=DEV)
    bad[[3, 7, 9]] = True
    assert not bool(torch.isnan(h[~bad]).any()) and not bool(torch.isnan(y[~bad]).any())
    assert bool(torch.isnan(h[3]).all()) and bool(torch.isnan(h[9, 0]))
    dh = torch.randn(40, 1037, device=DEV, generator=gen(1))
    dx, _, db, _, _ = rs.expert_norm_grad(dh, y, w, block=b, block_weight=a, gate=g)
    assert not bool(torch.isnan(dx[~bad]).any()) and not bool(torch.isnan(db[~bad]).any())


@pytest.mark.parametrize("dt", TYPES)
def test_no_rows(way, dt):
    x, w, b, a, g = inputs(0, 264, dt, gate=0)
    y, h = rs.expert_norm(x, w, block=b, block_weight=a, gate=g)
    assert y.shape == h.shape == (0, 264)
    got = rs.expert_norm_grad(x, x, w, dy=x, block=b, block_weight=a, gate=g)
    assert got[0].shape == (0, 264) and got[2].shape == (0, 264)
    assert all(bool((t == 0).all()) and t.shape == (264,) for t in (got[1], got[3], got[4]))


def test_sums_do_not_depend_on_timing_and_calls_can_be_captured():
    x, w, b, a, g = inputs(5000, 1040, "bf16", gate=8)
    dh, dy = (torch.randn(5000, 1040, device=DEV, generator=gen(s)).bfloat16() for s in (5, 6))

    def both():
        return (*rs.expert_norm(x, w, block=b, block_weight=a, gate=g),
                *rs.expert_norm_grad(dh, x, w, dy=dy, block=b, block_weight=a, gate=g))

    first = both()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        out = both()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, first))
    other = torch.cuda.Stream()
    got = rs.expert_norm_grad(dh, x, w, dy=dy, block=b, block_weight=a, gate=g, stream=other)
    other.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, first[2:]))


def test_parameters_are_copied_on_the_stream_that_reads_them():
    # strided parameters on another stream, which is busy when the call is made
    g = gen(4)
    x, b = (torch.randn(200, 264, device=DEV, generator=g).bfloat16() for _ in range(2))
    wide = torch.randn(3, 528, device=DEV, generator=g)
    w, a, gate = (wide[i, ::2] for i in range(3))
    want = rs.expert_norm(x, w, block=b, block_weight=a, gate=gate)
    grad = rs.expert_norm_grad(x, want[0], w, dy=b, block=b, block_weight=a, gate=gate)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kept = wide.clone()
    with torch.cuda.stream(side):
        wide.zero_()
        torch.cuda._sleep(100_000_000)
        wide.copy_(kept)
    got = rs.expert_norm(x, w, block=b, block_weight=a, gate=gate, stream=side)
    got_grad = rs.expert_norm_grad(x, want[0], w, dy=b, block=b, block_weight=a, gate=gate, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*got, *got_grad), (*want, *grad)))


def test_numbers(way):
    x, w, b, a, g = inputs(6, 264, "f32")
    check(x, w, b, a, g, scale=2)
    check(x, w, b, a, g, scale=0.0)
    with pytest.raises(TypeError):
        rs.expert_norm(x, w, block=b, residual_scale=torch.ones((), device=DEV))
    with pytest.raises(TypeError):
        rs.expert_norm(x, w, eps=torch.ones((), device=DEV))
    for number in (1e300, float("inf"), float("nan")):
        with pytest.raises(rs.RadixSortError):
            rs.expert_norm(x, w, block=b, residual_scale=number)
    for eps in (-1.0, float("inf"), float("nan")):
        with pytest.raises(rs.RadixSortError):
            rs.expert_norm(x, w, eps=eps)


def test_refusals(way):
    x, w, b, a, g = inputs(12, 264, "bf16", gate=4)
    for error, call in [
            (ValueError, lambda: rs.expert_norm(x, w[:200])), (TypeError, lambda: rs.expert_norm(x, w.half())),
            (ValueError, lambda: rs.expert_norm(x, w.cpu())), (ValueError, lambda: rs.expert_norm(x.T, w)),
            (ValueError, lambda: rs.expert_norm(x, w, gate=g)), (ValueError, lambda: rs.expert_norm(x, w, block_weight=a)),
            (ValueError, lambda: rs.expert_norm(x, w, block=b[:6])), (TypeError, lambda: rs.expert_norm(x, w, block=b.float())),
            (TypeError, lambda: rs.expert_norm(x, w, block=b, block_weight=a.bfloat16())),
            (ValueError, lambda: rs.expert_norm(x, w, block=b, gate=g.repeat(2, 1)[:5])),
            (ValueError, lambda: rs.expert_norm(x, w, block=b, gate=g[:0])),
            (ValueError, lambda: rs.expert_norm_grad(x[:6], x, w)), (TypeError, lambda: rs.expert_norm_grad(x, x, None, dy=x, block=b)),
            (TypeError, lambda: rs.expert_norm_grad(None, x, None, block=b)),
            (rs.RadixSortError, lambda: rs.expert_norm(x.new_zeros(2, 16392), w.new_zeros(16392)))]:
        with pytest.raises(error):
            call()


def test_long_matrices():
    # past 2^31 elements: the last rows are theirs
    rows, width = (1 << 19) + 3, 4104
    x = torch.full((rows, width), 0.5, dtype=torch.bfloat16, device=DEV)
    x[-40:] = torch.randn(40, width, device=DEV, generator=gen(2)).bfloat16()
    w = 1 + 0.1 * torch.randn(width, device=DEV, generator=gen(3))
    h = rs.expert_norm(x, w)
    _, _, want, bound = plain_norm(x[-40:], w, None, None, None, 1.0, 1e-6)
    held(h[-40:], want, bound)
    dx, dw, _, _, _ = rs.expert_norm_grad(h, x, w)
    want = plain_norm_grad(h[-40:], x[-40:], w, None, None, None, None, 1.0, 1e-6)
    held(dx[-40:], *want["dx"])
