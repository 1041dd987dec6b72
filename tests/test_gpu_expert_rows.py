"""expert_sort, expert_dispatch, expert_combine and their gradients on the
GPU against plain forms (whole numbers: equal; sums: 64 bits, bounds in
expert_util)."""
import pytest

import lsd_radix_sort_key_gb300 as rs
from lsd_radix_sort_key_gb300 import experts

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from expert_util import (ADD, DEV, TYPES, gen, held, make_plan, plain_combine, plain_combine_grad,  # noqa: E402
                         plain_dispatch, plain_order, rounded)


@pytest.fixture(scope="module", autouse=True)
def built():
    rs.build()
    rs.lib()
    experts._torch()
    assert experts._fast is not None  # the extension is part of the build


@pytest.fixture(params=["extension", "python"])
def way(request, monkeypatch):
    """Both forms of a call: the extension's, and the one in Python."""
    if request.param == "python":
        monkeypatch.setattr(experts, "_fast", None)


def check_sort(ids, experts):
    got = rs.expert_sort(ids, experts)
    want = plain_order(ids, experts)
    for name, g, w in zip(("order", "position", "offsets"), got, want):
        assert g.dtype == torch.int32 and torch.equal(g.cpu(), w), name


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 255, 256, 257, 511, 513, 4095, 4096, 4097, 8191, 8193, 16385, 65537,
                               300_001, 1_000_003])
@pytest.mark.parametrize("experts", [1, 2, 7, 64, 257])
def test_sort_sizes(n, experts):
    ids = torch.randint(0, experts, (n,), device=DEV, generator=gen(n + experts))
    check_sort(ids, experts)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,slots,experts", [(1, 1, 1), (1, 8, 128), (64, 8, 1024), (777, 6, 1023), (5003, 4, 512),
                                                  (40_000, 8, 1024)])
def test_sort_types_and_dropped(way, dtype, tokens, slots, experts):
    g = gen(tokens)
    ids = torch.randint(0, experts, (tokens, slots), device=DEV, generator=g)
    ids[torch.rand(tokens, slots, device=DEV, generator=g) < 0.3] = -1
    ids[torch.rand(tokens, slots, device=DEV, generator=g) < 0.05] = experts
    check_sort(ids.to(dtype), experts)


@pytest.mark.parametrize("experts", [1, 5, 1024])
def test_sort_extreme_ids(experts):
    # numbers whose low 32 bits alone would look like an expert are dropped too
    v = [0, -1, experts, experts - 1, 2**31, 2**32, 2**32 + 1, -2**32, 2**63 - 1, -2**63]
    check_sort(torch.tensor(v * 50, device=DEV), experts)
    check_sort(torch.tensor([-2**31, 2**31 - 1, 0, -1, experts] * 50, device=DEV, dtype=torch.int32), experts)


@pytest.mark.parametrize("n", [5, 4096, 100_000])
def test_sort_one_expert_takes_all_or_nothing_is_kept(n):
    check_sort(torch.full((n,), 3, device=DEV), 8)
    check_sort(torch.full((n,), -1, device=DEV), 8)
    check_sort(torch.arange(n, device=DEV) % 8, 8)
    check_sort((n - 1 - torch.arange(n, device=DEV)) * 8 // n, 8)


def test_sort_nothing(way):
    order, position, offsets = rs.expert_sort(torch.empty(0, 4, dtype=torch.int64, device=DEV), 6)
    assert order.shape == (0,) and position.shape == (0, 4) and offsets.tolist() == [0] * 7


WIDTHS = [1, 7, 8, 33, 64, 71, 105, 128, 129, 256, 1000, 1032, 2048, 4097]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("tokens,slots,drop", [(1, 1, 0.0), (1, 8, 0.5), (67, 3, 0.2), (1025, 6, 0.1), (300, 11, 0.1)])
def test_rows(dt, width, tokens, slots, drop):
    dtype, g = TYPES[dt], gen(width * 7 + tokens)
    position, offsets = make_plan(tokens, slots, 16, width + tokens, drop)
    x = torch.randn(tokens, width, device=DEV, generator=g).to(dtype)
    assert torch.equal(rs.expert_dispatch(x, position, offsets).double(), plain_dispatch(x, position, offsets))
    y = torch.randn(tokens * slots, width, device=DEV, generator=g).to(dtype)
    y[int(offsets[-1]):] = float("nan")  # dropped rows are not read
    want, mag = plain_combine(y, None, position, offsets)
    held(rs.expert_dispatch_grad(y, position, offsets), want, slots * ADD * mag + rounded(want, dtype))
    dout = torch.randn(tokens, width, device=DEV, generator=g).to(dtype)
    for wtype in {torch.float32, dtype}:
        weights = torch.rand(tokens, slots, device=DEV, generator=g).to(wtype)
        want, mag = plain_combine(y, weights, position, offsets)
        held(rs.expert_combine(y, weights, position, offsets), want, (slots + 1) * ADD * mag + rounded(want, dtype))
        dy, dw = rs.expert_combine_grad(dout, y, weights, position, offsets)
        want, want_w, mag = plain_combine_grad(dout, y, weights, position, offsets)
        assert dy.dtype == dtype and dw.dtype == wtype
        held(dy, want, want.abs() * ADD + rounded(want, dtype))
        held(dw, want_w, (width + 1) * ADD * mag + rounded(want_w, wtype))

@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("width", [1, 63, 64, 65, 71, 96, 129, 136, 160, 185, 192, 193, 255, 257, 777])
@pytest.mark.parametrize("tokens,slots", [(2047, 3), (2049, 2), (2111, 9)])
def test_rows_of_many_tokens(dt, width, tokens, slots):
    test_rows(dt, width, tokens, slots, 0.1)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("width", [1000, 1001])
def test_rows_strided_and_offset(way, dt, width):
    # rows inside a wider matrix, at an offset that is not 16-byte aligned, and one row for all
    dtype, g = TYPES[dt], gen(3)
    tokens, slots = 129, 4
    position, offsets = make_plan(tokens, slots, 8, 5, 0.1)
    wide = torch.randn(tokens * slots, width + 24, device=DEV, generator=g).to(dtype)
    weights = torch.rand(tokens, slots, device=DEV, generator=g)
    for first in (0, 8, 3):
        view = wide[:, first:first + width]
        assert torch.equal(rs.expert_dispatch(view[:tokens], position, offsets),
                           rs.expert_dispatch(view[:tokens].contiguous(), position, offsets))
        assert torch.equal(rs.expert_combine(view, weights, position, offsets),
                           rs.expert_combine(view.contiguous(), weights, position, offsets))
    one = wide[:1, :width].expand(tokens, width)
    assert torch.equal(rs.expert_dispatch(one, position, offsets),
                       rs.expert_dispatch(one.contiguous(), position, offsets))
    # the gradient of a sum over a token's row: one row of dout for all tokens
    y = wide[:, 8:8 + width]
    for got, want in zip(rs.expert_combine_grad(one, y, weights, position, offsets),
                         rs.expert_combine_grad(one.contiguous(), y.contiguous(), weights, position, offsets)):
        held(got, want.double(), want.double().abs() * 0 + 1e-30 if got.dim() == 2 and got.shape[1] == width
             else (width + 1) * 2 * ADD * y.double().abs().max() * one.double().abs().sum(1)[:, None])
    strided_w = torch.rand(tokens, 2 * slots, device=DEV, generator=g)[:, ::2]
    assert torch.equal(rs.expert_combine(y, strided_w, position, offsets),
                       rs.expert_combine(y, strided_w.contiguous(), position, offsets))


@pytest.mark.parametrize("width", [64, 65])
def test_infinities_and_nan_stay_in_their_tokens(width):
    position, offsets = make_plan(40, 3, 4, 9, 0.2)
    y = torch.randn(120, width, device=DEV, generator=gen(1))
    weights = torch.rand(40, 3, device=DEV, generator=gen(2))
    y[int(position[5, 1])] = float("inf")
    y[int(position[6, 0])] = float("nan")
    weights[7] = 0.0
    want, mag = plain_combine(y, weights, position, offsets)
    held(rs.expert_combine(y, weights, position, offsets), want, torch.nan_to_num(4 * ADD * mag, 0, 0) + 1e-30)


def test_all_slots_dropped_and_no_tokens(way):
    ids = torch.full((9, 4), -1, device=DEV)
    _, position, offsets = rs.expert_sort(ids, 5)
    x = torch.randn(9, 100, device=DEV)
    y = torch.full((36, 100), float("nan"), device=DEV)
    w = torch.rand(9, 4, device=DEV)
    assert not rs.expert_dispatch(x, position, offsets).any()
    assert not rs.expert_combine(y, w, position, offsets).any()
    dy, dw = rs.expert_combine_grad(x, y, w, position, offsets)
    assert not dy.any() and not dw.any()
    _, position, offsets = rs.expert_sort(ids[:0], 5)
    assert rs.expert_dispatch(x[:0], position, offsets).shape == (0, 100)
    assert rs.expert_combine(y[:0], w[:0], position, offsets).shape == (0, 100)
    assert rs.expert_combine_grad(x[:0], y[:0], w[:0], position, offsets)[0].shape == (0, 100)
    _, position, offsets = rs.expert_sort(ids, 5)
    dy, dw = rs.expert_combine_grad(x[:, :0], y[:, :0], w, position, offsets)  # a row of no elements
    assert dy.shape == (36, 0) and not dw.any()


@pytest.mark.parametrize("limit,bad", [(10**6, -1), (-5, 0), (36, 10**6)])
def test_a_wrong_plan_stays_inside_the_arrays(limit, bad):
    position, offsets = make_plan(9, 4, 5, 3)
    offsets[-1] = limit
    position[2, 1] = bad
    x, y, w = torch.randn(9, 64, device=DEV), torch.randn(36, 64, device=DEV), torch.rand(9, 4, device=DEV)
    rs.expert_dispatch(x, position, offsets)
    rs.expert_combine(y, w, position, offsets)
    rs.expert_combine_grad(x, y, w, position, offsets)
    torch.cuda.synchronize()
    assert rs.expert_sort(torch.zeros(3, dtype=torch.int64, device=DEV), 2)[2].tolist() == [0, 3, 3]


def test_gradients_against_differences():
    # combine is linear in y and in the weights: differences of the plain form are exact up to 64-bit rounding
    position, offsets = make_plan(23, 4, 6, 11, 0.15)
    g = gen(12)
    y, w = torch.randn(92, 40, device=DEV, generator=g), torch.rand(23, 4, device=DEV, generator=g)
    c = torch.randn(23, 40, device=DEV, generator=g)
    dy, dw = rs.expert_combine_grad(c, y, w, position, offsets)
    vy = torch.randn(y.shape, device=DEV, generator=g, dtype=torch.float64)
    vw = torch.randn(w.shape, device=DEV, generator=g, dtype=torch.float64)

    def value(h):
        return float((plain_combine(y.double() + h * vy, w.double() + h * vw, position, offsets)[0] * c).sum())

    slope = (value(1e-3) - value(-1e-3)) / 2e-3  # the second-order term cancels, there is no third
    got = float((dy.double() * vy).sum() + (dw.double() * vw).sum())
    size = float((dy.double() * vy).abs().sum() + 40 * (c.abs().max() * y.abs().max()) * vw.abs().sum())
    assert abs(got - slope) <= 42 * ADD * size + 1e-9 * size
    # dispatch: <dispatch(x), d> = <x, dispatch_grad(d)>
    x, d = torch.randn(23, 40, device=DEV, generator=g), torch.randn(92, 40, device=DEV, generator=g)
    left = float((rs.expert_dispatch(x, position, offsets).double() * d.double()).sum())
    right = float((x.double() * rs.expert_dispatch_grad(d, position, offsets).double()).sum())
    assert abs(left - right) <= 5 * ADD * float(x.abs().double().sum() * 4 * d.abs().max())


def test_another_stream_and_graph(way):
    position, offsets = make_plan(500, 4, 8, 21, 0.1)
    x = torch.randn(500, 264, device=DEV)
    w = torch.rand(500, 4, device=DEV)
    ids = torch.randint(-1, 8, (500, 4), device=DEV)
    want = (rs.expert_dispatch(x, position, offsets), rs.expert_sort(ids, 8)[0])
    want += (rs.expert_combine(want[0], w, position, offsets),)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        d = rs.expert_dispatch(x, position, offsets, stream=s)
        c = rs.expert_combine(d, w, position, offsets, stream=s)
        o = rs.expert_sort(ids, 8, stream=s)[0]
        side.synchronize()
        assert torch.equal(d, want[0]) and torch.equal(c, want[2]) and torch.equal(o, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, p, off = rs.expert_sort(ids, 8)
        d = rs.expert_dispatch(x, p, off)
        c = rs.expert_combine(d, w, p, off)
    ids.copy_(torch.randint(-1, 8, (500, 4), device=DEV))
    x.normal_()
    graph.replay()
    _, p2, off2 = rs.expert_sort(ids, 8)
    d2 = rs.expert_dispatch(x, p2, off2)
    assert torch.equal(d, d2) and torch.equal(c, rs.expert_combine(d2, w, p2, off2))


def test_positions_past_32_bit_offsets():
    # 2^31 + 2^30 elements in y: element offsets pass 32 bits
    tokens, slots, width = 3, 3 << 9, 1 << 20
    ids = torch.arange(tokens * slots, device=DEV).view(tokens, slots) % 5
    _, position, offsets = rs.expert_sort(ids, 5)
    x = torch.randn(tokens, width, device=DEV, generator=gen(4)).half()
    out = rs.expert_dispatch(x, position, offsets)
    assert out.numel() > 2**32
    for t, k in ((0, 0), (1, 700), (2, slots - 1)):
        assert torch.equal(out[int(position[t, k])], x[t])
    assert torch.equal(out[-1], x[2 if int(position[2].max()) == tokens * slots - 1 else
                                  [t for t in range(3) if int(position[t].max()) == tokens * slots - 1][0]])
    w = torch.zeros(tokens, slots, device=DEV)
    w[:, -1] = 1.0
    assert torch.equal(rs.expert_combine(out, w, position, offsets), x)


@pytest.mark.parametrize("n", [1000, 20_000, 32_768, 32_769, 200_000])
def test_sort_in_a_graph_and_beside_other_work(n):
    # one block, a cluster, a grid: captured, replayed on new numbers, and on two streams at once
    ids = torch.randint(-1, 60, (n,), device=DEV, generator=gen(n))
    rs.expert_sort(ids, 60)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rs.expert_sort(ids, 60)
    for seed in (1, 2):
        ids.copy_(torch.randint(-1, 61, (n,), device=DEV, generator=gen(n + seed)))
        graph.replay()
        for g, w in zip(got, plain_order(ids, 60)):
            assert torch.equal(g.cpu(), w)
    other = torch.randint(0, 60, (n,), device=DEV, generator=gen(n + 3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [(rs.expert_sort(ids, 60), rs.expert_sort(other, 60, stream=side)) for _ in range(20)]
    torch.cuda.synchronize()
    want = plain_order(ids, 60), plain_order(other, 60)
    for pair in outs:
        for got, w in zip(pair, want):
            assert all(torch.equal(g.cpu(), v) for g, v in zip(got, w))
