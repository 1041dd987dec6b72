"""Norms and their gradients at the edges: rows without columns, no
sequences, infinities and NaN."""
import pytest

import lsd_radix_sort_key_gb300 as rs
from lsd_radix_sort_key_gb300 import experts

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from block_util import plain_norm_grad  # noqa: E402
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


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows", [0, 1, 12])
def test_no_columns(way, dt, rows):
    x, w = torch.empty(rows, 0, dtype=TYPES[dt], device=DEV), torch.empty(0, device=DEV)
    assert rs.expert_norm(x, w).shape == (rows, 0)
    y, h = rs.expert_norm(x, w, block=x, block_weight=w, gate=w)
    assert y.shape == h.shape == (rows, 0)
    got = rs.expert_norm_grad(x, x, w)
    assert [None if t is None else tuple(t.shape) for t in got] == [(rows, 0), (0,), None, None, None]
    got = rs.expert_norm_grad(x, x, w, dy=x, block=x, block_weight=w, gate=w)
    assert [tuple(t.shape) for t in got] == [(rows, 0), (0,), (rows, 0), (0,), (0,)]
    torch.cuda.synchronize()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("sequences", [0, 5])
def test_no_rows_with_a_gate_for_each_sequence(way, dt, sequences):
    # an empty batch, of no sequences or of empty ones
    x, w = torch.empty(0, 264, dtype=TYPES[dt], device=DEV), torch.ones(264, device=DEV)
    gate = torch.ones(sequences, 264, device=DEV)
    y, h = rs.expert_norm(x, w, block=x, block_weight=w, gate=gate)
    assert y.shape == h.shape == (0, 264)
    got = rs.expert_norm_grad(x, y, w, dy=x, block=x, block_weight=w, gate=gate)
    assert [tuple(t.shape) for t in got] == [(0, 264), (264,), (0, 264), (264,), (sequences, 264)]
    assert all(bool((got[i] == 0).all()) for i in (1, 3, 4))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("width", [72, 264, 2048, 1037, 8192, 4100])
@pytest.mark.parametrize("gate", [None, 0, 4])
@pytest.mark.parametrize("weight", [False, True])
def test_a_block_without_a_weight_has_no_part_in_its_gradient(way, dt, width, gate, weight):
    # dblock = gate d, whatever the block holds; dgate takes it as it is
    g, dtype = gen(width), TYPES[dt]
    y, block, dy, dh = (torch.randn(24, width, device=DEV, generator=g).to(dtype) for _ in range(4))
    w = 1 + 0.3 * torch.randn(width, device=DEV, generator=g) if weight else None
    gates = None if gate is None else torch.randn(*((width,) if gate == 0 else (gate, width)), device=DEV, generator=g)
    block[3, 5], block[7, width - 1], block[11] = float("inf"), float("nan"), float("-inf")
    dh = dh if weight else None
    got = rs.expert_norm_grad(dh, y, w, dy=dy, block=block, gate=gates, residual_scale=0.7)
    want = plain_norm_grad(dh, y, w, dy, block, None, gates, 0.7, 1e-6)
    assert bool(torch.isfinite(got[2]).all())
    for name, t in zip(("dx", "dweight", "dblock"), got):
        if t is not None:
            held(t, *want[name])
    if gate is not None:
        bad = ~torch.isfinite(want["dgate"][0])
        assert torch.equal(~torch.isfinite(got[4].double()), bad)
        held(got[4][~bad], want["dgate"][0][~bad], want["dgate"][1][~bad])


@pytest.mark.parametrize("width", [264, 1037])
def test_infinities_and_nan_reach_what_the_formulas_say(way, width):
    # the rows that hold them, in every result and by the formula's own value
    g = gen(3)
    y, block, dh, dy = (torch.randn(16, width, device=DEV, generator=g) for _ in range(4))
    w, after, gate = (1 + 0.3 * torch.randn(width, device=DEV, generator=g) for _ in range(3))
    dy[2, 4], dy[5, 9], dh[8, 1] = float("inf"), float("nan"), float("inf")
    for a in (None, after):
        got = rs.expert_norm_grad(None, y, None, dy=dy, block=block, block_weight=a, gate=gate, residual_scale=0.5)
        dx = 0.5 * dy
        assert torch.equal(torch.isnan(got[0]), torch.isnan(dx)) and torch.equal(torch.isinf(got[0]), torch.isinf(dx))
        du = dy * gate
        rows = torch.isfinite(du).all(1)
        assert bool(torch.isfinite(got[2][rows]).all())
        if a is None:
            assert torch.equal(torch.nan_to_num(got[2], 9e9), torch.nan_to_num(du, 9e9))
        got = rs.expert_norm_grad(dh, y, w, block=block, block_weight=a, gate=gate)
        rows = torch.isfinite(dh).all(1)
        for t in (got[0], got[2]):
            assert bool(torch.isfinite(t[rows]).all()) and not bool(torch.isfinite(t[~rows]).any())
