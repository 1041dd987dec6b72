"""Norms and their gradients at the edges: rows without columns."""
import pytest

import lsd_radix_sort_key_gb300 as rs
from lsd_radix_sort_key_gb300 import experts

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from expert_util import DEV, TYPES  # noqa: E402


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
