"""The example layer's autograd Functions ask for the gradients that are wanted,
and for no others; the operators' calls are recorded and not run."""
import os
import sys

import pytest

import lsd_radix_sort_key_gb300 as rs

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer  # noqa: E402


@pytest.mark.parametrize("want", [w for w in range(1, 8)])
@pytest.mark.parametrize("activation", ["none", "silu"])
def test_a_product_asks_for_the_gradients_that_are_wanted(monkeypatch, want, activation):
    need = [bool(want >> i & 1) for i in range(3)]
    asked = []

    def matmul(x, w, offsets, *, bias=None, activation="none", residual=None, return_pre=False):
        y = x @ w[0].T
        return (y, y) if return_pre else y

    def matmul_grad(dy, x, w, offsets, *, pre=None, activation="none", bias=True, need_dx=True, need_dw=True):
        asked.append((need_dx, need_dw, bias))
        return tuple(torch.ones(s) if n else None for s, n in ((x.shape, need_dx), (w.shape, need_dw), (w.shape[:2], bias)))

    monkeypatch.setattr(rs, "expert_matmul", matmul)
    monkeypatch.setattr(rs, "expert_matmul_grad", matmul_grad)
    args = [torch.randn(s).requires_grad_(n) for s, n in zip(((5, 4), (2, 3, 4), (2, 3)), need)]
    expert_layer.Matmul.apply(*args, torch.tensor([0, 2, 5]), activation).sum().backward()
    assert asked == [tuple(need)]
    for t, n in zip(args, need):
        assert (t.grad is not None) == n
