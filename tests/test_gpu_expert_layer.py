"""The expert operators together, as a layer: examples/expert_layer.py against
a plain 64-bit form of the same layer, values and all gradients."""
import os
import sys

import pytest

import lsd_radix_sort_key_gb300 as rs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    rs.build()
    rs.lib()


def plain(layer, x, ids):
    """The layer in 64 bits, token by slot, with the routing given."""
    logits = (x @ layer["router"]).gather(1, ids)
    weights = torch.softmax(logits, dim=1)
    out = torch.zeros_like(x)
    for e in range(layer["up"].shape[0]):
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        mid = torch.nn.functional.silu(x[token] @ layer["up"][e].T + layer["up_bias"][e])
        row = mid @ layer["down"][e].T + layer["down_bias"][e]
        out = out.index_add(0, token, weights[token, slot, None] * row)
    return out


@pytest.mark.parametrize("dtype,steps", [(torch.float32, 2.0**-18), (torch.bfloat16, 2.0**-8), (torch.float16, 2.0**-11)])
@pytest.mark.parametrize("tokens,slots", [(1, 1), (3, 4), (500, 2)])
def test_layer_and_gradients(dtype, steps, tokens, slots):
    # Five roundings to dtype lie on the way (rows, mid, experts' rows, output
    # and, backwards, as many): relative to the largest value of each result,
    # whose terms add up with random signs, 8 times the unit covers them; float32
    # is held to 2^-18, a hundred additions of its unit.
    torch.manual_seed(1)
    layer = expert_layer.ExpertLayer(64, 96, 8, slots, dtype)
    x = torch.randn(tokens, 64, device="cuda").to(dtype).requires_grad_()
    ids = layer.route(x)[1]
    g = torch.randn(tokens, 64, device="cuda").to(dtype)
    y = layer(x)
    y.backward(g)
    want = {k: v.detach().double().requires_grad_() for k, v in layer.named_parameters()}
    x64 = x.detach().double().requires_grad_()
    y64 = plain(want, x64, ids)
    y64.backward(g.double())
    pairs = [("y", y, y64), ("x", x.grad, x64.grad)] + [(k, v.grad, want[k].grad) for k, v in layer.named_parameters()]
    for name, got, exact in pairs:
        off = float((got.detach().double() - exact.detach()).abs().max())
        assert off <= 8 * steps * float(exact.detach().abs().max()) + 1e-12, name


def test_example_learns():
    argv = sys.argv
    sys.argv = ["expert_layer.py", "--tokens", "1024", "--width", "128", "--steps", "20"]
    try:
        losses = expert_layer.main()
    finally:
        sys.argv = argv
    assert losses[-1] < 0.8 * losses[0]
