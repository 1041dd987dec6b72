"""The quantisers, products and norms together, as they are used: the block of
examples/expert_layer.py against plain 64-bit forms, its gradients, single
tokens, and the whole of it captured."""
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
from block_util import plain_norm, plain_quantize, same, values  # noqa: E402
from expert_util import ADD, gen, held, plain_combine, rounded  # noqa: E402
from test_gpu_expert_matmul_quantized import check_quantized, plain  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    rs.build()
    rs.lib()


def block_of(width, hidden, experts, slots, dtype, seed=1):
    torch.manual_seed(seed)
    block = expert_layer.ExpertBlock(width, hidden, experts, slots, dtype)
    with torch.no_grad():
        for p in (block.before, block.after, block.next, block.gate, block.layer.up_bias, block.layer.down_bias):
            p.add_(0.2 * torch.randn_like(p.float()).to(p.dtype))
    return block


def rms(v, w):
    return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6) * w


@pytest.mark.parametrize("dtype,steps", [(torch.float32, 2.0**-18), (torch.bfloat16, 2.0**-8), (torch.float16, 2.0**-11)])
@pytest.mark.parametrize("tokens,slots", [(1, 1), (3, 4), (500, 2)])
def test_the_block_and_its_gradients(dtype, steps, tokens, slots):
    # Nine roundings to dtype lie on the way, and as many backwards, relative to
    # the largest value of each result and with random signs: 16 times the unit
    # covers them (float32: 2^-18, as for the layer alone).
    block = block_of(64, 96, 8, slots, dtype)
    x = torch.randn(tokens, 64, device="cuda").to(dtype).requires_grad_()
    gy, gh = (torch.randn(tokens, 64, device="cuda").to(dtype) for _ in range(2))
    y, h = block(x)
    (y.float() * gy.float()).sum().add((h.float() * gh.float()).sum()).backward()
    want = {k: v.detach().double().requires_grad_() for k, v in block.named_parameters()}
    x64 = x.detach().double().requires_grad_()
    with torch.no_grad():
        _, ids = block.layer.route(rs.expert_norm(x.detach(), block.before.detach()))
    into = rms(x64, want["before"])
    weights = torch.softmax((into @ want["layer.router"]).gather(1, ids), dim=1)
    out = torch.zeros_like(x64)
    for e in range(8):
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        mid = torch.nn.functional.silu(into[token] @ want["layer.up"][e].T + want["layer.up_bias"][e])
        out = out.index_add(0, token, weights[token, slot, None] * (mid @ want["layer.down"][e].T + want["layer.down_bias"][e]))
    y64 = block.residual_scale * x64 + want["gate"] * rms(out, want["after"])
    h64 = rms(y64, want["next"])
    ((y64 * gy.double()).sum() + (h64 * gh.double()).sum()).backward()
    pairs = [("y", y, y64), ("h", h, h64), ("x", x.grad, x64.grad)] + [
        (k, v.grad, want[k].grad) for k, v in block.named_parameters()]
    for name, got, exact in pairs:
        off = float((got.detach().double() - exact.detach()).abs().max())
        assert off <= 16 * steps * float(exact.detach().abs().max()) + 1e-12, name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,width,hidden,experts,slots", [(1, 64, 96, 8, 2), (37, 136, 200, 5, 3), (700, 512, 1024, 16, 2)])
def test_every_step_of_serving(dtype, tokens, width, hidden, experts, slots):
    # each step against its definition, from what the step before gave
    block = block_of(width, hidden, experts, slots, dtype).quantize()
    layer = block.layer
    x = torch.randn(tokens, width, device="cuda", generator=gen(3)).to(dtype)
    with torch.no_grad():
        h = rs.expert_norm(x, block.before)
        _, _, want, bound = plain_norm(x, block.before, None, None, None, 1.0, 1e-6)
        held(h, want, bound)
        weights, ids = layer.route(h)
        _, position, offsets = rs.expert_sort(ids, experts)
        rows, scales = rs.expert_dispatch_quantized(h, position, offsets)
        qw, sw = plain_quantize(h)
        for k in range(slots):
            at = position[:, k].long()
            assert same(rows[at], qw) and torch.equal(scales[at].double(), sw)
        up, ups, down, downs = block.quantized
        for e in range(experts):
            q, s = plain_quantize(layer.up[e], 128)
            assert same(up[e], q) and torch.equal(ups[e].double(), s)
        mid, mids = rs.expert_matmul_quantized(rows, scales, up, ups, offsets, bias=layer.up_bias, activation="silu", dtype=dtype,
                                               quantize=True)
        y, _, mag = plain(rows, scales, up, ups, offsets, layer.up_bias, "silu")
        check_quantized(mid, mids, y, mag, width)
        back = rs.expert_matmul_quantized(mid, mids, down, downs, offsets, bias=layer.down_bias, dtype=dtype)
        y, _, mag = plain(mid, mids, down, downs, offsets, layer.down_bias)
        held(back, y, (hidden + 8) * ADD * mag + rounded(y, dtype) + 1e-30)
        out = rs.expert_combine(back, weights, position, offsets)
        want, mag = plain_combine(back, weights, position, offsets)
        held(out, want, (slots + 8) * ADD * mag + rounded(want, dtype) + 1e-30)
        served = block.serve(x)
        y, y_bound, h2, h_bound = plain_norm(x, block.next, out, block.after, block.gate, block.residual_scale, 1e-6, served[0])
        held(served[0], y, y_bound)
        held(served[1], h2, h_bound)


def test_the_quantised_products_are_near_the_others():
    # A quantised value is off by at most half a step, 2^-4 of it, so by 2^-4 / sqrt(3) =
    # 0.036 in the mean square; the two operands of a product by sqrt(2) times that
    # and the two products one after the other by 2 times: 0.072 of the layer's
    # output, of which y and h hold a part.
    block = block_of(512, 1024, 16, 2, torch.bfloat16).quantize()
    x = torch.randn(300, 512, device="cuda", generator=gen(5)).bfloat16()
    with torch.no_grad():
        y, h = block(x)
        y8, h8 = block.serve(x)
    for a, b in ((y8, y), (h8, h)):
        assert float((a.float() - b.float()).norm() / b.float().norm()) < 0.1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_single_tokens_against_the_batch(dtype):
    # the same sums in other tiles: float32 additions in another order at most, then
    # one rounding each of out, y and h, and what a value next to a border of e4m3 does
    # (2^-3 of one of 1024 terms)
    block = block_of(512, 1024, 16, 2, dtype).quantize()
    x = torch.randn(40, 512, device="cuda", generator=gen(6)).to(dtype)
    whole = block.serve(x)
    single = [torch.cat(t) for t in zip(*(block.serve(x[i:i + 1]) for i in range(40)))]
    for a, b in zip(whole, single):
        assert float((a.float() - b.float()).abs().max()) <= 2.0**-6 * float(b.float().abs().max())


def test_serving_captured():
    block = block_of(256, 512, 8, 2, torch.bfloat16).quantize()
    x = torch.randn(64, 256, device="cuda", generator=gen(7)).bfloat16()
    block.serve(x)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):  # two graphs over the same weights
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(block.serve(x))
        graphs.append(graph)
    for seed in (8, 9):
        x.copy_(torch.randn(64, 256, device="cuda", generator=gen(seed)).bfloat16())
        want = block.serve(x)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_a_training_step_captured_beside_an_eager_one():
    # a backward pass is captured while an eager graph of the same leaves lives
    block = block_of(64, 96, 8, 2, torch.bfloat16)
    x = torch.randn(50, 64, device="cuda", generator=gen(10)).bfloat16()

    def step():
        y, h = block(x)
        return torch.autograd.grad(y.float().square().sum() + h.float().sum(), [p for p in block.parameters()])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    want = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("before", ["nothing", "copy", "fill", "kernel", "join", "kernel and join", "join and kernel"])
def test_what_a_call_reads_is_there(captured, before):
    # The work before a call has ended when the call reads, whatever it is and
    # whichever stream it was on.
    rows, width = 4096, 512
    fresh = torch.randn(rows, width, device="cuda", generator=gen(4)).bfloat16()
    big, late = torch.empty(1 << 28, dtype=torch.uint8, device="cuda"), torch.empty_like(fresh)
    weight = torch.ones(width, device="cuda")
    w = torch.randn(1, 512, width, device="cuda", generator=gen(5)).bfloat16()
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    position = torch.arange(rows, dtype=torch.int32, device="cuda")[:, None]
    wq, ws = rs.expert_quantize_weights(w)
    q0, s0 = rs.expert_quantize(fresh)
    side = torch.cuda.Stream()

    def produce(into, source):
        if "join" in before:
            ready = torch.cuda.current_stream()
            side.wait_stream(ready)
            with torch.cuda.stream(side):
                torch.cuda._sleep(100000)
                into.copy_(source)
            if before.startswith("kernel"):
                big[:4096].add_(1)
            ready.wait_stream(side)
            if before.endswith("kernel"):
                big[:4096].add_(1)
        elif before != "nothing":
            torch.cuda._sleep(100000)
            if before == "copy":
                big[:1 << 27].copy_(big[1 << 27:])
                into.copy_(source)
            elif before == "fill":
                into.copy_(source)
                big.zero_()
            else:
                torch.mul(source.view(torch.uint8), 1, out=into.view(torch.uint8))
        else:
            into.copy_(source)

    def call():
        out = []
        q, s = torch.zeros_like(q0.view(torch.uint8)), torch.zeros_like(s0.view(torch.uint8))
        produce(late, fresh)
        out += [rs.expert_norm(late, weight)]
        late.zero_()
        produce(late, fresh)
        out += rs.expert_quantize(late)
        late.zero_()
        produce(late, fresh)
        out += rs.expert_dispatch_quantized(late, position, offsets)
        late.zero_()
        produce(late, fresh)
        out += rs.expert_norm_grad(late, late, weight)[:2]
        produce(q, q0.view(torch.uint8))
        produce(s, s0.view(torch.uint8))
        out += [rs.expert_matmul_quantized(q.view(q0.dtype), s.view(s0.dtype), wq, ws, offsets)]
        q.zero_()
        s.zero_()
        return [t.view(torch.uint8) if t.dtype.itemsize == 1 else t for t in out]

    def plain_calls():
        out = [rs.expert_norm(fresh, weight), *rs.expert_quantize(fresh),
               *rs.expert_dispatch_quantized(fresh, position, offsets), *rs.expert_norm_grad(fresh, fresh, weight)[:2],
               rs.expert_matmul_quantized(q0, s0, wq, ws, offsets)]
        torch.cuda.synchronize()
        return [t.view(torch.uint8) if t.dtype.itemsize == 1 else t for t in out]

    want = plain_calls()
    torch.cuda.synchronize()
    if captured:
        with torch.cuda.stream(side):
            call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        for _ in range(3):
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    else:
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(call(), want))


def test_the_example_runs():
    argv = sys.argv
    sys.argv = ["expert_layer.py", "--tokens", "256", "--width", "128", "--steps", "2"]
    try:
        assert len(expert_layer.main()) == 2
    finally:
        sys.argv = argv


def test_a_weight_update_reaches_the_quantised_weights():
    block = block_of(128, 256, 4, 2, torch.bfloat16).quantize()
    x = torch.randn(20, 128, device="cuda", generator=gen(11)).bfloat16()
    before = block.serve(x)[0]
    with torch.no_grad():
        block.layer.up.mul_(0.5)
    assert torch.equal(block.serve(x)[0], before)  # they are the caller's to make again
    assert not torch.equal(block.quantize().serve(x)[0], before)


def test_values_are_exact_in_32_bits():
    # q * scale as torch computes it is what the definition says
    x = torch.randn(50, 300, device="cuda", generator=gen(12))
    q, s = rs.expert_quantize(x)
    v = q.float() * s.float().repeat_interleave(128, -1)[..., :300]
    assert torch.equal(v.double(), values(q, s))
    assert float((v - x).abs().max() / x.abs().max()) <= 2.0**-4
