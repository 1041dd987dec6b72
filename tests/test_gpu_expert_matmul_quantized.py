"""The experts' products of quantised rows and weights against 64 bits."""
import threading

import pytest

import lsd_radix_sort_key_gb300 as rs
from lsd_radix_sort_key_gb300 import experts

pytestmark = pytest.mark.gpu

np = pytest.importorskip("numpy")
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from block_util import E8M0, aligned, plain_quantize, random_quantized, same, scale_of, values  # noqa: E402
from expert_util import ADD, DEV, act64, gen, held, matmul_bounds, rounded  # noqa: E402

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


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


def offsets_of(counts, unused=0):
    return torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device=DEV), sum(counts) + unused


def operands(counts, inner, outer, seed=1, unused=0, spread=3):
    g = gen(seed)
    off, rows = offsets_of(counts, unused)
    x, xs = random_quantized(g, rows, inner, spread=spread)
    w, ws = random_quantized(g, len(counts), outer, inner, down=128, spread=spread)
    # values around one: an inner product of `inner` terms of 60 * 60
    shift = int(round(np.log2(3600 * max(1, inner) ** 0.5))) // 2
    xs = (xs.view(torch.uint8) - shift).view(E8M0)
    ws = (ws.view(torch.uint8) - shift).view(E8M0)
    return x, xs, w, ws, off


def plain(x, xs, w, ws, off, bias=None, act="none", residual=None):
    """y, z and the magnitudes behind z in 64 bits, zero in unused rows."""
    xv, wv = values(x, xs), values(w, ws, 128)
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=DEV)
    z, mag = torch.zeros_like(y), torch.zeros_like(y)
    edge = off.tolist()
    for e, (a, b) in enumerate(zip(edge, edge[1:])):
        z[a:b], mag[a:b] = xv[a:b] @ wv[e].T, xv[a:b].abs() @ wv[e].abs().T
        if bias is not None:
            z[a:b] += bias[e].double()
            mag[a:b] += bias[e].double().abs()
        y[a:b] = act64(z[a:b], act)
        if residual is not None:
            y[a:b] += residual[a:b].double()
    return y, z, mag


# The activations of 16-bit results are approximate: the published cdf is off by at
# most 1.5e-7 in erf, so gelu by 2.1e-7 in value; the exponential and reciprocal
# of silu by a few 2^-22.
FAST = 2.5e-7


def check(y, z, got, pre, mag, inner, dtype, residual=None):
    yb, zb = matmul_bounds(y, z, mag, inner, dtype, residual)
    held(got, y, yb + FAST * (1 + y.abs()))
    if pre is not None:
        held(pre, z, zb)


def check_quantized(q, scales, y, mag, inner):
    """A quantised result: every value within half a step of the largest scale it
    may have, and the scales those of the values, but where a sum's error moves a
    block past a border."""
    r, n = y.shape
    off = 1.13 * (inner + 8) * ADD * mag + FAST * (1 + y.abs()) + 1e-30
    pad = -n % 128
    blocks = torch.nn.functional.pad(y.abs(), (0, pad)).view(r, -1, 128)
    offs = torch.nn.functional.pad(off, (0, pad)).view(r, -1, 128)
    low, high = scale_of((blocks - offs).clamp(min=0).amax(2)), scale_of((blocks + offs).amax(2))
    s = scales.double()
    live = blocks.amax(2) > 0
    assert bool(((s >= torch.where(live, low.clamp(max=high), s)) & (s <= torch.where(live, high, s)))[live].all())
    assert bool((s[~live] == 1).all() | (offs.amax(2)[~live] > 0).all())
    per = s.repeat_interleave(128, 1)[:, :n]
    got = q.double() * per
    # half a step: 2^-4 of the value, 2^-10 of the scale below the normal range
    held(got, y, off + (y.abs() + off) * 2.0**-4 + per * 2.0**-10)


SHAPES = [([1], 16, 16), ([3], 128, 128), ([0, 5, 0, 40], 129, 257), ([128, 128], 256, 256), ([129, 1, 255], 512, 130),
          ([300, 0, 700], 1000, 1160), ([7] * 64, 640, 264), ([1000], 37, 1000), ([500, 300], 2048, 384), ([40, 90], 1, 72),
          ([2, 3], 300, 1), ([600, 600, 600, 600], 896, 2048)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("counts,inner,outer", SHAPES)
def test_products(way, dt, counts, inner, outer):
    x, xs, w, ws, off = operands(counts, inner, outer, unused=5)
    y, z, mag = plain(x, xs, w, ws, off)
    got = rs.expert_matmul_quantized(x, xs, w, ws, off, dtype=TYPES[dt])
    assert got.dtype == TYPES[dt]
    check(y, z, got, None, mag, inner, TYPES[dt])
    assert bool((got[int(off[-1]):] == 0).all())


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("counts,inner,outer", [([300, 0, 700], 1000, 1160), ([9, 17], 256, 72), ([600] * 8, 640, 1024)])
def test_epilogues(way, dt, act, counts, inner, outer):
    dtype, g = TYPES[dt], gen(7)
    x, xs, w, ws, off = operands(counts, inner, outer, unused=9)
    bias = torch.randn(len(counts), outer, device=DEV, generator=g).to(dtype)
    residual = torch.randn(x.shape[0], outer, device=DEV, generator=g).to(dtype)
    for b, r, keep in ((bias, residual, True), (bias, None, False), (None, residual, False), (None, None, True)):
        y, z, mag = plain(x, xs, w, ws, off, b, act, r)
        got = rs.expert_matmul_quantized(x, xs, w, ws, off, bias=b, activation=act, residual=r, dtype=dtype, return_pre=keep)
        got, pre = got if keep else (got, None)
        check(y, z, got, pre, mag, inner, dtype, r)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("counts,inner,outer", [([1], 16, 16), ([300, 0, 700], 1000, 1160), ([9, 17], 256, 72), ([33], 512, 129),
                                                ([600] * 8, 640, 1024), ([700], 2048, 384)])
def test_quantized_results(way, act, counts, inner, outer):
    g = gen(11)
    x, xs, w, ws, off = operands(counts, inner, outer, unused=130)
    bias = torch.randn(len(counts), outer, device=DEV, generator=g).bfloat16()
    for b, keep in ((bias, True), (None, False)):
        y, z, mag = plain(x, xs, w, ws, off, b, act)
        got = rs.expert_matmul_quantized(x, xs, w, ws, off, bias=b, activation=act, return_pre=keep, quantize=True)
        assert len(got) == (3 if keep else 2)
        check_quantized(got[0], got[1], y, mag, inner)
        assert bool((got[0][int(off[-1]):].double() == 0).all()) and bool((got[1][int(off[-1]):].double() == 1).all())
        if keep:
            held(got[2], z, matmul_bounds(y, z, mag, inner, torch.bfloat16)[1])


def test_exact_sums_are_quantized_to_the_bit():
    # small whole numbers: every sum is exact, so the result is the definition's
    g = gen(2)
    counts, inner, outer = [70, 0, 150], 384, 300
    off, rows = offsets_of(counts)
    x = aligned(torch.randint(-8, 9, (rows, inner), device=DEV, generator=g).float().to(torch.float8_e4m3fn))
    w = aligned(torch.randint(-8, 9, (3, outer, inner), device=DEV, generator=g).float().to(torch.float8_e4m3fn))
    xs = torch.randint(120, 130, (rows, 3), dtype=torch.uint8, device=DEV, generator=g).view(E8M0)
    ws = torch.full((3, 3, 3), 127, dtype=torch.uint8, device=DEV).view(E8M0)
    y, _, _ = plain(x, xs, w, ws, off)
    q, scales = rs.expert_matmul_quantized(x, xs, w, ws, off, quantize=True)
    want, want_scales = plain_quantize(y)
    assert torch.equal(scales.double(), want_scales) and same(q, want)


@pytest.mark.parametrize("k", range(0, 640, 61))
def test_each_scale_meets_its_own_block(k):
    # one block of the reduction at a time is not zero, and every row and every
    # 128 x 128 weights have scales of their own
    counts, inner, outer = [130, 60], 640, 520
    off, rows = offsets_of(counts)
    g = gen(k)
    x, w = (torch.zeros(*s, device=DEV) for s in ((rows, inner), (2, outer, inner)))
    x[:, k], w[:, :, k] = 1, 1
    x, w = aligned(x.to(torch.float8_e4m3fn)), aligned(w.to(torch.float8_e4m3fn))
    xs = torch.randint(122, 132, (rows, 5), dtype=torch.uint8, device=DEV, generator=g).view(E8M0)
    ws = torch.randint(122, 132, (2, 5, 5), dtype=torch.uint8, device=DEV, generator=g).view(E8M0)
    y, _, _ = plain(x, xs, w, ws, off)
    assert torch.equal(rs.expert_matmul_quantized(x, xs, w, ws, off).double(), y)  # powers of two: exact


def test_many_rows_and_tiles():
    # several tiles per block, both accumulators and both sets of scales in use
    for counts, inner, outer in (([3000, 1, 5000, 4000], 1024, 2048), ([2500] * 2, 384, 4096)):
        x, xs, w, ws, off = operands(counts, inner, outer, seed=4)
        y, z, mag = plain(x, xs, w, ws, off)
        check(y, z, rs.expert_matmul_quantized(x, xs, w, ws, off, dtype=torch.float16), None, mag, inner, torch.float16)
        got = rs.expert_matmul_quantized(x, xs, w, ws, off, quantize=True)
        check_quantized(got[0], got[1], y, mag, inner)


@pytest.mark.parametrize("counts,inner,outer", [([0, 1, 3, 0] * 256, 128, 264), ([5], 65552, 40), ([3, 4], 64, 70000),
                                                ([900] * 3, 16400, 272)])
def test_many_experts_long_sums_and_wide_outputs(counts, inner, outer):
    x, xs, w, ws, off = operands(counts, inner, outer, unused=3)
    y, z, mag = plain(x, xs, w, ws, off)
    check(y, z, rs.expert_matmul_quantized(x, xs, w, ws, off, dtype=torch.float16), None, mag, inner, torch.float16)
    q, scales = rs.expert_matmul_quantized(x, xs, w, ws, off, quantize=True)
    check_quantized(q, scales, y, mag, inner)


def test_refusals(way):
    x, xs, w, ws, off = operands([33, 70], 272, 200)
    bias = torch.zeros(2, 200, dtype=torch.bfloat16, device=DEV)
    res = torch.zeros(103, 200, dtype=torch.bfloat16, device=DEV)
    tight = x.view(torch.uint8)[:, :271].contiguous().view(torch.float8_e4m3fn)  # rows of 271 bytes
    for error, call in [
            (TypeError, lambda: rs.expert_matmul_quantized(x.float(), xs, w, ws, off)),
            (TypeError, lambda: rs.expert_matmul_quantized(x, xs.float(), w, ws, off)),
            (TypeError, lambda: rs.expert_matmul_quantized(x, xs, w, ws.float(), off)),
            (ValueError, lambda: rs.expert_matmul_quantized(x, xs[:, :2], w, ws, off)),
            (ValueError, lambda: rs.expert_matmul_quantized(x, xs, w, ws[:1], off)),
            (ValueError, lambda: rs.expert_matmul_quantized(x[:, :256], xs[:, :2], w, ws, off)),
            (ValueError, lambda: rs.expert_matmul_quantized(tight, xs, w[:, :, :271], ws, off)),
            (ValueError, lambda: rs.expert_matmul_quantized(x[:, 1:257], xs[:, :2], w[:, :, :256], ws[:, :, :2].contiguous(), off)),
            (ValueError, lambda: rs.expert_matmul_quantized(x, xs, w.transpose(1, 2), ws, off)),
            (ValueError, lambda: rs.expert_matmul_quantized(x, xs, w[:, :100], ws[:, :1].contiguous(), off)),
            (ValueError, lambda: rs.expert_matmul_quantized(x, xs, w, ws, off[:2])),
            (TypeError, lambda: rs.expert_matmul_quantized(x, xs, w, ws, off.long())),
            (TypeError, lambda: rs.expert_matmul_quantized(x, xs, w, ws, off, bias=bias.half())),
            (ValueError, lambda: rs.expert_matmul_quantized(x, xs, w, ws, off, bias=bias[:1])),
            (ValueError, lambda: rs.expert_matmul_quantized(x, xs, w, ws, off, residual=res[:5])),
            (ValueError, lambda: rs.expert_matmul_quantized(x, xs, w, ws, off, residual=res, quantize=True)),
            (TypeError, lambda: rs.expert_matmul_quantized(x, xs, w, ws, off, dtype=torch.float32)),
            (ValueError, lambda: rs.expert_matmul_quantized(x, xs, w, ws, off, activation="tanh")),
            (ValueError, lambda: rs.expert_matmul_quantized(x, xs, w, ws.cpu(), off)),
            (TypeError, lambda: rs.expert_matmul_quantized(x, xs, w, ws, off, temp=torch.empty(100, device=DEV))),
            (rs.RadixSortError, lambda: rs.expert_matmul_quantized(x, xs, w, ws, off,
                                                                   temp=torch.empty(100, dtype=torch.uint8, device=DEV)))]:
        with pytest.raises(error):
            call()


def test_offsets_that_are_no_plan():
    # clamped to ascending values in [0, rows]: wrong rows, no access outside
    x, xs, w, ws, _ = operands([40, 60, 30], 256, 256)
    for off, used in (([5, 40, 20, 130], [0, 40, 40, 130]), ([0, 1 << 30, 7, 9], [0, 130, 130, 130]),
                      ([-3, -1, 50, 60], [0, 0, 50, 60])):
        off, used = (torch.tensor(o, dtype=torch.int32, device=DEV) for o in (off, used))
        y, z, mag = plain(x, xs, w, ws, used)
        check(y, z, rs.expert_matmul_quantized(x, xs, w, ws, off), None, mag, 256, torch.bfloat16)


def test_nan_and_infinity_stay_in_their_rows():
    x, xs, w, ws, off = operands([50, 90], 300, 260, unused=3)
    x.view(torch.uint8)[7, 100] = 0x7F       # NaN
    xs.view(torch.uint8)[60, 1] = 0xFF       # a NaN scale
    x.view(torch.uint8)[141] = 0x7F          # an unused row
    y, z, mag = plain(x, xs, w, ws, off)
    bad = torch.zeros(143, dtype=torch.bool, device=DEV)
    bad[7] = bad[60] = True
    assert bool(torch.isnan(y[bad]).all())
    got = rs.expert_matmul_quantized(x, xs, w, ws, off)
    held(got, y, matmul_bounds(y, z, torch.nan_to_num(mag), 300, torch.bfloat16)[0])
    q, scales = rs.expert_matmul_quantized(x, xs, w, ws, off, quantize=True)
    assert bool(torch.isnan(q.double()[bad]).all()) and not bool(torch.isnan(q.double()[~bad]).any())
    # a sum past float32's range is infinite in 16 bits and NaN in 8
    xs.view(torch.uint8)[20] = 254
    ws.view(torch.uint8)[0] = 160
    got = rs.expert_matmul_quantized(x, xs, w, ws, off)
    assert bool(torch.isinf(got[20]).any())
    q, scales = rs.expert_matmul_quantized(x, xs, w, ws, off, quantize=True)
    inf = torch.isinf(got[20])
    assert bool(torch.isnan(q[20].double()[inf]).all()) and bool((scales[20].double() <= 2.0**120).all())


@pytest.mark.parametrize("rows", [40, 4096])
@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_activations_of_infinity(rows, act):
    # sums of zero, so that the values before the activation are the biases
    x, xs, w, ws, off = operands([rows], 256, 512)
    x = torch.zeros_like(x.view(torch.uint8)).view(torch.float8_e4m3fn)
    bias = torch.randn(1, 512, device=DEV, generator=gen(3)).bfloat16()
    bias[0, :6] = torch.tensor([float("inf"), float("nan"), 3e38, -3e38, 1e20, -1e20])
    y = rs.expert_matmul_quantized(x, xs, w, ws, off, bias=bias, activation=act)
    assert bool(torch.isposinf(y[:, 0]).all()) and bool(torch.isnan(y[:, 1]).all())
    assert torch.equal(y[:, 2:6], torch.tensor([3e38, 0, 1e20, 0], device=DEV).bfloat16().expand(rows, 4))
    assert bool(torch.isfinite(y[:, 6:]).all())


def test_views_and_strides(way):
    g = gen(5)
    x, xs, w, ws, off = operands([33, 70], 272, 200)
    y, z, mag = plain(x, xs, w, ws, off)
    wide = torch.zeros(103, 272 + 48, dtype=torch.uint8, device=DEV)
    wide[:, 16:288] = x.view(torch.uint8)
    xv = wide[:, 16:288].view(torch.float8_e4m3fn)
    scales = torch.zeros(103, 10, dtype=torch.uint8, device=DEV)
    scales[:, 1:4] = xs.view(torch.uint8)
    sv = scales[:, 1:4].view(E8M0)
    wv = torch.zeros(2, 200, 320, dtype=torch.uint8, device=DEV)
    wv[:, :, :272] = w.view(torch.uint8)
    wv = wv[:, :, :272].view(torch.float8_e4m3fn)
    bias = torch.randn(3, 210, device=DEV, generator=g).bfloat16()
    res = torch.randn(1, 200, device=DEV, generator=g).bfloat16().expand(103, 200)
    check(y, z, rs.expert_matmul_quantized(xv, sv, wv, ws, off), None, mag, 272, torch.bfloat16)
    y, z, mag = plain(x, xs, w, ws, off, bias[1:, 5:205], "silu", res)
    got = rs.expert_matmul_quantized(xv, sv, wv, ws, off, bias=bias[1:, 5:205], activation="silu", residual=res)
    check(y, z, got, None, mag, 272, torch.bfloat16, res)


def test_outputs_behind_strides_are_left_alone():
    x, xs, w, ws, off = operands([33, 70], 256, 136)
    y, z, mag = plain(x, xs, w, ws, off)
    temp = torch.empty(1 << 12, dtype=torch.uint8, device=DEV)
    out = torch.full((105, 200), 7.0, dtype=torch.bfloat16, device=DEV)
    q = torch.full((105, 160), 0x55, dtype=torch.uint8, device=DEV)
    qs = torch.full((105, 5), 0x55, dtype=torch.uint8, device=DEV)
    d = rs.ExpertMatmulQuantizedDesc(2, 0, 2, 103, 256, 136, off.data_ptr(), x.data_ptr(), 256, xs.data_ptr(), 2, w.data_ptr(),
                                     256, ws.data_ptr(), None, 0, None, 0, out[1:].data_ptr(), 200, None, 0, None, 0, None, 0,
                                     temp.data_ptr(), temp.numel(), torch.cuda.current_stream().cuda_stream, 0)
    assert rs.rs_expert_matmul_quantized(d) == 0 and rs.rs_expert_matmul_status(temp) == 0
    check(y, z, out[1:104, :136], None, mag, 256, torch.bfloat16)
    assert bool((out[0] == 7).all()) and bool((out[104] == 7).all()) and bool((out[:, 136:] == 7).all())
    d.y, d.q, d.q_stride, d.q_scales, d.q_scales_stride = None, q[1:].data_ptr(), 160, qs[1:].data_ptr(), 5
    assert rs.rs_expert_matmul_quantized(d) == 0 and rs.rs_expert_matmul_status(temp) == 0
    check_quantized(q[1:104, :136].contiguous().view(torch.float8_e4m3fn), qs[1:104, :2].contiguous().view(E8M0), y, mag, 256)
    assert bool((q[0] == 0x55).all()) and bool((q[104] == 0x55).all()) and bool((q[1:104, 136:144] == 0).all())
    assert bool((q[:, 144:] == 0x55).all()) and bool((qs[1:104, 2:] == 0x55).all()) and bool((qs[0] == 0x55).all())


def test_the_gradient_of_x_with_transposed_weights():
    # dx = dy w: the same product with the weights quantised the other way round
    g = gen(12)
    counts, inner, outer = [90, 40], 200, 328
    off, rows = offsets_of(counts)
    w = torch.randn(2, outer, inner, device=DEV, generator=g).bfloat16()
    dy = torch.randn(rows, outer, device=DEV, generator=g).bfloat16()
    dq, ds = rs.expert_quantize(dy)
    wq, ws = rs.expert_quantize_weights(w)
    wt, wts = rs.expert_quantize_weights(w.transpose(1, 2))
    dx = rs.expert_matmul_quantized(dq, ds, wt, wts, off)
    dv, wv = values(dq, ds), values(wq, ws, 128)
    edge = off.tolist()
    want = torch.cat([dv[a:b] @ wv[e] for e, (a, b) in enumerate(zip(edge, edge[1:]))])
    mag = torch.cat([dv[a:b].abs() @ wv[e].abs() for e, (a, b) in enumerate(zip(edge, edge[1:]))])
    held(dx, want, (outer + 8) * ADD * mag + rounded(want, torch.bfloat16))


@pytest.mark.parametrize("quantize", [False, True])
def test_captured_replayed_and_repeated(quantize):
    x, xs, w, ws, off = operands([300, 0, 700], 640, 520)
    first = rs.expert_matmul_quantized(x, xs, w, ws, off, activation="silu", quantize=quantize)
    first = first if quantize else (first,)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        out = rs.expert_matmul_quantized(x, xs, w, ws, off, activation="silu", quantize=quantize)
        out = out if quantize else (out,)
    for _ in range(3):
        for t in out:
            t.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, first):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # other operands in the same places
    x2 = random_quantized(gen(77), *x.shape)[0]
    x.view(torch.uint8).copy_(x2.view(torch.uint8))
    graph.replay()
    fresh = rs.expert_matmul_quantized(x, xs, w, ws, off, activation="silu", quantize=quantize)
    fresh = fresh if quantize else (fresh,)
    torch.cuda.synchronize()
    for a, b in zip(out, fresh):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_on_other_streams_and_from_several_threads():
    x, xs, w, ws, off = operands([300, 40, 700], 512, 520)
    want = rs.expert_matmul_quantized(x, xs, w, ws, off)
    torch.cuda.synchronize()
    got = {}

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(5):
            got[i] = rs.expert_matmul_quantized(x, xs, w, ws, off, stream=s)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len(got) == 4 and all(torch.equal(g, want) for g in got.values())


@pytest.mark.parametrize("counts,quantize", [([40, 60], False), ([3000, 3000], False), ([3000, 3000], True), ([40], True)])
def test_a_wait_that_runs_out_is_reported(counts, quantize):
    # the operands of one tile are never copied: every wait for them has a limit
    x, xs, w, ws, off = operands(counts, 512, 512)
    temp = torch.empty(1 << 12, dtype=torch.uint8, device=DEV)
    out = torch.empty(x.shape[0], 512, dtype=torch.bfloat16, device=DEV)
    q = torch.empty(x.shape[0], 512, dtype=torch.uint8, device=DEV)
    qs = torch.empty(x.shape[0], 4, dtype=torch.uint8, device=DEV)
    d = rs.ExpertMatmulQuantizedDesc(2, 0, len(counts), x.shape[0], 512, 512, off.data_ptr(), x.data_ptr(), 512, xs.data_ptr(), 4,
                                     w.data_ptr(), 512, ws.data_ptr(), None, 0, None, 0, None if quantize else out.data_ptr(),
                                     512, q.data_ptr() if quantize else None, 512, qs.data_ptr(), 4, None, 0, temp.data_ptr(),
                                     temp.numel(), torch.cuda.current_stream().cuda_stream, 2)
    assert rs.rs_expert_matmul_quantized(d) == 0
    assert rs.rs_expert_matmul_status(temp) == 5
    d.stall_tile = 0  # the same memory works again
    assert rs.rs_expert_matmul_quantized(d) == 0 and rs.rs_expert_matmul_status(temp) == 0
    y, z, mag = plain(x, xs, w, ws, off)
    if quantize:
        check_quantized(q.view(torch.float8_e4m3fn), qs.view(E8M0), y, mag, 512)
    else:
        check(y, z, out, None, mag, 512, torch.bfloat16)


def test_rows_past_32_bits():
    # 2^17 + 300 rows of 2^15: offsets past 2^32 in x
    rows, inner, outer = (1 << 17) + 300, 1 << 15, 64
    x = torch.zeros(rows, inner, dtype=torch.uint8, device=DEV)
    g = gen(21)
    tail, tail_scales = random_quantized(g, 300, inner)
    x[-300:] = tail.view(torch.uint8)
    xs = torch.full((rows, 256), 110, dtype=torch.uint8, device=DEV)
    xs[-300:] = tail_scales.view(torch.uint8) - 17
    w, ws = random_quantized(g, 2, outer, inner, down=128)
    off = torch.tensor([0, rows - 200, rows], dtype=torch.int32, device=DEV)
    got = rs.expert_matmul_quantized(x.view(torch.float8_e4m3fn), xs.view(E8M0), w, ws, off)
    assert bool((got[:-300] == 0).all())
    y, z, mag = plain(x[-300:].view(torch.float8_e4m3fn), xs[-300:].view(E8M0), w, ws,
                      torch.tensor([0, 100, 300], dtype=torch.int32))
    check(y, z, got[-300:], None, mag, inner, torch.bfloat16)


@pytest.mark.parametrize("rows", [0, 1])
def test_no_rows_and_one(way, rows):
    x, xs, w, ws, off = operands([rows, 0], 256, 136)
    got = rs.expert_matmul_quantized(x, xs, w, ws, off)
    y, z, mag = plain(x, xs, w, ws, off)
    check(y, z, got, None, mag, 256, torch.bfloat16)
    q, scales = rs.expert_matmul_quantized(x, xs, w, ws, off, quantize=True)
    assert q.shape == (rows, 136) and scales.shape == (rows, 2)
    if rows:
        check_quantized(q, scales, y, mag, 256)
