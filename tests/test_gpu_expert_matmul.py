"""expert_matmul and its gradient on the GPU against plain 64-bit forms
(bounds in expert_util)."""
import pytest

import lsd_radix_sort_key_gb300 as rs
from lsd_radix_sort_key_gb300 import experts

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from expert_util import (DEV, TYPES, UNIT, gen, grad_bounds, held, matmul_bounds, plain_matmul,  # noqa: E402
                         plain_matmul_grad)

ACTS = ["none", "relu", "gelu", "silu"]


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


def make(counts, unused, inner, outer, dtype, seed, bias=True, residual=False):
    g = gen(seed)
    rows = sum(counts) + unused
    edge = [0]
    for c in counts:
        edge.append(edge[-1] + c)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, device=DEV, generator=g) * scale).to(dtype)

    return dict(x=normal(rows, inner), w=normal(len(counts), outer, inner, scale=max(inner, 1) ** -0.5),
                offsets=torch.tensor(edge, dtype=torch.int32, device=DEV),
                bias=normal(len(counts), outer) if bias else None, residual=normal(rows, outer) if residual else None)


def check_forward(a, act, dtype):
    y, pre = rs.expert_matmul(a["x"], a["w"], a["offsets"], bias=a["bias"], activation=act, residual=a["residual"],
                              return_pre=True)
    want, z, mag = plain_matmul(a["x"], a["w"], a["offsets"], a["bias"], act, a["residual"])
    by, bz = matmul_bounds(want, z, mag, a["x"].shape[1], dtype, a["residual"])
    held(y, want, by)
    held(pre, z, bz)
    last = int(a["offsets"][-1])
    assert not y[last:].any() and not pre[last:].any()
    only = rs.expert_matmul(a["x"], a["w"], a["offsets"], bias=a["bias"], activation=act, residual=a["residual"])
    assert torch.equal(only, y)
    return y, pre


def check_grad(a, act, dtype, seed):
    rows, outer = a["x"].shape[0], a["w"].shape[1]
    dy = torch.randn(rows, outer, device=DEV, generator=gen(seed + 1)).to(dtype)
    pre = torch.randn(rows, outer, device=DEV, generator=gen(seed + 2)).to(dtype) if act != "none" else None
    got = rs.expert_matmul_grad(dy, a["x"], a["w"], a["offsets"], pre=pre, activation=act)
    want, mags, errs = plain_matmul_grad(dy, a["x"], a["w"], a["offsets"], pre, act)
    most = int((a["offsets"][1:] - a["offsets"][:-1]).max())
    for g, v, b in zip(got, want, grad_bounds(want, mags, errs, (outer, most, most), dtype)):
        held(g, v, b)
    return dy, pre, got


COUNTS = [[1], [0, 0, 5, 0], [64, 128, 129], [1, 2, 3, 0, 130, 63, 65, 257], [300]]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("inner,outer", [(64, 64), (8, 8), (256, 264), (136, 520), (77, 65), (1, 1), (200, 1), (1, 129)])
@pytest.mark.parametrize("case", range(len(COUNTS)))
def test_forward_and_gradient(dt, inner, outer, case):
    dtype = TYPES[dt]
    act = ACTS[(case + inner) % 4]
    a = make(COUNTS[case], case * 3, inner, outer, dtype, case, residual=case % 2 == 0)
    check_forward(a, act, dtype)
    check_grad(a, act, dtype, case)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
def test_epilogues(way, dt, act, bias, residual):
    dtype = TYPES[dt]
    a = make([70, 0, 200, 3], 9, 192, 320, dtype, 5, bias, residual)
    check_forward(a, act, dtype)
    check_grad(a, act, dtype, 6)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("counts,inner,outer", [([1] * 64, 512, 384), ([0] * 31 + [7], 1024, 256),
                                                ([3, 0, 9, 17, 33, 1, 5, 2], 2048, 1032), ([16] * 300, 64, 72),
                                                ([1000, 500, 0, 1548], 1000, 1160), ([4096], 1024, 512),
                                                ([129] * 13, 72, 1024), ([700, 1, 0, 15, 64, 63, 65, 17], 264, 520),
                                                ([2000, 3], 136, 776), ([3000, 70], 128, 256), ([5001], 64, 128),
                                                ([777, 0, 1500, 64], 256, 136), ([9], 4096, 512), ([40, 2], 2048, 300),
                                                ([1, 0, 200, 31, 5], 1024, 128), ([6000, 2500], 512, 1032),
                                                ([1100, 129, 700, 640, 64, 900], 2048, 2056)])
def test_larger(dt, counts, inner, outer):
    dtype = TYPES[dt]
    a = make(counts, 11, inner, outer, dtype, 7)
    check_forward(a, "silu", dtype)
    check_grad(a, "gelu", dtype, 8)


@pytest.mark.parametrize("counts,inner,outer", [([300, 257, 0, 400], 1000, 1160), ([2000], 1000, 1032),
                                                ([700, 1, 0, 150, 64, 63, 65, 17], 520, 1000), ([64], 1030, 999),
                                                ([63], 1030, 999), ([64] * 40, 65, 193)])
def test_larger_float32(counts, inner, outer):
    a = make(counts, 11, inner, outer, torch.float32, 41)
    check_forward(a, "gelu", torch.float32)
    check_grad(a, "gelu", torch.float32, 42)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows", [2600, 5200, 10400, 20000])
@pytest.mark.parametrize("outer", [2056, 2055])
def test_gradient_of_many_rows(dt, rows, outer):
    a = make([rows // 2 - 7, 0, 7, rows // 2 - 40], 40, 8, outer, TYPES[dt], 43)
    check_grad(a, "silu", TYPES[dt], 44)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("inner,outer", [(128, 256), (130, 72)])
def test_layouts(way, dt, inner, outer):
    """Rows with a stride, unaligned bases, weights stored transposed, shared by all experts, or in a wider array."""
    dtype, g = TYPES[dt], gen(31)
    a = make([100, 0, 61, 7], 4, inner, outer, dtype, 9, residual=True)
    rows = a["x"].shape[0]

    def inside(t, first, pad):
        wide = torch.randn(t.shape[:-1] + (t.shape[-1] + pad,), device=DEV, generator=g).to(dtype)
        wide[..., first:first + t.shape[-1]] = t
        return wide[..., first:first + t.shape[-1]]

    for first, pad in ((0, 16), (8, 32), (3, 5)):
        b = dict(a, x=inside(a["x"], first, pad), w=inside(a["w"], first, pad), bias=inside(a["bias"], first, pad),
                 residual=inside(a["residual"], first, pad))
        check_forward(b, "silu", dtype)
        check_grad(b, "silu", dtype, 10)
    t = dict(a, w=a["w"].transpose(1, 2).contiguous().transpose(1, 2))
    check_forward(t, "gelu", dtype)
    check_grad(t, "gelu", dtype, 11)
    shared = dict(a, w=a["w"][:1].expand(4, outer, inner), bias=a["bias"][:1].expand(4, outer),
                  residual=a["residual"][:1].expand(rows, outer))
    check_forward(shared, "none", dtype)
    check_grad(shared, "relu", dtype, 12)
    one = dict(a, x=a["x"][:1].expand(rows, inner))
    check_forward(one, "relu", dtype)
    check_grad(one, "none", dtype, 13)


@pytest.mark.parametrize("dt", TYPES)
def test_bad_numbers_stay_in_their_rows(dt):
    """NaN and infinities in unused rows, in other experts' rows and weights do not spread."""
    dtype = TYPES[dt]
    a = make([40, 33, 0, 90], 20, 136, 200, dtype, 14)
    clean, cleanp = check_forward(a, "silu", dtype)
    dy, pre, (dx, dw, db) = check_grad(a, "silu", dtype, 15)
    x, w, bad_dy, bad_pre = a["x"].clone(), a["w"].clone(), dy.clone(), pre.clone()
    nan, inf = float("nan"), float("inf")
    for t in (x, bad_dy, bad_pre):
        t[163:] = nan
    x[40:73], w[1], bad_dy[40:73] = inf, nan, nan
    w[2] = nan
    keep = torch.ones(183, dtype=torch.bool, device=DEV)
    keep[40:73] = False
    y, p = rs.expert_matmul(x, w, a["offsets"], bias=a["bias"], activation="silu", return_pre=True)
    assert torch.equal(y[keep], clean[keep]) and torch.equal(p[keep], cleanp[keep])
    assert torch.isnan(p[40:73].float()).all()
    gx, gw, gb = rs.expert_matmul_grad(bad_dy, x, w, a["offsets"], pre=bad_pre, activation="silu")
    assert torch.equal(gx[keep], dx[keep])
    for e in (0, 2, 3):
        assert torch.equal(gw[e], dw[e]) and torch.equal(gb[e], db[e])
    assert torch.isnan(gw[1].float()).all() and torch.isnan(gb[1].float()).all()
    # one row's NaN reaches that row alone
    x = a["x"].clone()
    x[7, 3] = nan
    y = rs.expert_matmul(x, a["w"], a["offsets"], bias=a["bias"], activation="relu")
    assert torch.isnan(y[7].float()).all() and not torch.isnan(y[:7].float()).any() and not torch.isnan(y[8:].float()).any()


@pytest.mark.parametrize("dt", TYPES)
def test_wrong_offsets_stay_inside_the_arrays(dt):
    dtype = TYPES[dt]
    a = make([100, 100, 100], 0, 64, 128, dtype, 16)
    dy = torch.randn(300, 128, device=DEV).to(dtype)
    for off in ([0, 200, 100, 300], [5, 100, 200, 1 << 30], [0, -7, 50, 60], [0, 1 << 30, -1, 0]):
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        # what the clamped offsets say
        top, fixed = 0, [0]
        for v in off[1:]:
            top = max(top, min(max(v, 0), 300))
            fixed.append(top)
        f = torch.tensor(fixed, dtype=torch.int32, device=DEV)
        assert torch.equal(rs.expert_matmul(a["x"], a["w"], o, bias=a["bias"]),
                           rs.expert_matmul(a["x"], a["w"], f, bias=a["bias"]))
        for g, h in zip(rs.expert_matmul_grad(dy, a["x"], a["w"], o), rs.expert_matmul_grad(dy, a["x"], a["w"], f)):
            assert torch.equal(g, h)


@pytest.mark.parametrize("dt", TYPES)
def test_empty(way, dt):
    dtype = TYPES[dt]
    a = make([0, 0], 0, 64, 96, dtype, 17)
    assert rs.expert_matmul(a["x"], a["w"], a["offsets"]).shape == (0, 96)
    dx, dw, db = rs.expert_matmul_grad(torch.empty(0, 96, dtype=dtype, device=DEV), a["x"], a["w"], a["offsets"])
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    a = make([0, 0], 50, 64, 96, dtype, 18)  # rows, none of them used
    y, p = rs.expert_matmul(a["x"], a["w"], a["offsets"], bias=a["bias"], return_pre=True)
    assert y.shape == (50, 96) and not y.any() and not p.any()
    a = make([3, 4], 1, 0, 96, dtype, 19)  # a product of nothing: the bias alone
    y = rs.expert_matmul(a["x"], a["w"], a["offsets"], bias=a["bias"])
    want = torch.cat([a["bias"][:1].expand(3, 96), a["bias"][1:].expand(4, 96), torch.zeros_like(a["bias"][:1])])
    assert torch.equal(y, want)
    a = make([3, 4], 1, 64, 0, dtype, 20, bias=False)
    assert rs.expert_matmul(a["x"], a["w"], a["offsets"]).shape == (8, 0)
    dx, dw, _ = rs.expert_matmul_grad(torch.empty(8, 0, dtype=dtype, device=DEV), a["x"], a["w"], a["offsets"])
    assert dx.shape == (8, 64) and not dx.any() and dw.shape == (2, 0, 64)


def test_parts_of_the_gradient(way):
    a = make([50, 60], 5, 128, 136, torch.bfloat16, 21)
    dy, pre, full = check_grad(a, "silu", torch.bfloat16, 22)
    for want in range(8):
        need = [bool(want & 1), bool(want & 2), bool(want & 4)]
        got = rs.expert_matmul_grad(dy, a["x"], a["w"], a["offsets"], pre=pre, activation="silu", need_dx=need[0],
                                    need_dw=need[1], bias=need[2])
        for g, f, n in zip(got, full, need):
            assert (g is None) if not n else torch.equal(g, f)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", TYPES)
def test_gradients_against_differences(dt, act):
    dtype = TYPES[dt]
    a = make([17, 0, 40], 3, 40, 24, dtype, 23)
    g = gen(24)
    # stay clear of relu's corner, where there is no derivative: the step moves z by far less than this
    z = plain_matmul(a["x"], a["w"], a["offsets"], a["bias"])[1]
    pre64 = z.to(dtype)
    c = torch.randn(z.shape, device=DEV, generator=g).to(dtype)
    if act == "relu":
        c[(z.abs() < 1e-2)] = 0
    v = [torch.randn(t.shape, device=DEV, generator=g, dtype=torch.float64) for t in (a["x"], a["w"], a["bias"])]

    def value(h):
        p = [t.double() + h * d for t, d in zip((a["x"], a["w"], a["bias"]), v)]
        return float((plain_matmul(p[0], p[1], a["offsets"], p[2], act)[0] * c.double()).sum())

    h = 1e-5
    slope = (value(h) - value(-h)) / (2 * h)
    got = rs.expert_matmul_grad(c, a["x"], a["w"], a["offsets"], pre=pre64, activation=act)
    found = sum(float((t.double() * d).sum()) for t, d in zip(got, v))
    want, mags, errs = plain_matmul_grad(c, a["x"], a["w"], a["offsets"], pre64, act)
    allow = sum(float((b * d.abs()).sum()) for b, d in zip(grad_bounds(want, mags, errs, (24, 40, 40), dtype), v))
    if act in ("gelu", "silu"):
        # the derivative is taken at z rounded to the type: |act''| <= 0.8, so dz moves by at most 0.8 u |z| |c|
        _, moved, _ = plain_matmul_grad((c.double() * 0.8 * UNIT[dtype] * z.abs()), a["x"], a["w"], a["offsets"])
        allow += sum(float((m * d.abs()).sum()) for m, d in zip(moved, v))
    assert abs(found - slope) <= allow + 1e-6 * max(1.0, abs(slope))


def test_another_stream_and_graph(way):
    a = make([50, 60, 1], 5, 128, 136, torch.bfloat16, 25)
    args = (a["x"], a["w"], a["offsets"])
    dy = torch.randn(116, 136, device=DEV).bfloat16()
    y, pre = rs.expert_matmul(*args, bias=a["bias"], activation="silu", return_pre=True)
    want = rs.expert_matmul_grad(dy, *args, pre=pre, activation="silu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        y2, pre2 = rs.expert_matmul(*args, bias=a["bias"], activation="silu", return_pre=True, stream=s)
        got = rs.expert_matmul_grad(dy, *args, pre=pre2, activation="silu", stream=s)
        side.synchronize()
        assert torch.equal(y, y2) and all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, pre3 = rs.expert_matmul(*args, bias=a["bias"], activation="silu", return_pre=True)
        got = rs.expert_matmul_grad(dy, *args, pre=pre3, activation="silu")
    a["x"].normal_()
    a["offsets"].copy_(torch.tensor([0, 3, 70, 111], dtype=torch.int32))
    graph.replay()
    y4, pre4 = rs.expert_matmul(*args, bias=a["bias"], activation="silu", return_pre=True)
    assert torch.equal(y3, y4)
    for p, q in zip(got, rs.expert_matmul_grad(dy, *args, pre=pre4, activation="silu")):
        assert torch.equal(p, q)


def test_same_call_same_bits():
    a = make([700, 0, 1300, 48], 100, 1024, 1032, torch.bfloat16, 26)
    dy = torch.randn(2148, 1032, device=DEV).bfloat16()
    first = rs.expert_matmul_grad(dy, a["x"], a["w"], a["offsets"])
    y = rs.expert_matmul(a["x"], a["w"], a["offsets"])
    for _ in range(10):
        assert torch.equal(rs.expert_matmul(a["x"], a["w"], a["offsets"]), y)
        for p, q in zip(rs.expert_matmul_grad(dy, a["x"], a["w"], a["offsets"]), first):
            assert torch.equal(p, q)


# a reduction cut over a cluster, tiles of one block (128 and 256 columns), pairs of blocks
@pytest.mark.parametrize("rows,inner,outer", [(70, 1024, 512), (250, 256, 512), (900, 256, 4096), (6000, 1024, 1024)])
def test_a_wait_that_runs_out_is_reported(rows, inner, outer):
    a = make([rows + 50, rows - 50], 0, inner, outer, torch.bfloat16, 27)
    temp = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    y = rs.expert_matmul(a["x"], a["w"], a["offsets"], temp=temp)
    assert rs.rs_expert_matmul_status(temp) == 0
    out = torch.empty_like(y)
    d = rs.ExpertMatmulDesc(2, 0, 2, 2 * rows, inner, outer, a["offsets"].data_ptr(), a["x"].data_ptr(), inner,
                            a["w"].data_ptr(), inner * outer, inner, 1)
    d.y, d.y_stride, d.temp, d.temp_bytes = out.data_ptr(), outer, temp.data_ptr(), temp.numel()
    d.stream, d.stall_tile = torch.cuda.current_stream().cuda_stream, 4
    assert rs.rs_expert_matmul(d) == 0
    assert rs.rs_expert_matmul_status(temp) == 5  # RS_ERR_DEVICE_TIMEOUT
    d.stall_tile = 0  # the next call works
    assert rs.rs_expert_matmul(d) == 0
    assert rs.rs_expert_matmul_status(temp) == 0 and torch.equal(out, y)


def test_refusals_are_worded_whatever_the_way(way):
    a = make([3, 4], 1, 64, 96, torch.bfloat16, 30)
    x, w, off = a["x"], a["w"], a["offsets"]
    for kw, error in ((dict(activation="tanh"), ValueError), (dict(bias=a["bias"].float()), TypeError),
                      (dict(bias=a["bias"][:1]), ValueError), (dict(residual=x), ValueError)):
        with pytest.raises(error):
            rs.expert_matmul(x, w, off, **kw)
    with pytest.raises(ValueError):
        rs.expert_matmul(x, w, off[:-1])
    with pytest.raises(TypeError):
        rs.expert_matmul(x, w, off.long())
    with pytest.raises(TypeError):
        rs.expert_matmul_grad(x.new_zeros(8, 96), x, w, off, activation="silu")
    with pytest.raises(rs.RadixSortError):
        rs.expert_sort(torch.zeros(3, dtype=torch.int64, device=DEV), 2000)
    with pytest.raises(ValueError):
        rs.expert_dispatch(x.t(), torch.zeros(64, 1, dtype=torch.int32, device=DEV), off)
    with pytest.raises(TypeError):
        rs.expert_combine(x, None, torch.zeros(8, 1, dtype=torch.int32, device=DEV), off)


def test_a_gradient_being_recorded_is_no_obstacle(way):
    # the calls compute values only; tensors that require a gradient are as good as others
    a = make([30, 40], 0, 64, 96, torch.bfloat16, 31)
    want = rs.expert_matmul(a["x"], a["w"], a["offsets"])
    assert torch.equal(rs.expert_matmul(a["x"].requires_grad_(), torch.nn.Parameter(a["w"]), a["offsets"]), want)
