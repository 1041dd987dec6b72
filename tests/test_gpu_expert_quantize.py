"""Quantised rows and weights against their definition, to the bit."""
import pytest

import lsd_radix_sort_key_gb300 as rs
from lsd_radix_sort_key_gb300 import experts

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from block_util import E4M3, E8M0, plain_quantize, same  # noqa: E402
from expert_util import DEV, TYPES, gen, make_plan  # noqa: E402


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


def rows_of(g, r, w, dtype, wild=True):
    """Rows of very different sizes, zeros and ties among them."""
    x = torch.randn(r, w, device=DEV, generator=g)
    if wild:
        x = x * torch.exp2(torch.randint(-30 if dtype != torch.float16 else -12, 12, (r, 1), device=DEV, generator=g).float())
        x = torch.where(torch.rand(r, w, device=DEV, generator=g) < 0.1, torch.zeros_like(x), x)
        x[::5] = torch.round(x[::5] * 8) / 8  # ties
        if r > 3:
            x[3] = 0
    return x.to(dtype)


def check(q, scales, x, down=1):
    want, want_scales = plain_quantize(x, down)
    assert q.dtype == E4M3 and scales.dtype == E8M0
    assert q.shape == x.shape and tuple(scales.shape) == tuple(want_scales.shape)
    assert q.stride(0) % 16 == 0 and q.data_ptr() % 16 == 0
    assert torch.equal(scales.double(), want_scales)
    assert same(q, want)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("r,w", [(1, 1), (1, 128), (3, 127), (5, 129), (7, 8), (64, 4096), (33, 1032), (9, 1037), (1000, 72),
                                 (2, 16384), (4099, 264), (20000, 24)])
def test_rows(way, dt, r, w):
    x = rows_of(gen(r + w), r, w, TYPES[dt])
    check(*rs.expert_quantize(x), x)


@pytest.mark.parametrize("dt", TYPES)
def test_the_largest_smallest_and_borders(dt):
    dtype = TYPES[dt]
    top, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    x = torch.zeros(12, 256, device=DEV, dtype=dtype)
    x[0, 0], x[0, 1] = top, 1.0
    x[1, 5] = -top
    x[2, 0] = tiny
    x[3, 0] = tiny / 4
    x[4, 0] = 448.0            # exactly at the border: scale 1
    x[5, 0] = 448.0 * (1 + 2 * torch.finfo(dtype).eps)  # just past it: scale 2
    x[6, :2] = torch.tensor([448.0, 17.0], device=DEV)   # 17 is a tie between 16 and 18
    x[7, :4] = torch.tensor([448.0, 2.0**-10, 3 * 2.0**-10, 2.0**-9], device=DEV).to(dtype)  # below the normal range, ties
    x[8, 128] = -3.0
    x[9] = -0.0
    x[10, 7], x[10, 200] = 1.75, 1.8125
    check(*rs.expert_quantize(x), x)
    q, scales = rs.expert_quantize(x)
    assert float(scales[4, 0].float()) == 1 and float(scales[5, 0].float()) == 2
    assert float(q[6, 1].float()) == 16 and q[7, 1:4].float().tolist() == [0.0, 2.0**-8, 2.0**-9]
    assert float(scales[9, 0].float()) == 1


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("w", [256, 301])
def test_infinities_and_nan_stay_where_they_are(dt, w):
    x = rows_of(gen(3), 40, w, TYPES[dt])
    x[0, 3], x[0, 4] = float("inf"), float("nan")
    x[1, 200] = -float("inf")
    x[2] = float("nan")
    check(*rs.expert_quantize(x), x)
    q, scales = rs.expert_quantize_weights(x.view(1, 40, w))
    want, want_scales = plain_quantize(x, 128)
    assert same(q[0], want) and torch.equal(scales[0].double(), want_scales)


@pytest.mark.parametrize("dt", TYPES)
def test_strides_offsets_and_one_row_for_all(way, dt):
    g, dtype = gen(8), TYPES[dt]
    wide = rows_of(g, 50, 700, dtype)
    for x in (wide[:, 1:400], wide[:, 8:520], wide[:, 3:131], wide[::2, :512], wide[10:11].expand(30, 700), wide[1:2, 5:]):
        check(*rs.expert_quantize(x), x)


def test_padding_is_zero_and_nothing_else_is_written():
    x = rows_of(gen(1), 9, 37, torch.bfloat16)
    q = torch.full((11, 64), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((11, 3), 0x55, dtype=torch.uint8, device=DEV)
    assert rs.rs_expert_quantize("bfloat16", x, 37, 9, 37, q[1:], 64, s[1:], 3) == 0
    want, want_scales = plain_quantize(x)
    assert same(q[1:10, :37].contiguous().view(E4M3), want)
    assert torch.equal(s[1:10, :1].contiguous().view(E8M0).double(), want_scales)
    assert bool((q[1:10, 37:48] == 0).all()) and bool((q[1:10, 48:] == 0x55).all())
    assert bool((q[0] == 0x55).all()) and bool((q[10] == 0x55).all()) and bool((s[0] == 0x55).all())
    assert bool((s[10] == 0x55).all()) and bool((s[1:10, 1:] == 0x55).all())


@pytest.mark.parametrize("shape", [(0, 128), (5, 0), (0, 0)])
def test_nothing(way, shape):
    x = torch.empty(shape, device=DEV)
    q, scales = rs.expert_quantize(x)
    assert q.shape == shape and tuple(scales.shape) == (shape[0], -(-shape[1] // 128))


# --------------------------------------------------------------- dispatch

@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("t,k,e,w,drop", [(1, 1, 4, 128, 0.0), (64, 8, 128, 512, 0.0), (37, 3, 8, 1037, 0.3), (500, 2, 16, 72, 1.0),
                                          (5, 20, 32, 264, 0.2), (3001, 6, 160, 40, 0.1)])
def test_dispatch(way, dt, t, k, e, w, drop):
    x = rows_of(gen(t), t, w, TYPES[dt])
    position, offsets = make_plan(t, k, e, t + k, drop)
    q, scales = rs.expert_dispatch_quantized(x, position, offsets)
    want, want_scales = plain_quantize(x)
    rows = torch.zeros(t * k, w, dtype=torch.float64, device=DEV)
    rows_scales = torch.ones(t * k, want_scales.shape[1], dtype=torch.float64, device=DEV)
    for j in range(k):
        at = position[:, j].long()
        kept = at < offsets[-1]
        rows[at[kept]], rows_scales[at[kept]] = want[kept], want_scales[kept]
    assert same(q, rows) and torch.equal(scales.double(), rows_scales)
    # the same as quantising the dispatched rows
    q2, scales2 = rs.expert_quantize(rs.expert_dispatch(x, position, offsets))
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(scales.double(), scales2.double())


def test_a_bad_plan_writes_no_other_rows():
    x = rows_of(gen(4), 6, 64, torch.float16)
    position = torch.tensor([[0, -5], [1 << 30, 3], [12, 5], [7, 8], [9, 10], [11, 2]], dtype=torch.int32, device=DEV)
    offsets = torch.tensor([0, 1 << 30], dtype=torch.int32, device=DEV)  # more than there are: clamped
    q = torch.full((14, 64), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((14, 1), 0x55, dtype=torch.uint8, device=DEV)
    assert rs.rs_expert_dispatch_quantized("float16", x, 64, position, offsets[1:], 6, 2, 64, q[1:], 64, s[1:], 1) == 0
    want, _ = plain_quantize(x)
    written = {0: 0, 3: 1, 5: 2, 7: 3, 8: 3, 9: 4, 10: 4, 11: 5, 2: 5}
    for r in range(-1, 13):
        if r in written:
            assert same(q[r + 1:r + 2].view(E4M3), want[written[r]:written[r] + 1])
        else:
            assert bool((q[r + 1] == 0x55).all()) and int(s[r + 1]) == 0x55


# ---------------------------------------------------------------- weights

@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("e,n,k", [(1, 1, 1), (2, 128, 128), (3, 130, 257), (1, 1160, 1000), (2, 8, 1032), (4, 129, 16), (1, 1, 300),
                                   (2, 300, 1)])
@pytest.mark.parametrize("turned", [False, True])
def test_weights(way, dt, e, n, k, turned):
    g = gen(n + k)
    w = rows_of(g, e * n, k, TYPES[dt]).view(e, n, k)
    if turned:  # the same values with outer adjacent
        w = w.transpose(1, 2).contiguous().transpose(1, 2)
    q, scales = rs.expert_quantize_weights(w)
    assert q.shape == w.shape and tuple(scales.shape) == (e, -(-n // 128), -(-k // 128))
    for i in range(e):
        want, want_scales = plain_quantize(w[i], 128)
        assert same(q[i], want) and torch.equal(scales[i].double(), want_scales)
    # exchanged sides: the transposed values with the transposed scales
    qt, scales_t = rs.expert_quantize_weights(w.transpose(1, 2))
    assert torch.equal(qt.double(), q.double().transpose(1, 2))
    assert torch.equal(scales_t.double(), scales.double().transpose(1, 2))


@pytest.mark.parametrize("dt", TYPES)
def test_weights_of_other_strides(way, dt):
    big = rows_of(gen(9), 3 * 150, 400, TYPES[dt]).view(3, 150, 400)
    for w in (big[:, 3:141, 7:300], big[:, ::2, 16:272], big[::2], big[1:2].expand(3, 150, 400),
              big.transpose(1, 2)[:, 5:261, 1:140], big.transpose(1, 2)[:, :, 8:136]):
        q, scales = rs.expert_quantize_weights(w)
        for i in range(w.shape[0]):
            want, want_scales = plain_quantize(w[i], 128)
            assert same(q[i], want) and torch.equal(scales[i].double(), want_scales)


def test_past_32_bits():
    # 3 * 2^15 rows of 2^15: offsets of 3 * 2^30 values, and of rows beyond 2^31 bytes
    r, w = 3 << 15, 1 << 15
    x = torch.empty(r, w, dtype=torch.bfloat16, device=DEV).fill_(0.5)
    last = rows_of(gen(5), 130, w, torch.bfloat16)
    x[-130:] = last
    q, scales = rs.expert_quantize(x)
    check(q[-130:], scales[-130:], last)
    assert bool((q[:-130].view(torch.uint8)[::4097] == q[0, 0].view(torch.uint8)).all())
    del q, scales
    q, scales = rs.expert_quantize_weights(x.view(3, 1 << 15, w))
    want, want_scales = plain_quantize(last[2:], 128)
    assert same(q[2, -128:], want) and torch.equal(scales[2, -1:].double(), want_scales)
