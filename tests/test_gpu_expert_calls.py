"""The expert operators' calls at their edges: the caller's scratch, flags that
are not bools, numbers past 32 bits, layouts that only the C interface can name,
calls from several host threads, and waits of a gradient that run out."""
import threading

import pytest

import lsd_radix_sort_key_gb300 as rs
from lsd_radix_sort_key_gb300 import experts

pytestmark = pytest.mark.gpu

np = pytest.importorskip("numpy")
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from expert_util import (DEV, TYPES, gen, grad_bounds, held, matmul_bounds, plain_matmul,  # noqa: E402
                         plain_matmul_grad, plain_order)


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


def product(counts, inner, outer, dtype=torch.bfloat16, seed=1):
    g = gen(seed)
    off = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device=DEV)
    x = torch.randn(sum(counts), inner, device=DEV, generator=g).to(dtype)
    w = torch.randn(len(counts), outer, inner, device=DEV, generator=g).to(dtype)
    return x, w, off


# --------------------------------------------------------- caller's scratch

def calls(x, w, off, dy):
    """Both products, as functions of temp and the other keywords."""
    return (lambda **kw: (rs.expert_matmul(x, w, off, **kw),),
            lambda **kw: rs.expert_matmul_grad(dy, x, w, off, **kw))


def test_scratch_that_is_not_ours_to_use_is_refused():
    # refused on the host, before anything is enqueued
    x, w, off = product([30, 41], 64, 96)
    for call in calls(x, w, off, torch.randn(71, 96, device=DEV).bfloat16()):
        for temp, error in ((torch.empty(1 << 20, dtype=torch.uint8), ValueError),  # the host's
                            (torch.empty(1 << 20, dtype=torch.uint8, device="meta"), ValueError),
                            (torch.empty(1, dtype=torch.uint8, device=DEV).expand(1 << 20), ValueError),
                            (torch.empty(1 << 21, dtype=torch.uint8, device=DEV)[::2], ValueError),
                            (torch.empty(1 << 18, device=DEV), TypeError), (1 << 40, TypeError),
                            (torch.empty(100, dtype=torch.uint8, device=DEV), rs.RadixSortError),
                            (torch.empty(1 << 20, dtype=torch.uint8, device=DEV)[16:], rs.RadixSortError)):
            with pytest.raises(error):
                call(temp=temp)
        temp = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
        for got, want in zip(call(temp=temp), call()):
            assert torch.equal(got, want)


def test_scratch_of_another_stream_is_kept_until_that_stream_has_passed():
    x, w, off = product([30, 41], 64, 96)
    size = 33 << 20  # a block of its own in torch's allocator
    for call in calls(x, w, off, torch.randn(71, 96, device=DEV).bfloat16()):
        want, side = call(), torch.cuda.Stream()
        torch.cuda.synchronize()
        temp = torch.empty(size, dtype=torch.uint8, device=DEV)
        where = temp.data_ptr()
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000_000)  # half a second: the call is still to come when temp goes
        got = call(temp=temp, stream=side)
        del temp
        again = torch.empty(size, dtype=torch.uint8, device=DEV)
        assert not side.query() and again.data_ptr() != where
        side.synchronize()
        assert all(torch.equal(g, v) for g, v in zip(got, want))


# ------------------------------------------------------------------- flags

@pytest.mark.parametrize("yes,no", [(1, 0), (np.True_, np.False_), ("yes", ""), (True, None)])
def test_flags_are_taken_by_their_truth(way, yes, no):
    x, w, off = product([30, 0, 41], 64, 96)
    dy = torch.randn(71, 96, device=DEV, generator=gen(2)).bfloat16()
    y, pre = rs.expert_matmul(x, w, off, activation="silu", return_pre=True)
    got = rs.expert_matmul(x, w, off, activation="silu", return_pre=yes)
    assert isinstance(got, tuple) and torch.equal(got[0], y) and torch.equal(got[1], pre)
    assert torch.equal(rs.expert_matmul(x, w, off, activation="silu", return_pre=no), y)
    full = rs.expert_matmul_grad(dy, x, w, off, pre=pre, activation="silu")
    for want in range(8):
        need = [bool(want >> i & 1) for i in range(3)]
        flags = [yes if n else no for n in need]
        got = rs.expert_matmul_grad(dy, x, w, off, pre=pre, activation="silu", need_dx=flags[0], need_dw=flags[1],
                                    bias=flags[2])
        for g, f, n in zip(got, full, need):
            assert (g is None) if not n else torch.equal(g, f)


def test_a_flag_without_a_truth_is_refused(way):
    x, w, off = product([30, 41], 64, 96)
    dy = torch.randn(71, 96, device=DEV).bfloat16()
    with pytest.raises(RuntimeError):  # torch's own: a tensor of many values is neither
        rs.expert_matmul_grad(dy, x, w, off, bias=torch.zeros(2, 96, device=DEV))


# ----------------------------------------------------------------- numbers

def test_numbers_past_32_bits_are_refused(way):
    # not taken by their low 32 bits: 2^32 + 1 is not 1
    many = (1 << 32) + 1
    ids = torch.zeros(6, dtype=torch.int64, device=DEV)
    for count in (many, 1 << 32, -(1 << 32) + 1, 0, 1025):
        with pytest.raises(rs.RadixSortError):
            rs.expert_sort(ids, count)
    position = torch.empty(1, many, dtype=torch.int32, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    one = torch.zeros(1, 1, dtype=torch.float16, device=DEV)
    for call in (lambda: rs.expert_dispatch(one, position, off),
                 lambda: rs.expert_dispatch_grad(one.expand(many, 1), position, off),
                 lambda: rs.expert_combine(one.expand(many, 1), one.expand(1, many), position, off),
                 lambda: rs.expert_combine_grad(one, one.expand(many, 1), one.expand(1, many), position, off)):
        with pytest.raises(rs.RadixSortError):
            call()


# ------------------------------------------ layouts of the C interface alone

@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("inner,outer,so,si", [(1, 40, 6, 9), (1, 40, 6, 1), (1, 40, 1, 9), (1, 40, 8, 16), (24, 1, 9, 5),
                                               (24, 1, 9, 1), (24, 1, 1, 5), (1, 1, 9, 5)])
def test_weights_of_one_column_or_row_at_any_strides(dt, act, inner, outer, so, si):
    dtype, count = TYPES[dt], 3
    g, span = gen(inner + so), (outer - 1) * so + (inner - 1) * si + 1
    base = torch.randn(count, span + 11, device=DEV, generator=g).to(dtype)
    at = torch.arange(outer, device=DEV)[:, None] * so + torch.arange(inner, device=DEV) * si
    w = base[:, at]  # what the call has to read
    counts = [17, 0, 30]
    x, _, off = product(counts, inner, outer, dtype, 5)
    rows = sum(counts)
    dy = torch.randn(rows, outer, device=DEV, generator=g).to(dtype)
    y, pre = (torch.empty(rows, outer, dtype=dtype, device=DEV) for _ in range(2))
    temp = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    d = rs.ExpertMatmulDesc(list(TYPES).index(dt), rs.ACTIVATIONS[act], count, rows, inner, outer, off.data_ptr(),
                            x.data_ptr(), inner, base.data_ptr(), base.stride(0), so, si)
    d.y, d.y_stride, d.pre, d.pre_stride = y.data_ptr(), outer, pre.data_ptr(), outer
    d.temp, d.temp_bytes, d.stream = temp.data_ptr(), temp.numel(), torch.cuda.current_stream().cuda_stream
    assert rs.rs_expert_matmul_temp_bytes(d) <= temp.numel() and rs.rs_expert_matmul(d) == 0
    want, z, mag = plain_matmul(x, w, off, None, act)
    by, bz = matmul_bounds(want, z, mag, inner, dtype)
    held(y, want, by)
    held(pre, z, bz)
    dx, dw = torch.empty_like(x), torch.empty(count, outer, inner, dtype=dtype, device=DEV)
    d.y, d.dx, d.dx_stride, d.dw = dy.data_ptr(), dx.data_ptr(), inner, dw.data_ptr()
    assert rs.rs_expert_matmul_grad_temp_bytes(d) <= temp.numel() and rs.rs_expert_matmul_grad(d) == 0
    want, mags, errs = plain_matmul_grad(dy, x, w, off, pre, act)
    for got, v, b in zip((dx, dw), want, grad_bounds(want, mags, errs, (outer, 30, 30), dtype)):
        held(got, v, b)


# ------------------------------------------------------------ host threads

def in_threads(*calls):
    """Runs the calls at once, one thread and stream each; the first error of any is raised here."""
    errors, start = [], threading.Barrier(len(calls))

    def run(call):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            call(stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("n,few,many", [(1500, 400, 500), (20_000, 100, 500), (20_000, 600, 1024), (60_000, 300, 511)])
def test_sorts_of_two_threads(n, few, many):
    # the kernels' shared memory goes by the number of experts; the C calls run without the interpreter's lock
    def sorts(count, seed):
        ids = torch.randint(-1, count, (n,), device=DEV, generator=gen(seed))
        got = [torch.empty(k, dtype=torch.int32, device=DEV) for k in (n, n, count + 1)]
        tb = rs.rs_expert_sort_temp_bytes(n, count)
        temp = torch.empty(max(tb, 1), dtype=torch.uint8, device=DEV)
        want = plain_order(ids, count)
        torch.cuda.synchronize()

        def call(stream):
            s = stream.cuda_stream
            assert not any(rs.rs_expert_sort(ids, 8, n, count, *got, temp, tb, s) for _ in range(20_000))
            stream.synchronize()
            assert all(torch.equal(g.cpu(), w.flatten()) for g, w in zip(got, want))
        return call

    in_threads(sorts(few, 1), sorts(many, 2))


@pytest.mark.parametrize("inner,outer", [(64, 64), (1024, 128)])
def test_products_of_two_threads(inner, outer):
    def products(count, seed):
        x, w, off = product([1] * count, inner, outer, seed=seed)
        dy = torch.randn(count, outer, device=DEV, generator=gen(seed)).bfloat16()
        want = (rs.expert_matmul(x, w, off), *rs.expert_matmul_grad(dy, x, w, off))
        torch.cuda.synchronize()

        def call(stream):
            for _ in range(1500):
                got = (rs.expert_matmul(x, w, off, stream=stream), *rs.expert_matmul_grad(dy, x, w, off, stream=stream))
            stream.synchronize()
            assert all(torch.equal(g, v) for g, v in zip(got, want))
        return call

    in_threads(products(8, 3), products(1024, 4))


# ------------------------------------------------------ waits that run out

# dw cut over a cluster, by tiles of one block (128 and 256 columns), by pairs; then dx
@pytest.mark.parametrize("which,rows,inner,outer", [("dw", 2000, 128, 128), ("dw", 250, 512, 256), ("dw", 1000, 4096, 384),
                                                    ("dw", 8000, 4096, 384), ("dx", 70, 512, 1024), ("dx", 6000, 1024, 1024)])
def test_a_wait_that_runs_out_in_a_gradient_is_reported(which, rows, inner, outer):
    x, w, off = product([rows // 2 + 5, rows // 2 - 5], inner, outer)  # both end in a partial slice
    dy = torch.randn(rows, outer, device=DEV, generator=gen(6)).bfloat16()
    temp = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    want = rs.expert_matmul_grad(dy, x, w, off, bias=False, need_dx=which == "dx", need_dw=which == "dw", temp=temp)
    want = want[0] if which == "dx" else want[1]
    assert rs.rs_expert_matmul_status(temp) == 0
    out = torch.empty_like(want)
    d = rs.ExpertMatmulDesc(2, 0, 2, rows, inner, outer, off.data_ptr(), x.data_ptr(), inner, w.data_ptr(),
                            inner * outer, inner, 1)
    d.y, d.y_stride, d.dx_stride = dy.data_ptr(), outer, inner
    setattr(d, which, out.data_ptr())
    d.temp, d.temp_bytes, d.stream = temp.data_ptr(), temp.numel(), torch.cuda.current_stream().cuda_stream
    d.stall_tile = 2
    assert rs.rs_expert_matmul_grad(d) == 0
    assert rs.rs_expert_matmul_status(temp) == 5  # RS_ERR_DEVICE_TIMEOUT
    d.stall_tile = 0  # the next call works
    assert rs.rs_expert_matmul_grad(d) == 0
    assert rs.rs_expert_matmul_status(temp) == 0 and torch.equal(out, want)
