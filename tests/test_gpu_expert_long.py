"""The expert operators on inputs as long as their interface takes: sorts whose
blocks go through several tiles, reductions that last longer than any other
wait of a kernel's own, and products whose element offsets pass 32 bits."""
import pytest

import lsd_radix_sort_key_gb300 as rs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from expert_util import DEV, TYPES, gen, plain_order  # noqa: E402

SMS = torch.cuda.get_device_properties(0).multi_processor_count


@pytest.fixture(scope="module", autouse=True)
def built():
    rs.build()
    rs.lib()


# ------------------------------------------------------------------- sorts

def check_sort(ids, count):
    for name, got, want in zip(("order", "position", "offsets"), rs.expert_sort(ids, count), plain_order(ids, count)):
        assert torch.equal(got.cpu(), want), name


# a block has one tile of 8192 slots up to SMS * 8192 slots, several above
@pytest.mark.parametrize("n", [SMS * 8192, SMS * 8192 + 1, 1_300_003, 5_000_011])
@pytest.mark.parametrize("count", [7, 257, 511, 512, 1024])
def test_sorts_of_several_tiles_per_block(n, count):
    g = gen(n + count)
    ids = torch.randint(0, count, (n,), device=DEV, generator=g)
    ids[torch.rand(n, device=DEV, generator=g) < 0.1] = -1
    check_sort(ids, count)


@pytest.mark.parametrize("n", [SMS * 8192 + 1, 3_000_001])
@pytest.mark.parametrize("count", [8, 1024])
def test_sorts_of_several_tiles_one_expert_takes_all_or_none(n, count):
    check_sort(torch.full((n,), count - 1, device=DEV, dtype=torch.int32), count)
    check_sort(torch.full((n,), -1, device=DEV), count)
    check_sort((n - 1 - torch.arange(n, device=DEV)) * count // n, count)


# -------------------------------------------------------------- reductions

def test_a_long_reduction_runs_to_its_end():
    # One block sums 2^30 rows of the first expert in one tile of dw, some four
    # seconds, and then the only other rows, those of the expert numbered SMS:
    # more experts than SMs, so the reduction is not cut over several blocks.
    count, rows, last = SMS + 8, 1 << 30, (1 << 30) - 64
    off = torch.full((count + 1,), last, dtype=torch.int32, device=DEV)
    off[0] = 0
    off[SMS + 1:] = last + 5
    x, dy = (torch.zeros(rows, 8, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    want = torch.zeros(count, 8, 8, device=DEV)
    g = gen(1)
    for row in (0, 63, 64, 123_456_789, last - 1, last, last + 4):  # small whole numbers: every sum is exact
        x[row], dy[row] = (torch.randint(-8, 9, (8,), device=DEV, generator=g).bfloat16() for _ in range(2))
        want[0 if row < last else SMS] += dy[row].float()[:, None] * x[row].float()
    x[last + 5:] = float("nan")  # unused rows
    w = torch.zeros(count, 8, 8, dtype=torch.bfloat16, device=DEV)
    temp = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    dw = rs.expert_matmul_grad(dy, x, w, off, bias=False, need_dx=False, temp=temp)[1]
    end.record()
    assert rs.rs_expert_matmul_status(temp) == 0
    assert begin.elapsed_time(end) > 2500  # ms: past the 2^32 clocks of the other waits
    assert torch.equal(dw.float(), want)


# ----------------------------------------------------------------- products

@pytest.mark.parametrize("dt", TYPES)
def test_products_past_32_bit_offsets(dt):
    # x and dy (or y and pre) of more than 2^32 elements, all zero but for rows of
    # small whole numbers at the ends and around 2^32 elements: every sum is exact
    dtype, g = TYPES[dt], gen(2)
    wide, narrow, rows = 2056, 8, (1 << 21) + (1 << 18) + 77
    at = (1 << 32) // wide
    marked = [0, 1, at - 1, at, at + 1, rows - 52, rows - 51]  # the last one lies past the last expert's rows
    off = torch.tensor([0, 5, at, rows - 51], dtype=torch.int32, device=DEV)
    expert = [0, 0, 1, 2, 2, 2]

    def some(width):
        t = torch.zeros(rows, width, dtype=dtype, device=DEV)
        for r in marked:
            t[r] = torch.randint(-4, 5, (width,), device=DEV, generator=g).to(dtype)
        return t

    def only_marked(t):
        left = t.clone()
        left[marked] = 0
        return not left.any()

    for inner, outer in ((wide, narrow), (narrow, wide)):
        x, dy = some(inner), some(outer)
        assert max(x.numel(), dy.numel()) > 1 << 32
        w = torch.randint(-2, 3, (3, outer, inner), device=DEV, generator=g).to(dtype)
        y, pre = rs.expert_matmul(x, w, off, activation="relu", return_pre=True)
        for r, e in zip(marked, expert):
            z = (w[e].double() @ x[r].double()).to(dtype)
            assert torch.equal(pre[r], z) and torch.equal(y[r], z.clamp(min=0))
        assert not y[marked[-1]].any() and only_marked(y) and only_marked(pre)
        dx, dw, db = rs.expert_matmul_grad(dy, x, w, off, pre=pre, activation="relu")
        want_w, want_b = torch.zeros(3, outer, inner, dtype=torch.float64, device=DEV), torch.zeros(3, outer, device=DEV)
        for r, e in zip(marked, expert):
            dz = dy[r].double() * (pre[r] > 0)
            assert torch.equal(dx[r], (dz @ w[e].double()).to(dtype))
            want_w[e] += dz[:, None] * x[r].double()
            want_b[e] += dz.float()
        assert not dx[marked[-1]].any() and only_marked(dx)
        assert torch.equal(dw, want_w.to(dtype)) and torch.equal(db, want_b.to(dtype))
