"""The expert operators on inputs as long as their interface takes: reductions
that last longer than any other wait of a kernel's own."""
import pytest

import lsd_radix_sort_key_gb300 as rs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from expert_util import DEV, gen  # noqa: E402

SMS = torch.cuda.get_device_properties(0).multi_processor_count


@pytest.fixture(scope="module", autouse=True)
def built():
    rs.build()
    rs.lib()


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
