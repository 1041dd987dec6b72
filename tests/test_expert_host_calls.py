"""What the Python forms of the expert operators check themselves, as far as it
needs no GPU."""
import pytest

from lsd_radix_sort_key_gb300 import _build, experts

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    experts._torch()


@pytest.mark.parametrize("temp,error", [
    (torch.empty(4096, dtype=torch.uint8), ValueError), (torch.empty(1024, device="meta"), TypeError),
    (torch.empty(1, dtype=torch.uint8, device="meta").expand(4096), ValueError),
    (torch.empty(8192, dtype=torch.uint8, device="meta")[::2], ValueError), (1 << 40, TypeError)])
def test_scratch_is_checked_as_other_tensors_are(temp, error):
    x = torch.empty(4, 4, device="meta")
    with pytest.raises(error):
        experts._scratch(temp, x)
    experts._scratch(torch.empty(4096, dtype=torch.uint8, device="meta"), x)
