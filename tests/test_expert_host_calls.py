"""What the Python forms of the expert operators check themselves, as far as it
needs no GPU."""
import re
import shutil
import subprocess

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


@pytest.mark.skipif(shutil.which("nm") is None, reason="reads the library's symbols")
def test_each_split_kernel_has_a_count_of_its_own():
    # how many clusters of a kernel are resident is kept per kernel, not per its type
    names = subprocess.run(["nm", "-C", _build.LIB], capture_output=True, text=True, check=True).stdout
    kernels = set(re.findall(r"rsx::k_product_split<(__\w+, \w+, \w+)>\(CUtensorMap_st, CUtensorMap_st", names))
    counts = set(re.findall(r"resident_clusters<.*k_product_split<(__\w+, \w+, \w+)>.*::known$", names, re.M))
    assert len(kernels) == 6 and counts == kernels
