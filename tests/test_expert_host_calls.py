"""What the Python forms of the expert operators check themselves, as far as it
needs no GPU."""
import os
import re
import shutil
import subprocess
import sysconfig

import pytest

import lsd_radix_sort_key_gb300 as rs
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


F = 1 << 40  # 256-byte aligned addresses that are never dereferenced


def desc(**kw):
    d = rs.ExpertMatmulDesc(2, 3, 4, 100, 64, 128, F, 2 * F, 64, 3 * F, 64 * 128, 64, 1, 4 * F, 128, 5 * F, 128,
                            6 * F, 128, 7 * F, 128, 8 * F, 64, 9 * F, 10 * F, 11 * F, 1 << 62, None)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw", [dict(type=t, **{name: (1 << 40) // size}) for t, size in ((0, 4), (1, 2), (2, 2))
                                for name in ("w_expert_stride", "w_outer_stride")] +
                         [dict(w_outer_stride=1, w_inner_stride=1 << 39), dict(w_outer_stride=1 << 63)])
def test_weight_strides_past_a_tensor_map_are_refused_first(kw):
    assert rs.rs_expert_matmul(desc(**kw)) == 1
    assert rs.rs_expert_matmul_grad(desc(**kw)) == 1


def test_overlap_is_seen_however_long_a_matrix_is():
    # x spans all but 2^34 of the 2^64 bytes: its end lies past the last address
    long = dict(type=0, rows=1 << 30, x_stride=1 << 32)
    for name, at in (("y", 6), ("pre", 7), ("temp", 11)):
        assert rs.rs_expert_matmul(desc(**long, **{name: at * F})) == 3
    assert rs.rs_expert_matmul_grad(desc(**long)) == 3


def test_more_slots_than_an_int_holds_are_refused():
    # 2^32 + 1 would count as 1
    offsets = torch.empty(3, dtype=torch.int32, device="meta")
    with pytest.raises(rs.RadixSortError):
        experts._plan(torch.empty(1, (1 << 32) + 1, dtype=torch.int32, device="meta"), offsets, offsets.device)
    assert experts._plan(torch.empty(2, 5, dtype=torch.int32, device="meta"), offsets, offsets.device)[:2] == (2, 5)
    text = open(os.path.join(_build.INCLUDE, "rs_experts.h")).read()
    assert int(re.search(r"#define RS_EXPERT_SLOTS_MAX (\d+)u", text).group(1)) == experts.SLOTS_MAX


@pytest.mark.skipif(not _build.torch_dir(), reason="torch without CUDA has no extension")
@pytest.mark.parametrize("fails", ["headers", "no compiler"])
def test_the_library_is_built_where_the_extension_is_not(tmp_path, monkeypatch, fails):
    monkeypatch.setattr(_build, "LIBDIR", str(tmp_path))
    assert sysconfig.get_config_var("SOABI") in _build.torch_ext()
    run = subprocess.run

    def broken(cmd, **kw):
        if cmd[0] != "g++":
            return run(cmd, **kw)
        if fails == "no compiler":
            raise FileNotFoundError("g++")
        return subprocess.CompletedProcess(cmd, 1, "", "no such header")

    with open(_build.torch_ext(), "w") as f:
        f.write("of older sources")
    monkeypatch.setattr(_build.subprocess, "run", broken)
    monkeypatch.setattr(_build, "_stale", lambda: False)  # librs.so as it is
    with pytest.warns(RuntimeWarning, match="go through Python"):
        os.utime(_build.torch_ext(), (0, 0))
        assert _build.build() == _build.LIB
    assert not os.path.exists(_build.torch_ext())  # not the older one either
