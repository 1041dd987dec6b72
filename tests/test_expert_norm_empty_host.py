"""Norms of rows without columns, and of no rows: sizes that need no GPU."""
import ctypes

import pytest

import lsd_radix_sort_key_gb300 as rs
from lsd_radix_sort_key_gb300 import _build

F = 1 << 40  # an address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return rs.lib()


@pytest.mark.parametrize("block", [None, F])
@pytest.mark.parametrize("rows", [0, 12])
@pytest.mark.parametrize("type", [0, 1, 2])
def test_no_columns_need_no_memory(type, rows, block):
    d = rs.ExpertNormDesc(type, 0, rows, 0, 1e-6, 0.7, 4 if block else 0, F, 1, block, 1, F, block, block)
    assert rs.rs_expert_norm_grad_temp_bytes(d) == 0
    d.dx, d.dweight, d.dh = F, F, F
    assert rs.rs_expert_norm(d) == 0 and rs.rs_expert_norm_grad(d) == 0


def test_a_refused_size_is_still_refused():
    d = rs.ExpertNormDesc(2, 0, 12, 0, -1.0, 0.7, 0, F, 1)
    assert rs.rs_expert_norm_grad_temp_bytes(d) == ctypes.c_size_t(-1).value
