"""The expert operators' argument checks, which need no GPU: nothing is
enqueued before they pass."""
import ctypes
import os
import re

import pytest

import lsd_radix_sort_key_gb300 as rs
from lsd_radix_sort_key_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = 1 << 40  # 256-byte aligned addresses that are never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return rs.lib()


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "rs_experts.h")).read()
    assert int(re.search(r"#define RS_EXPERTS_MAX (\d+)", text).group(1)) == rs.EXPERTS_MAX
    for name, value in rs.ACTIVATIONS.items():
        assert int(re.search(rf"RS_ACT_{name.upper()} = (\d)", text).group(1)) == value
    for name, value in (("RS_FLOAT32", "float32"), ("RS_FLOAT16", "float16"), ("RS_BFLOAT16", "bfloat16")):
        assert int(re.search(rf"{name} = (\d)", text).group(1)) == rs.FLOAT_TYPES[value]


def test_desc_matches_the_header():
    text = open(os.path.join(ROOT, "include", "rs_experts.h")).read()
    body = re.search(r"typedef struct rs_expert_matmul_desc \{(.*?)\}", text, re.S).group(1)
    names = re.findall(r"(\w+);", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
    assert names == [n for n, _ in rs.ExpertMatmulDesc._fields_]


def test_the_packed_descriptor_is_the_structure():
    from lsd_radix_sort_key_gb300 import experts
    assert experts._DESC.size == ctypes.sizeof(rs.ExpertMatmulDesc)
    values = [3 + i for i in range(len(rs.ExpertMatmulDesc._fields_))]
    assert experts._DESC.pack(*values) == bytes(rs.ExpertMatmulDesc(*values))


@pytest.mark.parametrize("kw,code", [
    (dict(ids=None), 1), (dict(order=None), 1), (dict(position=None), 1), (dict(offsets=None), 1),
    (dict(temp=None), 1), (dict(id_bytes=2), 1), (dict(ids=F + 4), 1), (dict(order=2 * F + 2), 1),
    (dict(temp=5 * F + 16), 1), (dict(experts=0), 1), (dict(experts=1025), 1), (dict(n=(1 << 30) + 1), 1),
    (dict(temp_bytes=0), 2), (dict(position=2 * F), 3), (dict(order=F + 8), 3), (dict(offsets=5 * F), 3),
])
def test_sort_refuses(kw, code):
    a = dict(ids=F, id_bytes=8, n=100_000, experts=16, order=2 * F, position=3 * F, offsets=4 * F, temp=5 * F,
             temp_bytes=1 << 20)
    a.update(kw)
    assert rs.rs_expert_sort(a["ids"], a["id_bytes"], a["n"], a["experts"], a["order"], a["position"], a["offsets"],
                             a["temp"], a["temp_bytes"], 0) == code


def test_sort_temp_bytes():
    bad = ctypes.c_size_t(-1).value
    assert rs.rs_expert_sort_temp_bytes(0, 4) == 0
    assert rs.rs_expert_sort_temp_bytes(512, 128) == 0
    assert 0 < rs.rs_expert_sort_temp_bytes(100_000, 4) < 1 << 20
    assert rs.rs_expert_sort_temp_bytes(1 << 30, 1024) < 1 << 31
    assert rs.rs_expert_sort_temp_bytes((1 << 30) + 1, 4) == bad
    assert rs.rs_expert_sort_temp_bytes(1, 0) == bad and rs.rs_expert_sort_temp_bytes(1, 1025) == bad


ROWS = dict(x=F, xs=64, position=2 * F, routed=3 * F, tokens=10, slots=4, width=64, out=4 * F, os=64)
BAD_ROWS = [(dict(x=None), 1), (dict(out=None), 1), (dict(position=None), 1), (dict(routed=None), 1),
            (dict(x=F + 1), 1), (dict(out=4 * F + 1), 1), (dict(position=2 * F + 1), 1), (dict(slots=0), 1),
            (dict(xs=63), 1), (dict(os=63), 1), (dict(os=0), 1), (dict(width=(1 << 20) + 1), 1),
            (dict(tokens=1 << 29), 1), (dict(tokens=1 << 62), 1), (dict(out=F), 3), (dict(out=2 * F), 3),
            (dict(routed=4 * F), 3), (dict(tokens=0), 0), (dict(width=0), 0)]


@pytest.mark.parametrize("kw,code", BAD_ROWS)
def test_row_movers_refuse(kw, code):
    a = dict(ROWS, **kw)
    assert rs.rs_expert_dispatch("bfloat16", a["x"], a["xs"], a["position"], a["routed"], a["tokens"], a["slots"],
                                 a["width"], a["out"], a["os"], 0) == code
    assert rs.rs_expert_combine("float16", a["x"], a["xs"], None, "float32", a["position"], a["routed"], a["tokens"],
                                a["slots"], a["width"], a["out"], a["os"], 0) == code


def grad(**kw):
    a = dict(t="bfloat16", dout=F, ds=64, y=2 * F, ys=64, weights=3 * F, wt="float32", position=4 * F, routed=5 * F,
             tokens=10, slots=4, width=64, dy=6 * F, dys=64, dweights=7 * F)
    a.update(kw)
    return rs.rs_expert_combine_grad(a["t"], a["dout"], a["ds"], a["y"], a["ys"], a["weights"], a["wt"],
                                     a["position"], a["routed"], a["tokens"], a["slots"], a["width"], a["dy"],
                                     a["dys"], a["dweights"], 0)


@pytest.mark.parametrize("kw,code", [
    (dict(dout=None), 1), (dict(y=None), 1), (dict(weights=None), 1), (dict(dy=None), 1), (dict(dweights=None), 1),
    (dict(wt="float16"), 1), (dict(weights=3 * F + 2), 1), (dict(ys=10), 1), (dict(dys=0), 1), (dict(dy=2 * F), 3),
    (dict(dweights=3 * F), 3), (dict(dy=7 * F), 3), (dict(tokens=0), 0),
])
def test_combine_grad_refuses(kw, code):
    assert grad(**kw) == code


def test_combine_refuses_weights_of_a_third_type():
    assert rs.rs_expert_combine("float16", F, 64, 2 * F, "bfloat16", 3 * F, 4 * F, 10, 4, 64, 5 * F, 64, 0) == 1
    assert rs.rs_expert_combine("float16", F, 64, 2 * F + 1, "float16", 3 * F, 4 * F, 10, 4, 64, 5 * F, 64, 0) == 1


def desc(**kw):
    d = rs.ExpertMatmulDesc(2, 3, 4, 100, 64, 128, F, 2 * F, 64, 3 * F, 64 * 128, 64, 1, 4 * F, 128, 5 * F, 128,
                            6 * F, 128, 7 * F, 128, 8 * F, 64, 9 * F, 10 * F, 11 * F, 1 << 30, None)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


MATMUL = [(dict(type=3), 1), (dict(type=-1), 1), (dict(activation=4), 1), (dict(num_experts=0), 1),
          (dict(num_experts=1025), 1), (dict(rows=(1 << 30) + 1), 1), (dict(inner=(1 << 20) + 1), 1),
          (dict(outer=(1 << 20) + 1), 1), (dict(stall_tile=-1), 1), (dict(temp=None), 1),
          (dict(temp=11 * F + 128), 1), (dict(temp_bytes=100), 2), (dict(offsets=None), 1), (dict(offsets=F + 2), 1), (dict(y=None), 1)]


@pytest.mark.parametrize("kw,code", MATMUL + [
    (dict(x=None), 1), (dict(w=None), 1), (dict(x_stride=63), 1), (dict(y_stride=0), 1), (dict(y_stride=127), 1),
    (dict(pre_stride=127), 1), (dict(bias_stride=5), 1), (dict(residual_stride=5), 1), (dict(w=3 * F + 1), 1),
    (dict(bias=4 * F + 1), 1), (dict(w_inner_stride=2, w_outer_stride=128), 1), (dict(w_expert_stride=1 << 41), 1),
    (dict(y=2 * F), 3), (dict(y=3 * F + 256), 3), (dict(y=4 * F), 3), (dict(y=5 * F), 3), (dict(pre=6 * F), 3),
    (dict(pre=F), 3), (dict(rows=0), 0), (dict(outer=0), 0)])
def test_matmul_refuses(kw, code):
    assert rs.rs_expert_matmul(desc(**kw)) == code


@pytest.mark.parametrize("kw,code", MATMUL + [
    (dict(pre=None), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(dx_stride=63), 1), (dict(dw=9 * F + 1), 1),
    (dict(dbias=10 * F + 1), 1),
    (dict(dx=2 * F), 3), (dict(dx=3 * F), 3), (dict(dw=6 * F), 3), (dict(dbias=7 * F), 3), (dict(dx=11 * F), 3),
    (dict(dx=9 * F), 3), (dict(dx=None, dw=None, dbias=None), 0)])
def test_matmul_grad_refuses(kw, code):
    assert rs.rs_expert_matmul_grad(desc(**kw)) == code


def test_matmul_temp_bytes():
    bad = ctypes.c_size_t(-1).value
    assert rs.rs_expert_matmul_temp_bytes(desc(type=7)) == bad
    assert rs.rs_expert_matmul_grad_temp_bytes(desc(num_experts=0)) == bad
    both = rs.rs_expert_matmul_grad_temp_bytes(desc())
    assert both >= 100 * 128 * 2  # dz
    assert rs.rs_expert_matmul_grad_temp_bytes(desc(activation=0)) < both
    assert rs.rs_expert_matmul_grad_temp_bytes(desc(activation=0, dbias=None)) == rs.rs_expert_matmul_temp_bytes(desc())
    assert rs.rs_expert_matmul_status(None, 0) == 1
    # rows that are not 16-byte aligned are copied into temp
    plain = rs.rs_expert_matmul_temp_bytes(desc())
    assert rs.rs_expert_matmul_temp_bytes(desc(x=2 * F + 2)) >= plain + 100 * 64 * 2
    assert rs.rs_expert_matmul_temp_bytes(desc(w=3 * F + 2)) >= plain + 4 * 128 * 64 * 2
    assert rs.rs_expert_matmul_temp_bytes(desc(x_stride=0)) >= plain + 100 * 64 * 2
    assert rs.rs_expert_matmul_temp_bytes(desc(type=0, x=2 * F + 4)) == plain
    assert rs.rs_expert_matmul_grad_temp_bytes(desc(x=2 * F + 2)) >= both + 100 * 64 * 2


def test_the_binding_checks_its_tensors():
    torch = pytest.importorskip("torch")
    ids = torch.zeros(4, 2, dtype=torch.int64)
    with pytest.raises(ValueError):
        rs.expert_sort(ids, 4)  # not on a GPU
    with pytest.raises(TypeError):
        rs.expert_sort(ids.float(), 4)
    position, offsets = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        rs.expert_dispatch(x, position, offsets)
    with pytest.raises(TypeError):
        rs.expert_dispatch(x.double(), position, offsets)
    with pytest.raises(TypeError):
        rs.expert_combine(x, None, position, offsets)
    with pytest.raises(ValueError):
        rs.expert_matmul(x, torch.zeros(2, 8, 8), offsets)
    with pytest.raises(ValueError):
        rs.expert_matmul(x, torch.zeros(2, 8, 8), offsets, activation="tanh")
