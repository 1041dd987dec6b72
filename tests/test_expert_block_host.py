"""Argument checks of the quantisers, their products and the norms, which need
no GPU: nothing is enqueued before they pass."""
import ctypes
import os
import re

import pytest

import lsd_radix_sort_key_gb300 as rs
from lsd_radix_sort_key_gb300 import _build, expert_block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = 1 << 40  # 256-byte aligned addresses that are never dereferenced
BAD = ctypes.c_size_t(-1).value
HEADER = open(os.path.join(ROOT, "include", "rs_expert_block.h")).read()


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return rs.lib()


def test_constants_match_the_header():
    assert int(re.search(r"#define RS_QUANT_BLOCK (\d+)", HEADER).group(1)) == rs.QUANT_BLOCK
    assert int(re.search(r"#define RS_EXPERT_NORM_WIDTH_MAX (\d+)", HEADER).group(1)) == rs.NORM_WIDTH_MAX


@pytest.mark.parametrize("name,cls,packed", [
    ("rs_expert_matmul_quantized_desc", rs.ExpertMatmulQuantizedDesc, expert_block._MATMUL),
    ("rs_expert_norm_desc", rs.ExpertNormDesc, expert_block._NORM)])
def test_descriptors_match_the_header(name, cls, packed):
    body = re.search(r"typedef struct %s \{(.*?)\}" % name, HEADER, re.S).group(1)
    names = re.findall(r"(\w+);", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
    assert names == [n for n, _ in cls._fields_]
    assert packed.size == ctypes.sizeof(cls)
    values = [3 + i for i in range(len(cls._fields_))]
    assert packed.pack(*values) == bytes(cls(*values))


def test_every_entry_has_a_signature():
    for name in re.findall(r"\b(rs_expert_\w+)\(", HEADER):
        assert name in rs.SIGNATURES and hasattr(rs, name)


ROWS = dict(t="bfloat16", x=F, xs=300, rows=10, width=300, q=2 * F, qs=304, s=3 * F, ss=3)
BAD_ROWS = [(dict(x=None), 1), (dict(x=F + 1), 1), (dict(xs=299), 1), (dict(q=None), 1), (dict(q=2 * F + 8), 1), (dict(qs=300), 1),
            (dict(qs=288), 1), (dict(s=None), 1), (dict(ss=2), 1), (dict(width=(1 << 20) + 1), 1), (dict(rows=(1 << 30) + 1), 1),
            (dict(rows=1 << 30, width=1 << 20, xs=1 << 20, qs=1 << 20, ss=1 << 13), 1), (dict(q=F), 3), (dict(s=F + 100), 3),
            (dict(s=2 * F), 3), (dict(s=2 * F + 9 * 304 + 303), 3), (dict(rows=0), 0), (dict(width=0), 0)]


@pytest.mark.parametrize("kw,code", BAD_ROWS)
def test_quantize_refuses(kw, code):
    a = dict(ROWS, **kw)
    assert rs.rs_expert_quantize(a["t"], a["x"], a["xs"], a["rows"], a["width"], a["q"], a["qs"], a["s"], a["ss"], 0) == code


@pytest.mark.parametrize("kw,code", [b for b in BAD_ROWS if "rows" not in b[0]] + [
    (dict(position=None), 1), (dict(position=4 * F + 2), 1), (dict(routed=None), 1), (dict(slots=0), 1), (dict(tokens=1 << 29), 1),
    (dict(tokens=1 << 62), 1), (dict(position=2 * F), 3), (dict(routed=3 * F), 3), (dict(tokens=0), 0)])
def test_dispatch_refuses(kw, code):
    a = dict(ROWS, position=4 * F, routed=5 * F, tokens=10, slots=4)
    a.update(kw)
    assert rs.rs_expert_dispatch_quantized(a["t"], a["x"], a["xs"], a["position"], a["routed"], a["tokens"], a["slots"], a["width"],
                                           a["q"], a["qs"], a["s"], a["ss"], 0) == code


@pytest.mark.parametrize("kw,code", [
    (dict(w=None), 1), (dict(w=F + 1), 1), (dict(sk=2), 1), (dict(sn=1 << 40), 1), (dict(se=1 << 40), 1), (dict(e=0), 1), (dict(e=1025), 1),
    (dict(n=(1 << 20) + 1), 1), (dict(k=(1 << 20) + 1), 1), (dict(q=2 * F + 4), 1), (dict(qs=264), 1), (dict(qs=240), 1),
    (dict(s=None), 1), (dict(q=F + 64), 3), (dict(s=F + 64), 3), (dict(s=2 * F), 3), (dict(n=0), 0), (dict(k=0), 0)])
def test_quantize_weights_refuses(kw, code):
    a = dict(w=F, se=140 * 256, sn=256, sk=1, e=4, n=140, k=256, q=2 * F, qs=256, s=3 * F)
    a.update(kw)
    assert rs.rs_expert_quantize_weights("float16", a["w"], a["se"], a["sn"], a["sk"], a["e"], a["n"], a["k"], a["q"], a["qs"], a["s"],
                                         0) == code


def matmul(**kw):
    d = rs.ExpertMatmulQuantizedDesc(2, 3, 4, 100, 300, 130, F, 2 * F, 304, 3 * F, 3, 4 * F, 304, 5 * F, 6 * F, 130, 7 * F, 130, 8 * F,
                                     130, None, 0, None, 0, 11 * F, 130, 12 * F, 1 << 20, None, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


QUANTIZED = dict(y=None, residual=None, q=9 * F, q_stride=144, q_scales=10 * F, q_scales_stride=2)


@pytest.mark.parametrize("kw,code", [
    (dict(type=0), 1), (dict(type=3), 1), (dict(activation=4), 1), (dict(num_experts=0), 1), (dict(num_experts=1025), 1),
    (dict(rows=(1 << 30) + 1), 1), (dict(inner=0), 1), (dict(inner=(1 << 20) + 1), 1), (dict(outer=(1 << 20) + 1), 1),
    (dict(stall_tile=-1), 1), (dict(offsets=None), 1), (dict(offsets=F + 2), 1), (dict(x=None), 1), (dict(x=2 * F + 8), 1),
    (dict(x_stride=300), 1), (dict(x_stride=288), 1), (dict(x_stride=0), 1), (dict(x_scales=None), 1), (dict(x_scales_stride=2), 1),
    (dict(w=None), 1), (dict(w=4 * F + 1), 1), (dict(w_stride=296), 1), (dict(w_scales=None), 1), (dict(bias=6 * F + 1), 1),
    (dict(bias_stride=5), 1), (dict(residual_stride=5), 1), (dict(y=None), 1), (dict(y=8 * F + 1), 1), (dict(y_stride=0), 1),
    (dict(pre_stride=100), 1), (dict(q=9 * F, q_stride=144, q_scales=10 * F, q_scales_stride=2), 1),
    (dict(QUANTIZED, residual=7 * F), 1), (dict(QUANTIZED, q=9 * F + 8), 1), (dict(QUANTIZED, q_stride=136), 1),
    (dict(QUANTIZED, q_scales=None), 1), (dict(QUANTIZED, q_scales_stride=1), 1), (dict(QUANTIZED, q_scales=9 * F + 100), 3),
    (dict(QUANTIZED, q=2 * F), 3), (dict(temp=None), 1), (dict(temp=12 * F + 16), 1), (dict(temp_bytes=100), 2), (dict(y=2 * F), 3),
    (dict(y=3 * F), 3), (dict(y=4 * F + 304), 3), (dict(pre=5 * F), 3), (dict(pre=6 * F), 3), (dict(y=7 * F), 3), (dict(pre=8 * F), 3),
    (dict(pre=F), 3), (dict(temp=2 * F), 3), (dict(rows=0), 0), (dict(outer=0), 0)])
def test_matmul_refuses(kw, code):
    assert rs.rs_expert_matmul_quantized(matmul(**kw)) == code


def test_matmul_temp_bytes():
    assert rs.rs_expert_matmul_quantized_temp_bytes(matmul(type=0)) == BAD
    assert rs.rs_expert_matmul_quantized_temp_bytes(matmul(inner=0)) == BAD
    assert 0 < rs.rs_expert_matmul_quantized_temp_bytes(matmul()) <= 1 << 12


def norm(grad=False, **kw):
    d = rs.ExpertNormDesc(2, 0, 12, 264, 1e-6, 0.7, 4, F, 264, 2 * F, 264, 3 * F, 4 * F, 5 * F)
    if grad:
        more = dict(dh=8 * F, dh_stride=264, dy=9 * F, dy_stride=264, dx=10 * F, dx_stride=264, dblock=11 * F, dblock_stride=264,
                    dweight=12 * F, dblock_weight=13 * F, dgate=14 * F, temp=15 * F, temp_bytes=1 << 30)
    else:
        more = dict(y=6 * F, y_stride=264, h=7 * F, h_stride=264)
    for k, v in {**more, **kw}.items():
        setattr(d, k, v)
    return d


NORM = [(dict(type=3), 1), (dict(param_type=1), 1), (dict(width=16385), 1), (dict(rows=(1 << 30) + 4), 1), (dict(eps=-1.0), 1),
        (dict(eps=float("inf")), 1), (dict(eps=float("nan")), 1), (dict(residual_scale=float("inf")), 1),
        (dict(residual_scale=float("nan")), 1), (dict(gate_rows=5), 1), (dict(gate_rows=24), 1), (dict(gate=None), 1),
        (dict(x=None), 1), (dict(x=F + 1), 1), (dict(x_stride=263), 1), (dict(block=2 * F + 1), 1), (dict(block_stride=10), 1),
        (dict(weight=3 * F + 2), 1), (dict(block_weight=4 * F + 2), 1), (dict(gate=5 * F + 2), 1), (dict(block=None), 1),
        (dict(width=0), 0)]


@pytest.mark.parametrize("kw,code", NORM + [
    (dict(y=None), 1), (dict(y=6 * F + 1), 1), (dict(y_stride=0), 1), (dict(h=None), 1), (dict(h_stride=100), 1),
    (dict(block=None, block_weight=None, gate_rows=0, weight=None), 1), (dict(y=F), 3), (dict(h=2 * F), 3), (dict(h=6 * F + 264), 3),
    (dict(y=3 * F), 3), (dict(h=4 * F), 3), (dict(h=5 * F + 3 * 264 * 4), 3), (dict(rows=0), 0)])
def test_norm_refuses(kw, code):
    assert rs.rs_expert_norm(norm(**kw)) == code


@pytest.mark.parametrize("kw,code", NORM + [
    (dict(dh=None), 1), (dict(weight=None), 1), (dict(dh=8 * F + 1), 1), (dict(dh_stride=5), 1), (dict(dy_stride=5), 1),
    (dict(dx_stride=0), 1), (dict(dblock_stride=7), 1), (dict(dweight=12 * F + 1), 1), (dict(dgate=14 * F + 2), 1),
    (dict(dh=None, weight=None), 1), (dict(dh=None, weight=None, dy=None, dweight=None), 1),
    (dict(block_weight=None), 1), (dict(gate_rows=0), 1), (dict(temp=None), 1), (dict(temp=15 * F + 1), 1), (dict(temp_bytes=100), 2),
    (dict(dx=F), 3), (dict(dx=8 * F), 3), (dict(dblock=9 * F), 3), (dict(dblock=10 * F), 3), (dict(dweight=3 * F), 3),
    (dict(dblock_weight=12 * F + 4), 3), (dict(dgate=15 * F), 3), (dict(dgate=5 * F), 3),
    (dict(dx=None, dblock=None, dweight=None, dblock_weight=None, dgate=None), 0)])
def test_norm_grad_refuses(kw, code):
    assert rs.rs_expert_norm_grad(norm(True, **kw)) == code


def test_norm_grad_temp_bytes():
    assert rs.rs_expert_norm_grad_temp_bytes(norm(True, width=16385)) == BAD
    assert 0 < rs.rs_expert_norm_grad_temp_bytes(norm(True)) <= 4 * 12 * 264 * 4 + 256


def test_the_binding_checks_its_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 256)
    q, s = x.to(torch.float8_e4m3fn), torch.zeros(4, 2, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    position, offsets = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        rs.expert_quantize(x)  # not on a GPU
    with pytest.raises(TypeError):
        rs.expert_quantize(x.double())
    with pytest.raises(TypeError):
        rs.expert_quantize(q)
    with pytest.raises(ValueError):
        rs.expert_dispatch_quantized(x, position, offsets)
    with pytest.raises(ValueError):
        rs.expert_quantize_weights(x[None])
    with pytest.raises(ValueError):
        rs.expert_matmul_quantized(q, s, q[None], s[None], offsets)
    with pytest.raises(TypeError):
        rs.expert_matmul_quantized(x, s, q[None], s[None], offsets)
    with pytest.raises(ValueError):
        rs.expert_matmul_quantized(q, s, q[None], s[None], offsets, activation="tanh")
    with pytest.raises(TypeError):
        rs.expert_matmul_quantized(q, s, q[None], s[None], offsets, dtype=torch.float32)
    w = torch.ones(256)
    with pytest.raises(ValueError):
        rs.expert_norm(x, w)
    with pytest.raises(TypeError):
        rs.expert_norm(x, None)
    with pytest.raises(TypeError):
        rs.expert_norm(x.double(), w)
    with pytest.raises(TypeError):
        rs.expert_norm_grad(None, x, w)
    with pytest.raises(TypeError):
        rs.expert_norm_grad(None, x, None)
