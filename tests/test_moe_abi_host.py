"""Host-side checks of the second part of the C ABI (include/fp8bw_moe.h): its
calls are exported and bound, and bad arguments come back as the documented
codes before any GPU is touched (no GPU needed)."""
import os
import re

import pytest
import torch

from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import build, moe
from mxfp8_precision_gemms_fp8bw_gb300 import moe_binding as MB

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp8bw_moe.h")
P = 1 << 20  # a fake, 16-byte aligned "device" address; never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return MB.lib()


def test_header_binding_and_library_agree(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*\w+\s+(\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(MB._SIGNATURES)
    assert all(hasattr(L, n) for n in names)


def route(L, logits=P, kind=0, bias=None, M=4, E=8, k=2, groups=1, kept=1, top=1, score=0, experts=2 * P, weights=3 * P):
    return L.fp8bw_moe_route(logits, kind, bias, M, E, k, groups, kept, top, score, 1, 1.0, experts, weights, None)


@pytest.mark.parametrize("code,kw", [
    ("NULL", dict(logits=None)), ("NULL", dict(experts=None)), ("NULL", dict(weights=None)),
    ("SHAPE", dict(M=0)), ("SHAPE", dict(E=0)), ("SHAPE", dict(E=1025)), ("SHAPE", dict(k=0)), ("SHAPE", dict(k=9)),
    ("SHAPE", dict(E=64, k=33)), ("SHAPE", dict(groups=3)), ("SHAPE", dict(groups=0)), ("SHAPE", dict(groups=64, E=64)),
    ("SHAPE", dict(groups=2, kept=3)), ("SHAPE", dict(groups=4, kept=1, k=3)), ("SHAPE", dict(groups=2, kept=0)),
    ("ALIGN", dict(logits=P + 4)), ("ALIGN", dict(bias=5 * P + 4)), ("ALIGN", dict(weights=3 * P + 8)),
    ("ARG", dict(kind=2)), ("ARG", dict(score=2)), ("ARG", dict(top=3)),
    ("LAYOUT", dict(experts=P + 64)), ("LAYOUT", dict(weights=2 * P + 16)),
])
def test_route_refusals(L, code, kw):
    assert route(L, **kw) == getattr(B, "ERR_" + code)
    assert B.last_error()


def test_route_bwd_refusals(L):
    f = lambda *a: L.fp8bw_moe_route_bwd(*a, None)  # noqa: E731
    ok = (P, 2 * P, 0, 3 * P, 4, 8, 2, 0, 1, 1.0, 4 * P)
    for i in (0, 1, 3, 10):
        assert f(*ok[:i], None, *ok[i + 1:]) == B.ERR_NULL
    assert f(*ok[:4], 0, *ok[5:]) == B.ERR_SHAPE
    assert f(*ok[:10], 4 * P + 2) == B.ERR_ALIGN
    assert f(*ok[:7], 7, *ok[8:]) == B.ERR_ARG
    assert f(*ok[:10], 2 * P + 64) == B.ERR_LAYOUT


def test_plan_rows_and_workspace(L):
    rows = MB.fp8bw_moe_plan_rows
    assert rows(1, 1, 1) == 32 and rows(17, 64, 4) == 2048 and rows(8192, 8, 2) == 16608
    assert rows(1, 64, 4) == 128          # 4 entries over at most 4 experts: a block each
    assert rows(0, 8, 2) == rows(8, 0, 2) == rows(8, 8, 9) == rows(1 << 30, 8, 4) == 0
    assert MB.fp8bw_moe_plan_workspace_bytes(16, 8, 2) == 0       # few entries need none
    assert MB.fp8bw_moe_plan_workspace_bytes(16384, 8, 2) > 0
    assert MB.fp8bw_moe_plan_workspace_bytes(16, 2000, 2) == 0


def test_plan_refusals(L):
    rows, n = MB.fp8bw_moe_plan_rows(16384, 8, 2), MB.fp8bw_moe_plan_workspace_bytes(16384, 8, 2)
    ok = [P, 16384, 8, 2, rows, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, n, None]
    f = lambda **kw: L.fp8bw_moe_plan(*[kw.get("a%d" % i, v) for i, v in enumerate(ok)])  # noqa: E731
    for i in (0, 5, 6, 7, 8, 9):
        assert f(**{"a%d" % i: None}) == B.ERR_NULL
        assert f(**{"a%d" % i: ok[i] + 8}) == B.ERR_ALIGN
    assert f(a4=rows - 32) == B.ERR_SHAPE and "plan_rows" in B.last_error()
    assert f(a4=rows + 1) == B.ERR_SHAPE
    assert f(a1=0) == B.ERR_SHAPE and f(a2=1) == B.ERR_SHAPE and f(a3=33) == B.ERR_SHAPE
    assert f(a10=n - 1) == B.ERR_ARG
    assert f(a5=P) == B.ERR_LAYOUT and f(a8=4 * P + 64) == B.ERR_LAYOUT


def test_gather_quant_refusals(L):
    ok = [P, None, 2 * P, 16, 2, 64, 96, 3 * P, 4 * P, 5 * P, 6 * P, 0, None]
    f = lambda **kw: L.mxfp8_moe_gather_quant(*[kw.get("a%d" % i, v) for i, v in enumerate(ok)])  # noqa: E731
    for i in (0, 2, 7, 8, 9, 10):   # qT without e8T and the other way round too
        assert f(**{"a%d" % i: None}) == B.ERR_NULL
        assert f(**{"a%d" % i: ok[i] + 8}) == B.ERR_ALIGN
    for kw in (dict(a3=0), dict(a4=0), dict(a4=33), dict(a5=48), dict(a6=80), dict(a6=0)):
        assert f(**kw) == B.ERR_SHAPE
    assert f(a11=2) == B.ERR_ARG
    assert f(a7=P + 1024) == B.ERR_LAYOUT and f(a9=3 * P + 16) == B.ERR_LAYOUT


def test_combine_refusals(L):
    ok = [P, None, 2 * P, None, 16, 2, 64, 96, 3 * P, None]
    f = lambda **kw: L.fp8bw_moe_combine(*[kw.get("a%d" % i, v) for i, v in enumerate(ok)])  # noqa: E731
    for i in (0, 2, 8):
        assert f(**{"a%d" % i: None}) == B.ERR_NULL
        assert f(**{"a%d" % i: ok[i] + 8}) == B.ERR_ALIGN
    for kw in (dict(a4=0), dict(a5=0), dict(a6=31), dict(a7=4)):
        assert f(**kw) == B.ERR_SHAPE
    assert f(a8=P) == B.ERR_LAYOUT
    assert f(a3=3 * P + 16) == B.ERR_LAYOUT      # base may be out itself, not shifted against it
    ok = [P, 2 * P, 3 * P, 16, 2, 64, 96, 4 * P, None]
    f = lambda **kw: L.fp8bw_moe_combine_dweights(*[kw.get("a%d" % i, v) for i, v in enumerate(ok)])  # noqa: E731
    for i in (0, 1, 2, 7):
        assert f(**{"a%d" % i: None}) == B.ERR_NULL
        assert f(**{"a%d" % i: ok[i] + 4}) == B.ERR_ALIGN
    assert f(a3=0) == B.ERR_SHAPE and f(a7=P + 16) == B.ERR_LAYOUT


def test_swiglu_refusals(L):
    ok = [P, 64, 96, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, 0, None]
    f = lambda **kw: L.mxfp8_swiglu(*[kw.get("a%d" % i, v) for i, v in enumerate(ok)])  # noqa: E731
    for i in (0, 3, 4, 5, 6, 7, 8):
        assert f(**{"a%d" % i: None}) == B.ERR_NULL
        assert f(**{"a%d" % i: ok[i] + 8}) == B.ERR_ALIGN
    for kw in (dict(a1=0), dict(a1=48), dict(a2=0), dict(a2=40)):
        assert f(**kw) == B.ERR_SHAPE
    assert f(a9=-1) == B.ERR_ARG and f(a3=P) == B.ERR_LAYOUT and f(a7=2 * P + 16) == B.ERR_LAYOUT
    ok = [P, 2 * P, 3 * P, 64, 96, 4 * P, 5 * P, 6 * P, 7 * P, 0, None]
    f = lambda **kw: L.mxfp8_swiglu_bwd(*[kw.get("a%d" % i, v) for i, v in enumerate(ok)])  # noqa: E731
    for i in (0, 1, 2, 5, 6, 7, 8):
        assert f(**{"a%d" % i: None}) == B.ERR_NULL
        assert f(**{"a%d" % i: ok[i] + 8}) == B.ERR_ALIGN
    assert f(a3=16) == B.ERR_SHAPE and f(a9=2) == B.ERR_ARG and f(a5=2 * P) == B.ERR_LAYOUT


def test_binding_refuses_wrong_types_shapes_and_devices():
    z = torch.zeros
    with pytest.raises(TypeError):
        MB.fp8bw_moe_route(z(4, 8, dtype=torch.float16), None, 2, z(4, 2, dtype=torch.int32), z(4, 2))
    with pytest.raises(ValueError):       # CPU tensors
        moe.route(z(4, 8), 2)
    with pytest.raises(ValueError):
        moe.route(z(4, 8), 2, score="relu")
    with pytest.raises(ValueError):       # an odd width is no [gate | up]
        moe.swiglu(z(32, 65, dtype=torch.bfloat16))
    with pytest.raises(B.Fp8bwError) as e:
        moe.plan(z(5, 2, dtype=torch.int32), 0)
    assert e.value.code == B.ERR_SHAPE
