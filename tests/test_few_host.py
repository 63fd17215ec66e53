"""Host-side checks of the third part of the C ABI (include/fp8bw_few.h) and of the functions over it (no GPU needed)."""
import os
import re

import pytest
import torch

from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import build, moe
from mxfp8_precision_gemms_fp8bw_gb300 import few_binding as FB
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp8bw_few.h")
P = 1 << 20  # a fake, 16-byte aligned "device" address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return FB.lib()


def test_header_binding_and_library_agree(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*\w+\s+(\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(FB._SIGNATURES)
    assert all(hasattr(lib, n) for n in names)
    assert re.search(r"define FP8BW_FEW_TOKENS (\d+)", text).group(1) == str(FB.FEW_TOKENS)


@pytest.mark.parametrize("code,kw", [
    ("NULL", dict(a0=None)), ("NULL", dict(a3=None)), ("NULL", dict(a4=None)), ("SHAPE", dict(a1=0)),
    ("SHAPE", dict(a2=48)), ("SHAPE", dict(a2=0)), ("SHAPE", dict(a1=-1)), ("ALIGN", dict(a0=P + 8)),
    ("ALIGN", dict(a4=5 * P + 1)), ("ARG", dict(a5=2)), ("LAYOUT", dict(a3=P + 64)), ("LAYOUT", dict(a4=4 * P)),
])
def test_quant_refusals(lib, code, kw):
    ok = [P, 4, 64, 4 * P, 5 * P, 0, None]
    assert lib.mxfp4_quant_1x32_row(*[kw.get(f"a{i}", v) for i, v in enumerate(ok)]) == getattr(B, "ERR_" + code)
    assert B.last_error()


@pytest.mark.parametrize("code,kw", [
    ("NULL", dict(a0=None)), ("NULL", dict(a3=None)), ("SHAPE", dict(a1=0)), ("SHAPE", dict(a2=16)),
    ("ALIGN", dict(a3=2 * P + 4)), ("LAYOUT", dict(a3=P + 16)),
])
def test_widen_refusals(lib, code, kw):
    ok = [P, 4, 64, 2 * P, None]
    assert lib.mxfp4_to_mxfp8(*[kw.get(f"a{i}", v) for i, v in enumerate(ok)]) == getattr(B, "ERR_" + code)


@pytest.mark.parametrize("code,kw", [
    ("NULL", dict(a0=None)), ("NULL", dict(a1=None)), ("NULL", dict(a2=None)), ("NULL", dict(a7=None)), ("NULL", dict(a8=None)),
    ("SHAPE", dict(a4=0)), ("SHAPE", dict(a4=33)), ("SHAPE", dict(a5=0)), ("SHAPE", dict(a6=40)), ("SHAPE", dict(a6=0)),
    ("SHAPE", dict(a6=(1 << 22) + 32)), ("ALIGN", dict(a0=P + 2)), ("ALIGN", dict(a2=3 * P + 4)), ("ALIGN", dict(a7=4 * P + 2)),
    ("ALIGN", dict(a8=50 * P + 8)), ("ARG", dict(a3=6)), ("ARG", dict(a3=16)), ("ARG", dict(a9=100)),
    ("LAYOUT", dict(a7=P + 16)), ("LAYOUT", dict(a7=2 * P)), ("LAYOUT", dict(a7=30 * P)), ("LAYOUT", dict(a8=2 * P + 4096)),
    ("LAYOUT", dict(a8=40 * P)),
])
def test_linear_refusals(lib, code, kw):
    M, N, K = 32, 65, 2048
    ok = [P, 2 * P, 30 * P, 4, M, N, K, 40 * P, 50 * P, lib.mx_few_linear_workspace_bytes(M, N, K), None]
    assert lib.mx_few_linear(*[kw.get(f"a{i}", v) for i, v in enumerate(ok)]) == getattr(B, "ERR_" + code)


def test_linear_workspace(lib):
    size = lib.mx_few_linear_workspace_bytes
    assert size(2, 640, 5120) == 0 and size(32, 640, 5120) >= 32 * 5120 * 2 and size(1, 640, 1 << 20) >= 2 << 20
    assert size(1, 1 << 20, 5120) >= 2 * 5120
    assert size(0, 640, 5120) == size(33, 640, 5120) == size(32, 640, 5100) == size(32, 640, (1 << 22) + 32) == 0
    assert size(32, 0, 5120) == size(32, 1 << 31, 5120) == 0


def test_layer_workspace(lib):
    size = lib.mx_few_moe_workspace_bytes
    assert size(1, 8, 2, 256, 512) > 0
    for bad in ((0, 8, 2, 256, 512), (33, 8, 2, 256, 512), (1, 0, 2, 256, 512), (1, 1025, 2, 256, 512), (1, 8, 9, 256, 512),
                (1, 8, 0, 256, 512), (1, 64, 33, 256, 512), (1, 8, 2, 250, 512), (1, 8, 2, 256, 0), (1, 8, 2, 256, 520),
                (1, 8, 2, (1 << 22) + 32, 32), (1, 512, 2, 256, 1 << 22), (1, 1024, 2, 1 << 22, 256)):
        assert size(*bad) == 0, bad


@pytest.mark.parametrize("code,kw", [
    *(("NULL", {f"a{i}": None}) for i in (0, 1, 3, 4, 5, 6, 19, 20)),
    *(("ALIGN", {f"a{i}": 77 * P + 4}) for i in (0, 1, 2, 3, 4, 5, 6, 19, 20)),
    ("ARG", dict(a7=5)), ("SHAPE", dict(a8=0)), ("SHAPE", dict(a8=33)), ("SHAPE", dict(a9=0)), ("SHAPE", dict(a10=9)),
    ("SHAPE", dict(a11=80)), ("SHAPE", dict(a12=31)), ("SHAPE", dict(a13=3)), ("SHAPE", dict(a13=0)),
    ("SHAPE", dict(a13=4, a14=5)), ("SHAPE", dict(a13=8, a14=1)), ("ARG", dict(a15=3)), ("ARG", dict(a16=2)),
    ("ARG", dict(a21=0)), ("LAYOUT", dict(a19=P)), ("LAYOUT", dict(a20=2 * P)), ("LAYOUT", dict(a19=30 * P, a20=30 * P)),
])
def test_layer_refusals(lib, code, kw):
    M, E, k, C, F = 3, 8, 2, 64, 96
    ok = [P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, 4, M, E, k, C, F, 1, 1, 1, 0, 1, 1.0, 8 * P, 9 * P,
          lib.mx_few_moe_workspace_bytes(M, E, k, C, F), None]
    assert lib.mx_few_moe(*[kw.get(f"a{i}", v) for i, v in enumerate(ok)]) == getattr(B, "ERR_" + code)
    assert B.last_error()


# ------------------------------------------------------------------ the functions

def held4(*shape):
    *lead, K = shape
    n = 1
    for d in lead:
        n *= d
    return L.Mx4Weights(torch.zeros(*lead, K // 2, dtype=torch.uint8), torch.zeros(n, K // 32, dtype=torch.uint8))


def test_gradients_are_refused():
    x = torch.zeros(2, 64, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(RuntimeError, match="no gradient"):
        L.mx_linear_few(x, held4(8, 64))
    with pytest.raises(RuntimeError, match="no gradient"):
        moe.ffn_few(x, torch.zeros(4, 64), held4(4, 128, 64), held4(4, 64, 64), 2)
    with pytest.raises(RuntimeError, match="no gradient"):
        moe.ffn_few(x.detach(), torch.zeros(4, 64, requires_grad=True), held4(4, 128, 64), held4(4, 64, 64), 2)
    layer = moe.MxMoEFFN(256, 512, 4, 2)
    with pytest.raises(RuntimeError, match="no gradient"):
        layer.decode(torch.zeros(2, 256, dtype=torch.bfloat16, requires_grad=True), None)


def test_widths_must_agree():
    w8 = L.MxExpertWeights(torch.zeros(4, 64, 64, dtype=torch.uint8), torch.zeros(256, 2, dtype=torch.uint8), None, None)
    with pytest.raises(ValueError, match="bits"):
        moe.ffn_few(torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(4, 64), held4(4, 128, 64), w8, 2)
    with pytest.raises(ValueError, match="bits"):
        moe.MxMoEFFN(256, 512, 4, 2).weight_codes(bits=6)


def test_too_many_tokens_and_empty_batches():
    w13, w2 = held4(4, 128, 64), held4(4, 64, 64)
    with pytest.raises(B.Fp8bwError, match="at most 32"):
        moe.ffn_few(torch.zeros(33, 64, dtype=torch.bfloat16), torch.zeros(4, 64), w13, w2, 2)
    assert moe.ffn_few(torch.zeros(0, 64, dtype=torch.bfloat16), torch.zeros(4, 64), w13, w2, 2).shape == (0, 64)
    assert L.mx_linear_few(torch.zeros(0, 64, dtype=torch.bfloat16), held4(7, 64)).shape == (0, 7)


def test_tensors_that_are_not_what_the_kernels_read():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        L.mx_linear_few(x, held4(8, 64))
    with pytest.raises(TypeError):
        L.mx_linear_few(x.float(), held4(8, 64))
    with pytest.raises(ValueError, match="CUDA"):
        L.mx4_quantize(torch.zeros(4, 64, dtype=torch.bfloat16))


@pytest.mark.parametrize("which", [0, 1])
def test_codes_of_other_weights_are_refused(which):
    layer = moe.MxMoEFFN(256, 512, 4, 2)
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    codes = [held4(4, 1024, 256), held4(4, 256, 512)]
    with torch.no_grad(), pytest.raises(ValueError, match="codes"):
        layer.decode(x, tuple(codes[::-1]))
    for name in ("q", "e8"):
        bad = list(codes)
        bad[which] = L.Mx4Weights(**{**vars(codes[which]), name: getattr(codes[which], name)[1:]})
        with torch.no_grad(), pytest.raises(ValueError, match=name):
            layer.decode(x, tuple(bad))
        with torch.no_grad(), pytest.raises(ValueError, match=name):
            layer(x, tuple(bad))
    with pytest.raises(ValueError, match="4 bits"):
        layer(x.requires_grad_(), tuple(codes))
