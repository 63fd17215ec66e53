"""More host-side checks of the calls for a few tokens (no GPU needed)."""
import ctypes

import pytest
import torch
from torch.autograd import forward_ad

from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import build, moe
from mxfp8_precision_gemms_fp8bw_gb300 import few_binding as FB
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L

P = 1 << 20  # a fake, 16-byte aligned "device" address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return FB.lib()


def test_self_tests_take_the_calls_arguments_and_a_limit(lib):
    n = lib.mx_few_linear_workspace_bytes(5, 64, 2048)
    linear = [P, 2 * P, 3 * P, 4, 5, 64, 2048, 4 * P, 5 * P, n]
    assert lib.fp8bw_selftest_few_linear(*linear, 2_000_000_001, None) == B.ERR_ARG
    assert "wait_ns" in B.last_error()
    assert lib.fp8bw_selftest_few_linear(*linear[:6], 40, *linear[7:], 0, None) == B.ERR_SHAPE
    n = lib.mx_few_moe_workspace_bytes(3, 8, 2, 64, 96)
    layer = [P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, 4, 3, 8, 2, 64, 96, 1, 1, 1, 0, 1, 1.0, 8 * P, 9 * P, n]
    assert lib.fp8bw_selftest_few_moe(*layer, 2_000_000_001, None) == B.ERR_ARG
    assert lib.fp8bw_selftest_few_moe(*layer[:7], 5, *layer[8:], 0, None) == B.ERR_ARG


# ------------------------------------------------------------------ gradients

def codes4(*shape):
    *lead, K = shape
    n = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    return L.Mx4Weights(torch.zeros(*lead, K // 2, dtype=torch.uint8), torch.zeros(n, K // 32, dtype=torch.uint8))


def calls(x, router, bias):
    layer = moe.MxMoEFFN(256, 512, 4, 2)
    wide = torch.zeros(2, 256, dtype=torch.bfloat16)
    yield lambda: L.mx_linear_few(x(wide), codes4(8, 256))
    yield lambda: moe.ffn_few(x(wide), torch.zeros(4, 256), codes4(4, 128, 256), codes4(4, 256, 64), 2)
    yield lambda: moe.ffn_few(wide, router(torch.zeros(4, 256)), codes4(4, 128, 256), codes4(4, 256, 64), 2)
    yield lambda: moe.ffn_few(wide, torch.zeros(4, 256), codes4(4, 128, 256), codes4(4, 256, 64), 2, bias=bias(torch.zeros(4)))
    yield lambda: layer.decode(x(wide), (codes4(4, 1024, 256), codes4(4, 256, 512)))


def test_dual_tensors_are_refused():
    """Their tangents would be dropped without a word."""
    dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
    with forward_ad.dual_level():
        for no_grad in (False, True):
            with torch.set_grad_enabled(not no_grad):
                for call in calls(dual, dual, dual):
                    with pytest.raises(RuntimeError, match="dual"):
                        call()


@pytest.mark.parametrize("transform", ["jvp", "grad", "vmap"])
def test_function_transforms_are_refused(transform):
    w = codes4(8, 256)
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises((RuntimeError, ValueError)):
        if transform == "jvp":
            torch.func.jvp(lambda t: L.mx_linear_few(t, w), (x,), (torch.ones_like(x),))
        elif transform == "grad":
            torch.func.grad(lambda t: L.mx_linear_few(t, w).float().sum())(x)
        else:
            torch.func.vmap(lambda t: L.mx_linear_few(t, w))(x[None])


def test_decode_takes_a_layer_whose_parameters_require_gradients():
    """Up to the check that this machine has a device: gradients are on, the layer's are not asked for."""
    layer = moe.MxMoEFFN(256, 512, 4, 2)
    assert all(p.requires_grad for p in layer.parameters())
    with pytest.raises(ValueError, match="CUDA"):
        layer.decode(torch.zeros(2, 256, dtype=torch.bfloat16), (codes4(4, 1024, 256), codes4(4, 256, 512)))


def test_shapes_refuse_what_the_calls_refuse(lib):
    out = (ctypes.c_int32 * 6)()
    assert lib.mx_few_linear_shape(33, 64, 2048, 4, out) == B.ERR_SHAPE
    assert lib.mx_few_linear_shape(1, 64, 2048, 5, out) == B.ERR_ARG
    assert lib.mx_few_linear_shape(1, 64, 2048, 4, None) == B.ERR_NULL
    assert lib.mx_few_moe_shape(1, 8, 9, 64, 96, 4, out, out, out) == B.ERR_SHAPE
    assert lib.mx_few_moe_shape(1, 8, 2, 64, 96, 6, out, out, out) == B.ERR_ARG
    for i in range(3):
        assert lib.mx_few_moe_shape(1, 8, 2, 64, 96, 4, *(None if i == j else out for j in range(3))) == B.ERR_NULL
