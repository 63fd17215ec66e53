"""The gated activation where the sigmoid leaves the normal range of fp32: blocks of nothing but far negative gates."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import f32, lib, u8
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import moe
from oracle import moe as O
from test_gpu_swiglu import check_codes, t

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


def ups(r, shape, size):
    return r.choice([-1.0, 1.0], size=shape) * r.uniform(0.5, 2.0, size=shape) * size


# check_codes allows 2^-15 of a value.  Here: 64 units of 2^-24 of the exponent's argument, and a subnormal sigmoid of at
# least 2^-128 (and its products with da and up of at least 1/2 each, 2^-130) rounded to a multiple of 2^-149: 2^-18 + 3 * 2^-20.
@pytest.mark.parametrize("mode", [B.MX_RCEIL, B.MX_FLOOR])
@pytest.mark.parametrize("gates", [(-88.5, -88.0, -87.5), (-87.5, -87.0, -86.5), (-80.0, -60.0)])
def test_forward(gates, mode):
    r = np.random.default_rng(int(-2 * gates[0]))
    for size in (1.0, 2.0 ** 20):
        h = np.concatenate([r.choice(gates, size=(64, 96)), ups(r, (64, 96), size)], axis=1).astype(np.float32)
        h = torch.from_numpy(h).bfloat16().cuda()
        a, _ = moe.swiglu(h, mode=mode)
        B.fp8bw_sync_status()
        ref = O.swiglu(f32(h))
        check_codes(a.q, a.e8, ref, mode)
        check_codes(a.qT, a.e8T, t(ref), mode)


@pytest.mark.parametrize("gate", [-88.0, -80.0, -64.0])
def test_gradient(gate):
    """Gates that e4m3 holds exactly, so that the kept ones are these."""
    r = np.random.default_rng(int(-gate))
    h = np.concatenate([np.full((64, 96), gate), ups(r, (64, 96), 1.0)], axis=1).astype(np.float32)
    _, kept = moe.swiglu(torch.from_numpy(h).bfloat16().cuda())
    values = oracle.mx_dequant_row(u8(kept.q), u8(kept.e8))
    assert np.all(values[:, :96] == gate)
    da = torch.from_numpy(ups(r, (64, 96), 1.0).astype(np.float32)).bfloat16().cuda()
    dh = moe.swiglu_backward(da, kept)
    B.fp8bw_sync_status()
    ref = O.swiglu_bwd(f32(da), values)
    check_codes(dh.q, dh.e8, ref, B.MX_RCEIL)
    check_codes(dh.qT, dh.e8T, t(ref), B.MX_RCEIL)


def test_beyond_fp32_the_sigmoid_is_zero():
    """1 + exp(89) is over fp32: zeros, finite, in the activation and in its gradient."""
    h = torch.cat([torch.full((32, 32), -96.0), torch.ones(32, 32)], dim=1).bfloat16().cuda()
    a, kept = moe.swiglu(h)
    dh = moe.swiglu_backward(torch.ones(32, 32, device="cuda").bfloat16(), kept)
    B.fp8bw_sync_status()
    assert not (a.q & 0x7F).any() and not a.e8.any() and not (dh.q & 0x7F).any() and not dh.e8.any()
