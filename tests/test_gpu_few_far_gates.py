"""Gates far below 0 in the layer for a few tokens, where sigmoid(gate) leaves the normal range of fp32 and large up's bring the
activation back into it."""
import numpy as np
import pytest
import torch

from gpu_util import f32
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L
from mxfp8_precision_gemms_fp8bw_gb300 import moe

pytestmark = pytest.mark.gpu
BF16 = torch.finfo(torch.bfloat16).eps / 2
GATES = [-60.0, -79.5, -80.5, -87.0, -88.5, -89.0, -90.5, -92.0, -95.0, -98.0, -100.0]


@pytest.mark.parametrize("M", [1, 11, 32])
@pytest.mark.parametrize("size", [2.0 ** 50, 2.0 ** 80])
def test_against_64_bits(M, size):
    """gate = x[0], up = x[32] * size, y = the activation.  expf is off by 2 units in the last place, and where its result is
    subnormal by 2^-148; gate * e, that and up, the division and 1 + e are rounded."""
    B.lib(build_if_missing=True)
    C = F = 64
    w13, w2 = torch.zeros(1, 2 * F, C, dtype=torch.uint8), torch.zeros(1, C, F, dtype=torch.uint8)
    e13, e2 = torch.full((2 * F, 2), 127, dtype=torch.uint8), torch.full((C, 2), 127, dtype=torch.uint8)
    w13[0, :F, 0], w13[0, F:, 32] = 0x38, 0x38
    e13[F:, 1] += int(np.log2(size))
    w2[0, torch.arange(C), torch.arange(C)] = 0x38
    gate = np.array((GATES * 3)[:M])
    up = np.random.default_rng(M).choice([-1.5, 1.0, 3.0], M)
    x = torch.zeros(M, C)
    x[:, 0], x[:, 32] = torch.from_numpy(gate), torch.from_numpy(up)
    y = moe.ffn_few(x.bfloat16().cuda(), torch.zeros(1, C, device="cuda"), L.MxExpertWeights(w13.cuda(), e13.cuda(), None, None),
                    L.MxExpertWeights(w2.cuda(), e2.cuda(), None, None), 1)
    want = (gate / (1 + np.exp(-gate)) * up * size)[:, None]
    bound = BF16 + 8 * 2.0 ** -24 + 2.0 ** -148 / np.exp(gate)[:, None]
    off = np.abs(f32(y) / want - 1)
    assert (off <= bound).all(), (off / bound).max(axis=1)
