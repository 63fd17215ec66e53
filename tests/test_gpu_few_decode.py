"""``MxMoEFFN.decode`` with a balance that shifts or masks the choice, against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

from gpu_util import f32
from mxfp8_precision_gemms_fp8bw_gb300 import moe
from oracle import few as OF
from oracle.moe import moe_route
from test_gpu_few_layer import BF16, clear_choice, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("balance", ["zero", "shifts", "masks"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [1, 4, 20])
def test_the_balance_is_the_bias_of_the_choice(M, bits, balance):
    torch.manual_seed(M + bits)
    rng = np.random.default_rng(M + bits)
    E, k, C, F = 8, 2, 256, 512
    layer = moe.MxMoEFFN(C, F, E, k, score="sigmoid", device="cuda")
    bias = np.zeros(E, np.float32)
    if balance == "shifts":
        bias[:] = rng.permutation(E) * np.float32(0.125)
    elif balance == "masks":
        bias[rng.permutation(E)[:5]] = -np.inf
    x = clear_choice(rng, M, C, f32(layer.router), bias, k, dict(score="sigmoid"))
    codes = layer.weight_codes(colwise=False, bits=bits)
    with torch.no_grad():
        layer.balance.copy_(torch.from_numpy(bias))
    y = layer.decode(torch.from_numpy(x).bfloat16().cuda(), codes)  # gradients are on: the parameters are constants in it
    assert y.grad_fn is None and not y.requires_grad
    want, bound, experts = OF.few_layer(x, f32(layer.router), values(codes[0], (E, 2 * F, C)), values(codes[1], (E, C, F)), k,
                                        bias=bias, score="sigmoid")
    assert (np.abs(f32(y) - want) <= 1.01 * bound + BF16 * (np.abs(want) + bound) + 1e-37).all()
    plain = moe_route(x.astype(np.float64) @ f32(layer.router).astype(np.float64).T, k, score="sigmoid")[0]
    assert balance == "zero" or M == 1 or not np.array_equal(np.sort(plain), np.sort(experts))
