"""Choices without an expert have weight 0, whatever stands beside them in the row."""
import pytest
import torch

from gpu_util import lib
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(8, 4), (16, 3), (64, 8), (160, 12), (600, 5)])
def test_weight_zero_beside_nan_and_infinity(E, k, score, dtype):
    """Two experts left by the mask, one of them NaN or, for the softmax, infinite: the empty choices stay 0."""
    x = torch.full((3, E), float("-inf"), device="cuda")
    x[:, 1], x[:, E - 1] = 0.5, 0.25
    x[0, E - 1] = float("nan")
    x[1, E - 1] = float("inf")
    for renormalize in (True, False):
        experts, weights = moe.route(x.to(dtype), k, score=score, renormalize=renormalize, scale=2.0)
        B.fp8bw_sync_status()
        assert bool((experts[:, 2:] == -1).all()) and not bool((experts[:, :2] == -1).any())
        assert bool((weights[:, 2:] == 0).all())
        assert bool(weights[0].isnan().any()) and bool(weights[2].isfinite().all())


def test_weight_zero_under_an_infinite_scale():
    x = torch.full((1, 8), float("-inf"), device="cuda")
    x[0, 2] = 0.0
    experts, weights = moe.route(x, 2, scale=float("inf"))
    assert experts.tolist() == [[2, -1]] and weights.tolist() == [[float("inf"), 0.0]]
