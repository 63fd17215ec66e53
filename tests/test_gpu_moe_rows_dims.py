"""Tokens and plans that do not belong together are refused, without tokens too."""
import pytest
import torch

from gpu_util import lib
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


@pytest.mark.parametrize("planned,given", [(5, 0), (0, 5), (5, 4), (4, 5)])
def test_tokens_that_are_not_the_plans(planned, given):
    bf = lambda *shape: torch.ones(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    p = moe.plan(torch.zeros(planned, 1, dtype=torch.int32, device="cuda"), 4)
    right, wrong, y = torch.ones(planned, 1, device="cuda"), torch.ones(given, 1, device="cuda"), bf(p.rows, 64)
    for call in (lambda: moe.dispatch(bf(given, 64), p), lambda: moe.combine_backward(bf(given, 64), y, right, p),
                 lambda: moe.combine_backward(bf(given, 64), y, wrong, p),
                 lambda: moe.combine_backward(bf(planned, 64), y, wrong, p)):
        with pytest.raises(ValueError):
            call()
    B.fp8bw_sync_status()
    moe.dispatch(bf(planned, 64), p)
    moe.combine_backward(bf(planned, 64), y, right, p)
    B.fp8bw_sync_status()
