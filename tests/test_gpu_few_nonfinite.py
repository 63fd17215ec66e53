"""Tokens with an infinity or a NaN in a layer: NaN, whatever the router makes of them, and nothing for the others."""
import numpy as np
import pytest
import torch

from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L
from mxfp8_precision_gemms_fp8bw_gb300 import moe

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(autouse=True)
def built():
    B.lib(build_if_missing=True)


def layer(M, E, C=160, F=96):
    rng = np.random.default_rng(M + 10 * E)
    new = lambda size, *s: torch.from_numpy((size * rng.standard_normal(s)).astype(np.float32)).bfloat16().cuda()  # noqa: E731
    return new(1, M, C), new(0.1, E, C).float(), L.mx4_quantize(new(0.05, E, 2 * F, C)), L.mx4_quantize(new(0.05, E, C, F))


WAYS = [dict(), dict(score="sigmoid"), dict(score="sigmoid", renormalize=False)]
GROUPS = dict(groups=2, groups_kept=1, group_top=2)
SIZES = [(1, 1, 1), (1, 8, 2), (3, 1, 1), (14, 8, 3), (20, 4, 1)]


@pytest.mark.parametrize("value", [INF, -INF, float("nan")])
@pytest.mark.parametrize("router", ["as it is", "positive", "negative", "powers of two"])
@pytest.mark.parametrize("size,how", [(s, h) for s in SIZES for h in WAYS] + [(s, GROUPS) for s in SIZES if s[1] > 1])
def test_the_whole_row_is_nan(size, router, value, how):
    M, E, k = size
    x, r, w13, w2 = layer(M, E)
    if router == "positive":
        r = r.abs()
    elif router == "negative":
        r = -r.abs()
    elif router == "powers of two":  # whose second and third parts are zeros
        r = torch.full_like(r, -0.125)
    clean = moe.ffn_few(x, r, w13, w2, k, **how)
    for feature in (0, 77, 159):
        bad = x.clone()
        rows = sorted({0, M // 2})
        bad[rows, feature] = value
        y = moe.ffn_few(bad, r, w13, w2, k, **how)
        assert bool(torch.isnan(y[rows]).all())
        others = [t for t in range(M) if t not in rows]
        assert torch.equal(y[others], clean[others])
    assert bool(torch.isfinite(clean).all())


def test_no_expert_is_still_zero():
    x, r, w13, w2 = layer(3, 4)
    x[1, 5] = INF
    assert not moe.ffn_few(x, r, w13, w2, 2, bias=torch.full((4,), -INF, device="cuda")).any()


@pytest.mark.parametrize("M", [1, 5])
def test_logits_that_leave_fp32_are_the_routers(M):
    """Finite tokens and an infinite router weight: -inf masks that expert, as in the routing itself."""
    x, r, w13, w2 = layer(M, 4)
    x[:, 9] = x[:, 9].abs() + 1
    off = r.clone()
    off[2, 9] = -INF
    bias = torch.tensor([0.0, 0.0, -INF, 0.0], device="cuda")
    r[2] = 0
    want = moe.ffn_few(x, r, w13, w2, 3, bias=bias, score="sigmoid")
    assert torch.equal(moe.ffn_few(x, off, w13, w2, 3, score="sigmoid"), want)
