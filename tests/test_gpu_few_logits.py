"""The router's logits in the layer for a few tokens: fp32 sums, seen through the choice and through the weights."""
import numpy as np
import pytest
import torch

from gpu_util import f32
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L
from mxfp8_precision_gemms_fp8bw_gb300 import moe

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def built():
    B.lib(build_if_missing=True)


def experts_that_name_themselves(E, C):
    """Expert e gives 32 in feature e and zeros elsewhere, to tokens whose last feature is 1 (silu(32) is 32 in fp32)."""
    F = (E + 31) // 32 * 32
    w13, w2 = np.zeros((E, 2 * F, C), np.uint8), np.zeros((E, C, F), np.uint8)
    w13[:, :, -1] = 0x38  # 1.0
    e = np.arange(E)
    w2[e, e, e] = 0x38
    e13, e2 = np.full((E, 2 * F, C // 32), 127, np.uint8), np.full((E * C, F // 32), 127, np.uint8)
    e13[:, :F, -1] += 5
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return (L.MxExpertWeights(dev(w13), dev(e13.reshape(E * 2 * F, -1)), None, None), L.MxExpertWeights(dev(w2), dev(e2), None, None))


@pytest.mark.parametrize("E,C", [(8, 160), (40, 608), (40, 5120), (8, 5120), (3, 8192), (200, 2048), (300, 1536)])
@pytest.mark.parametrize("M", [1, 3, 9, 17, 32])
def test_sums_of_whole_numbers_are_exact(M, E, C):
    """Logits are whole numbers (times 2^-14) below 2^24, and so are all their partial sums: experts differ by a few units of
    2^23, many not at all, and the choice is the first of the largest."""
    rng = np.random.default_rng(M + 3 * E + 5 * C)
    x = rng.integers(-40, 41, (M, C)).astype(np.float64)
    wide = rng.permutation(C - 1)[:24]  # router weights of 17 and more bits: two and three parts
    x[:, wide] = rng.choice([-1, 1], (M, 24))
    x[:, -1] = 1
    base = rng.integers(-40, 41, C).astype(np.float64)
    base[wide] = rng.integers(1 << 17, 1 << 18, 24) * rng.choice([-1, 1], 24)
    base[-1] = 0
    router = np.tile(base, (E, 1))
    router[:, wide[:6]] += rng.choice([-1, 0, 1], (E, 6))  # the only ones in which experts differ
    assert (np.abs(x) @ np.abs(router).T).max() < 2 ** 24
    logits = x @ router.T
    want = logits.argmax(axis=1)
    assert np.ptp(logits, axis=1).max() <= 12
    w13, w2 = experts_that_name_themselves(E, C)
    y = moe.ffn_few(torch.from_numpy(x).bfloat16().cuda(), torch.from_numpy(router * 2.0 ** -14).float().cuda(), w13, w2, 1)
    expected = np.zeros((M, C), np.float32)
    expected[np.arange(M), want] = 32
    assert np.array_equal(f32(y), expected)


@pytest.mark.parametrize("E,C", [(8, 160), (16, 2048), (64, 5120), (8, 8192)])
@pytest.mark.parametrize("M", [1, 4, 20, 32])
def test_what_is_left_of_sums_that_cancel(M, E, C):
    """Logits of about -5 that are left of magnitudes which add up to thousands.  A weight is sigmoid(logit), so that bf16 shows
    a logit to 2^-9.

    The sum's error: C / 256 features a block, at least 32, 16 at a time, are at most 32 additions (with the parts that warps of
    the block add up), and 16 of blocks, each off by 2^-24 of at most the sum S of magnitudes; 16 features' products are cut off
    at 2^-23 of their largest, 48 times at most, which over all pieces is 48 * 2^-23 / 16 of S if the products are alike, and
    never over 48 * 2^-23 S / 2 with one product for half of S: 72 * 2^-24 S."""
    rng = np.random.default_rng(M + 3 * E + 5 * C)
    x = torch.from_numpy(rng.standard_normal((M, C)).astype(np.float32)).bfloat16()
    own = 64 + np.arange(M)  # a feature that is one token's alone: its router weight brings the logit to about -5
    x[:, own] = 0
    x[np.arange(M), own] = 1
    x[:, -1] = 1
    xd = x.double().numpy()
    router = (1.25 * 5120 / C * rng.standard_normal((E, C))).astype(np.float32)
    router[:, -1] = 0
    router[:, own] = 0
    aim = rng.uniform(-6, -4, (M, E))
    router[:, own] = (aim - xd @ router.astype(np.float64).T).T.astype(np.float32)
    rd = router.astype(np.float64)
    logits, S = xd @ rd.T, np.abs(xd) @ np.abs(rd).T
    assert S.max() > 2000 * min(1, C / 5120) and np.abs(logits - aim).max() < 0.01
    w13, w2 = experts_that_name_themselves(E, C)
    k = min(E, 32)
    y = f32(moe.ffn_few(x.cuda(), torch.from_numpy(router).cuda(), w13, w2, k, score="sigmoid", renormalize=False))[:, :E]
    want = 1 / (1 + np.exp(-logits)) * 32
    chosen = y > 0
    assert (chosen.sum(axis=1) == k).all()
    # a relative error of a weight is one of its logit, of rounding (2^-8) and of the sigmoid (an ulp or two of fp32)
    off = np.abs(np.where(chosen, y, want) / want - 1)
    assert (off <= 1.05 * 72 * 2.0 ** -24 * S + 2.0 ** -8 + 2.0 ** -20).all(), float((off / (72 * 2.0 ** -24 * S + 2.0 ** -8)).max())
