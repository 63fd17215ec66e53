"""The layer for a few tokens at a decoder's widths: clusters that share the up product's contraction, stages that are filled again,
warps that share the router's features; and weights past 2^31 bytes.  Against the formulas in 64 bits, of the chosen experts."""
import numpy as np
import pytest
import torch

from gpu_util import f32, u8
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import few_binding as FB
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L
from mxfp8_precision_gemms_fp8bw_gb300 import moe
from oracle import few as OF
from test_gpu_few_layer import BF16, Case, clear_choice

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def built():
    B.lib(build_if_missing=True)


class Decoded:
    """Experts' weights in 64 bits, each when it is asked for."""
    def __init__(self, w):
        (self.q, self.e8, self.bits), self.kept = L._held(w), {}
        E, R, n = self.q.shape
        self.shape = (E, R, n * 8 // self.bits)

    def __getitem__(self, e):
        if e not in self.kept:
            R = self.shape[1]
            self.kept[e] = OF.mx_weight(u8(self.q[e]), u8(self.e8[e * R:(e + 1) * R]), self.bits)
        return self.kept[e]


class Wide(Case):
    def want(self):
        return OF.few_layer(self.x, self.router, Decoded(self.w13), Decoded(self.w2), self.k, bias=self.bias, **self.how)


LAYERS = [(2, 1, 1536, 96), (2, 2, 2080, 64), (8, 2, 5120, 96), (8, 3, 8192, 64), (4, 2, 4128, 1056), (32, 4, 1184, 992)]
TOKENS = [1, 8, 17, 32]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("E,k,C,F", LAYERS)
def test_against_64_bits(E, k, C, F, M, bits):
    c = Wide(M, E, k, C, F, bits)
    y = c.run()
    c.check(y)
    assert torch.equal(c.run(), y)


def test_these_layers_take_every_path():
    shapes = [(M, *FB.mx_few_moe_shape(M, *layer, bits)) for layer in LAYERS for M in TOKENS for bits in (4, 8)]
    for late in (False, True):  # over 16 tokens, sums meet where the stages were
        up = [u for M, u, _, _ in shapes if (M > 16) == late]
        down = [d for M, _, d, _ in shapes if (M > 16) == late]
        assert {u.cluster for u in up} >= {1, 4, 6, 8} and {d.cluster for d in down} >= {1, 4, 8}
        for spread in (0, 1):
            assert any(u.cluster > 1 and u.spread == spread and u.chunks > u.stages for u in up)
            assert any(u.in_turn and u.spread == spread and u.chunks > u.stages for u in up) or late and spread
            assert any(d.cluster > 1 and d.spread == spread and d.chunks > d.stages for d in down)
    assert {s for *_, s in shapes} >= {6, 10, 16}


@pytest.mark.parametrize("bits,how", [(4, dict(score="sigmoid", groups=8, groups_kept=4, group_top=2, scale=2.5)), (8, dict())])
def test_past_2_to_the_31_bytes(bits, how):
    """256 experts of 7168 x 2048, the last and the first among those chosen."""
    E, k, C, F = 256, 8, 7168, 2048
    g = torch.Generator("cuda").manual_seed(bits)
    rng = np.random.default_rng(bits)

    def held(R, K):
        if bits == 4:
            q = torch.empty(E, R, K // 2, dtype=torch.uint8, device="cuda").random_(0, 256, generator=g)
        else:  # no NaN among the codes
            q = torch.empty(E, R, K, dtype=torch.uint8, device="cuda").random_(0, 0x7F, generator=g)
            q += 128 * torch.empty(E, R, 1, dtype=torch.uint8, device="cuda").random_(0, 2, generator=g)
        e8 = torch.empty(E * R, K // 32, dtype=torch.uint8, device="cuda").random_(*((118, 122) if bits == 4 else (112, 116)), generator=g)
        return (L.Mx4Weights(q, e8) if bits == 4 else L.MxExpertWeights(q, e8, None, None))

    w13, w2 = held(2 * F, C), held(C, F)
    assert L._held(w13)[0].numel() > 2 ** 31 and E * C * F > 2 ** 31
    router = (1.5 / np.sqrt(C) * rng.standard_normal((E, C))).astype(np.float32)
    bias = np.zeros(E, np.float32)
    bias[[0, 64, 254, 255]] = 1.0
    for M in (1, 32):
        x = clear_choice(rng, M, C, router, bias, k, how)
        dev = [torch.from_numpy(a).cuda() for a in (x, router, bias)]
        y = moe.ffn_few(dev[0].bfloat16(), dev[1], w13, w2, k, bias=dev[2], **how)
        rows = sorted({0, M // 2, M - 1})
        want, bound, chosen = OF.few_layer(x[rows], router, Decoded(w13), Decoded(w2), k, bias=bias, **how)
        assert (chosen == 255).any(axis=1).all() and (chosen == 0).any(axis=1).all()
        off = np.abs(f32(y)[rows] - want)
        assert (off <= 1.01 * bound + BF16 * (np.abs(want) + bound) + 1e-37).all()
        assert np.linalg.norm(off) <= 1.05 * BF16 * np.linalg.norm(want)
