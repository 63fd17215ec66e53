"""The layer for a few tokens at a decoder's widths: clusters that share the up product's contraction, stages that are filled again,
warps that share the router's features.  Against the formulas in 64 bits, of the chosen experts."""
import pytest
import torch

from gpu_util import u8
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import few_binding as FB
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L
from oracle import few as OF
from test_gpu_few_layer import Case

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
