"""The layer for a few tokens where every value and sum is a whole number that fp32 holds: nothing may be lost on the way.

The gate is 32 or more, where silu(gate) is the gate itself in fp32 (1 + e^-32 rounds to 1), up is any number of 24 bits, put
together from the powers of two that the blocks' scales are, and the second product takes differences.  So the result is the
exact difference, rounded once to bf16: no tolerance.
"""
import numpy as np
import pytest
import torch

from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L
from mxfp8_precision_gemms_fp8bw_gb300 import moe
from test_gpu_few_layer import Case, clear_choice

pytestmark = pytest.mark.gpu
ONE = {4: 2, 8: 0x38}     # codes of 1.0
MINUS = {4: 10, 8: 0xB8}  # and of -1.0


@pytest.fixture(autouse=True)
def built():
    B.lib(build_if_missing=True)


def pack(codes, e8, bits):
    codes, e8 = torch.from_numpy(codes), torch.from_numpy(e8.reshape(-1, e8.shape[-1])).cuda()
    if bits == 8:
        return L.MxExpertWeights(codes.cuda(), e8, None, None)
    return L.Mx4Weights((codes[..., 0::2] | codes[..., 1::2] << 4).cuda(), e8)


def whole_numbers(M, E, C, F, bits):
    """x, router, w13, w2 and the result in fp32: token t goes to expert t % E, times 4^(t % 3)."""
    rng = np.random.default_rng(M + 5 * E + 7 * C + 11 * F + bits)
    A = rng.integers(1 << 22, 1 << 24, (E, F))
    A[:, rng.permutation(F)[:F // 4]] >>= rng.integers(0, 20, F // 4)  # and smaller ones among them
    q13, e13 = np.zeros((E, 2 * F, C), np.uint8), np.full((E, 2 * F, C // 32), 127, np.uint8)
    for b in range(24):
        q13[:, F:, 32 * b] = np.where(A >> b & 1, ONE[bits], 0)
        e13[:, F:, b] = 127 + b
    q13[:, :F, 32 * 24] = ONE[bits]
    e13[:, :F, 24] = 127 + 5
    q2 = np.zeros((E, C, F), np.uint8)
    first = rng.integers(0, F, (E, C))
    second = (first + rng.integers(1, F, (E, C))) % F
    np.put_along_axis(q2, first[..., None], ONE[bits], 2)
    np.put_along_axis(q2, second[..., None], MINUS[bits], 2)
    x, router = np.zeros((M, C), np.float32), np.zeros((E, C), np.float32)
    t = np.arange(M)
    size = 2.0 ** (t % 3)
    x[:, :25 * 32:32] = size[:, None]
    x[t, 24 * 32 + 1 + t % E] = 1
    router[np.arange(E), 24 * 32 + 1 + np.arange(E)] = 8
    want = np.take_along_axis(A, first, 1) - np.take_along_axis(A, second, 1)
    y = torch.from_numpy((want[t % E] * (32 * size * size)[:, None]).astype(np.float32)).bfloat16()
    return (torch.from_numpy(x).bfloat16().cuda(), torch.from_numpy(router).cuda(), pack(q13, e13, bits),
            pack(q2, np.full((E, C, F // 32), 127, np.uint8), bits), y)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("C,F", [(832, 96), (896, 384), (1024, 1056)])
@pytest.mark.parametrize("M,E", [(1, 1), (1, 5), (2, 1), (5, 2), (8, 1), (16, 3), (17, 17), (19, 1), (20, 1), (22, 1), (23, 1), (25, 1),
                                 (26, 1), (29, 1), (32, 1), (32, 3)])
def test_no_bit_of_the_activation_is_lost(M, E, C, F, bits):
    x, router, w13, w2, want = whole_numbers(M, E, C, F, bits)
    assert torch.equal(moe.ffn_few(x, router, w13, w2, 1).cpu(), want)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("E,F", [(256, 160), (1024, 96)])
def test_one_expert_of_many_that_every_token_chooses(E, F, bits):
    """The down product's stages are at their largest, beside a plan of hundreds of experts."""
    M, k, C = 32, 32, 64
    c = Case(M, E, k, C, F, bits)
    c.bias = np.zeros(E, np.float32)
    c.bias[E // 2] = 1.0
    c.x = clear_choice(np.random.default_rng(E), M, C, c.router, c.bias, k, {})
    c.tx, c.tbias = torch.from_numpy(c.x).bfloat16().cuda(), torch.from_numpy(c.bias).cuda()
    chosen = c.want()[2]
    assert (chosen == E // 2).any(axis=1).all() and len(np.unique(chosen)) > 128
    c.check(c.run())
