"""MXFP4 weights on the GPU: codes and scales byte for byte, and their widening to MXFP8."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import adversarial_bf16, f32, u8
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import few_binding as FB
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L
from oracle import few as OF

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def built():
    B.lib(build_if_missing=True)


def check(w, mode=B.MX_RCEIL):
    got = L.mx4_quantize(w.cuda(), mode)
    q, e8 = OF.mx4_quant_row(f32(w).reshape(-1, w.shape[-1]), mode)
    assert np.array_equal(u8(got.e8), e8)
    assert np.array_equal(u8(got.q).reshape(q.shape), q)
    wide = L.mx4_widen(got)
    assert wide.e8_row is got.e8 and wide.qT_col is None
    assert np.array_equal(u8(wide.q_row).reshape(-1, w.shape[-1]), OF.mx4_widen(q))
    return got


@pytest.mark.parametrize("mode", [B.MX_RCEIL, B.MX_FLOOR])
@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (7, 416), (288, 2080), (65, 1056), (2, 17, 96), (4, 256, 512)])
def test_codes_equal_the_oracle(shape, mode):
    rng = np.random.default_rng(sum(shape))
    w = rng.standard_normal(shape).astype(np.float32) * np.exp2(rng.integers(-40, 41, (*shape[:-1], 1))).astype(np.float32)
    check(torch.from_numpy(w).bfloat16(), mode)


@pytest.mark.parametrize("mode", [B.MX_RCEIL, B.MX_FLOOR])
def test_adversarial_blocks(mode):
    check(adversarial_bf16(96, 1024, 3, block=32), mode)


@pytest.mark.parametrize("mode", [B.MX_RCEIL, B.MX_FLOOR])
def test_every_finite_bf16_as_a_largest_magnitude(mode):
    bits = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    w = torch.zeros(bits.numel(), 32, dtype=torch.bfloat16)
    w[:, 5] = bits
    w[:, 17] = -bits
    w[:, 20] = bits / 3
    check(w, mode)


def test_ties_go_to_the_even_code():
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    w = torch.zeros(3, 32)
    for r, s in enumerate((1.0, 2.0 ** -20, 2.0 ** 33)):
        w[r, 0] = 6.0 * s
        w[r, 1:8] = ties * s
        w[r, 8:15] = -ties * s
    got = check(w.bfloat16())
    assert u8(got.e8).ravel().tolist() == [127, 107, 160]


def test_blocks_that_are_not_finite_are_nan():
    w = torch.randn(4, 96).bfloat16()
    w[1, 40], w[2, 0], w[3, 95] = float("nan"), float("inf"), float("-inf")
    got = L.mx4_quantize(w.cuda())
    e8 = u8(got.e8)
    bad = {(1, 1), (2, 0), (3, 2)}
    assert all((e8[r, b] == 255) == ((r, b) in bad) for r in range(4) for b in range(3))
    ok = OF.mx4_quant_row(np.where(np.isfinite(f32(w)), f32(w), 0))[0].reshape(4, 3, 16)
    for r in range(4):
        for b in range(3):
            if (r, b) not in bad:
                assert np.array_equal(u8(got.q).reshape(4, 3, 16)[r, b], ok[r, b])


def test_every_byte_widens():
    q = torch.arange(256, dtype=torch.uint8).repeat(3).view(3, 256).cuda()
    out = torch.empty(3, 512, dtype=torch.uint8, device="cuda")
    FB.mxfp4_to_mxfp8(q, out)
    assert np.array_equal(u8(out), OF.mx4_widen(u8(q)))


def test_nothing_is_written_behind_the_outputs():
    w = torch.randn(5, 96).bfloat16().cuda()
    q, e8, wide = (torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda") for n in (240, 15, 480))
    FB.mxfp4_quant_1x32_row(w, q[:240].view(5, 48), e8[:15].view(5, 3))
    FB.mxfp4_to_mxfp8(q[:240].view(5, 48), wide[:480].view(5, 96))
    assert all(bool((t[n:] == 0xA5).all()) for t, n in ((q, 240), (e8, 15), (wide, 480)))


def test_layouts_are_refused():
    w = torch.randn(8, 64, device="cuda").bfloat16()
    with pytest.raises(ValueError, match="contiguous"):
        L.mx4_quantize(w.t().contiguous().t()[:, :32])
    with pytest.raises(B.Fp8bwError):
        L.mx4_quantize(torch.randn(8, 48, device="cuda").bfloat16())
    with pytest.raises(TypeError):
        L.mx4_quantize(w.float())


def test_past_2_to_the_31_weights():
    R, C = 65664, 32768  # 2^31 + 4194304 weights
    w = torch.empty(R, C, dtype=torch.bfloat16, device="cuda").normal_(0, 0.02)
    got = L.mx4_quantize(w)
    wide = L.mx4_widen(got)
    for r in (0, 65535, 65536, R - 1):
        q, e8 = OF.mx4_quant_row(f32(w[r:r + 1]))
        assert np.array_equal(u8(got.q[r:r + 1]), q) and np.array_equal(u8(got.e8[r:r + 1]), e8)
        assert np.array_equal(u8(wide.q_row[r:r + 1]), OF.mx4_widen(q))
