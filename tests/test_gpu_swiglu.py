"""GPU parity of the gated activation with its 8-bit checkpoint, and of its gradient, against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import f32, lib, u8
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import moe
from oracle import moe as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


# fp32 evaluation of the formulas: exp of a rounded argument up to 100 in magnitude (100 u) with a few ulp of its own, a
# reciprocal, and up to eight products and sums, all of them of terms of one sign or bounded by |gate| + 1
REL = 2.0 ** -15


def check_codes(q, e8, ref, mode, slack=None):
    """Codes q, e8 of 64-bit values ref [R, C], blocks along C, where the kernel's fp32 value is within REL of ref (plus
    slack): the exponent is the rule's for an amax that close, and each code is within half an e4m3 step of the value."""
    q, e8 = u8(q), u8(e8)
    R, C = ref.shape
    amax = np.abs(ref).reshape(R, C // 32, 32).max(axis=2)
    extra = np.zeros_like(amax) if slack is None else slack.reshape(R, C // 32, 32).max(axis=2)
    lo = oracle.e8m0_exponent(np.maximum(amax * (1 - REL) - extra, 0), mode)
    hi = oracle.e8m0_exponent(amax * (1 + REL) + extra, mode)
    E = e8.astype(np.int64) - 127
    assert np.all((lo <= E) & (E <= hi))
    # the exponent is the exact rule's but for the blocks whose amax lies that close to a power of two's boundary
    assert np.mean(lo != hi) < 0.01
    step = np.repeat(np.ldexp(1.0, E), 32, axis=1)
    got = oracle.mx_dequant_row(q, e8)
    top = 448 * step
    want = np.clip(ref, -top, top)      # FLOOR saturates the top of a block
    half = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * step)
    wide = REL * np.abs(ref) + (0 if slack is None else slack)
    assert np.all(np.abs(got - want) <= half * (1 + 2.0 ** -10) + wide)


def t(a):
    return np.ascontiguousarray(a.T)


SHAPES = [(32, 32), (32, 64), (64, 96), (96, 160), (128, 128), (160, 2080), (4064, 64)]


@pytest.mark.parametrize("mode", [B.MX_RCEIL, B.MX_FLOOR])
@pytest.mark.parametrize("R,F", SHAPES)
def test_forward_and_backward(R, F, mode):
    r = np.random.default_rng(R + F)
    hn = r.standard_normal((R, 2 * F)).astype(np.float32)
    hn *= np.exp2(r.integers(-6, 4, size=(R, 1))).astype(np.float32)
    hn[0, :32] = 0                        # an all-zero block
    hn[1, 3], hn[1, F + 3] = -90.0, 50.0    # a gate whose sigmoid is tiny
    h = torch.from_numpy(hn).bfloat16().cuda()
    a, kept = moe.swiglu(h, mode=mode)
    B.fp8bw_sync_status()
    ref = O.swiglu(f32(h))
    check_codes(a.q, a.e8, ref, mode)
    check_codes(a.qT, a.e8T, t(ref), mode)
    # the checkpoint is a plain quantization of h: exact
    hq, he = oracle.mx_quant_1x32_row(f32(h), mode)
    assert np.array_equal(u8(kept.q), hq) and np.array_equal(u8(kept.e8), he)

    da = torch.from_numpy((r.standard_normal((R, F)) * 1e-3).astype(np.float32)).bfloat16().cuda()
    dh = moe.swiglu_backward(da, kept, mode=mode)
    B.fp8bw_sync_status()
    values = oracle.mx_dequant_row(hq, he)
    ref = O.swiglu_bwd(f32(da), values)
    # 1 + gate (1 - sig) cancels near gate = -1.28: what it loses is relative to its terms
    gate, up = values[:, :F], values[:, F:]
    with np.errstate(over="ignore"):
        sig = 1 / (1 + np.exp(-gate))
    slack = np.concatenate([2.0 ** -21 * np.abs(f32(da) * up * sig) * (1 + np.abs(gate)), np.zeros_like(gate)], axis=1)
    check_codes(dh.q, dh.e8, ref, mode, slack)
    check_codes(dh.qT, dh.e8T, t(ref), mode, t(slack))


def test_parts_on_request_are_the_same():
    h = torch.randn(96, 384, device="cuda").bfloat16()
    a, kept = moe.swiglu(h)
    for keep in (False, True):
        for colwise in (False, True):
            b, k2 = moe.swiglu(h, keep=keep, colwise=colwise)
            assert torch.equal(a.q, b.q) and torch.equal(a.e8, b.e8)
            assert (b.qT is not None) == colwise and (k2 is not None) == keep
            if colwise:
                assert torch.equal(a.qT, b.qT) and torch.equal(a.e8T, b.e8T)
            if keep:
                assert torch.equal(kept.q, k2.q) and torch.equal(kept.e8, k2.e8)
    B.fp8bw_sync_status()


def test_extreme_gates_stay_finite_and_nan_shows():
    h = torch.zeros(32, 128, device="cuda").bfloat16()
    h[0, 0], h[0, 64] = -3.0e38, 1.0
    h[1, 0], h[1, 64] = 3.0e38, 1.0
    h[2, 33], h[2, 97] = float("nan"), 1.0
    a, kept = moe.swiglu(h)
    da = torch.ones(32, 64, device="cuda").bfloat16()
    dh = moe.swiglu_backward(da, kept)
    B.fp8bw_sync_status()
    v = oracle.mx_dequant_row(u8(a.q), u8(a.e8))
    assert v[0, 0] == 0 and np.isfinite(v[0]).all() and 2.5e38 < v[1, 0] < 3.3e38
    assert int(a.q[2, 33]) & 0x7F == 0x7F and int(a.qT[33, 2]) & 0x7F == 0x7F
    d = oracle.mx_dequant_row(u8(dh.q), u8(dh.e8))
    assert np.isfinite(d[:2]).all() and np.isnan(d[2, 33])


def test_gradient_against_differences():
    """The gradient of sum(da * a) by differences of the 64-bit activation at the kept values, within the codes' step."""
    r = np.random.default_rng(8)
    h = torch.from_numpy(r.standard_normal((32, 64)).astype(np.float32)).bfloat16().cuda()
    da = torch.from_numpy(r.standard_normal((32, 32)).astype(np.float32)).bfloat16().cuda()
    _, kept = moe.swiglu(h)
    dh = moe.swiglu_backward(da, kept)
    values = oracle.mx_dequant_row(u8(kept.q), u8(kept.e8))
    d = 1e-6
    slope = np.zeros_like(values)
    for c in range(64):
        up, down = values.copy(), values.copy()
        up[:, c] += d
        down[:, c] -= d
        slope[:, c] = (f32(da) * (O.swiglu(up) - O.swiglu(down))).sum(axis=1) / (2 * d)
    check_codes(dh.q, dh.e8, slope, B.MX_RCEIL, slack=np.full_like(slope, 1e-7))


def test_past_2_to_the_31_elements():
    """h, its codes and the gradient's past the int32 range of flat offsets, checked on the last rows."""
    R, F = 524352, 2080
    h = torch.empty(R, 2 * F, dtype=torch.bfloat16, device="cuda").normal_()
    a, kept = moe.swiglu(h)
    tail = h[-32:].contiguous()
    b, k2 = moe.swiglu(tail)
    assert h.numel() > 2 ** 31
    assert torch.equal(a.q[-32:], b.q) and torch.equal(a.qT[:, -32:], b.qT) and torch.equal(a.e8T[:, -1:], b.e8T)
    assert torch.equal(kept.q[-32:], k2.q) and torch.equal(kept.e8[-32:], k2.e8)
    del a
    da = torch.empty(R, F, dtype=torch.bfloat16, device="cuda").normal_()
    dh = moe.swiglu_backward(da, kept)
    dt = moe.swiglu_backward(da[-32:].contiguous(), k2)
    B.fp8bw_sync_status()
    assert torch.equal(dh.q[-32:], dt.q) and torch.equal(dh.e8[-32:], dt.e8)
    assert torch.equal(dh.qT[:, -32:], dt.qT) and torch.equal(dh.e8T[:, -1:], dt.e8T)


def test_replays_in_a_graph_on_another_stream():
    h = torch.randn(64, 256, device="cuda").bfloat16()
    da = torch.randn(64, 128, device="cuda").bfloat16()
    ref = moe.swiglu_backward(da, moe.swiglu(h)[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, kept = moe.swiglu(h)
        dh = moe.swiglu_backward(da, kept)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g.replay()
    side.synchronize()
    assert torch.equal(dh.q, ref.q) and torch.equal(dh.qT, ref.qT)
