"""y = x W^T for a few tokens with MX weights, against the product in 64 bits.

Bound of an element: products are exact in fp32 (8 bits times 4), K of them are summed with at most K roundings (or
truncations) of 2^-23 of the sum of magnitudes; a token is held in two parts of e4m3 in
blocks of 32: the first leaves at most 1/14 of the block's largest element (half a step, 16, of more than 224), the second's
power of two is thus at most 2^-11 of that element and its smallest step 2^-9 of its power of two, so that what is left of an
element is nothing, or at most 2^-21 of the largest; and the result is rounded once to bf16, 2^-8 of it, or, below 2^-126, where bf16 values are
2^-133 apart, 2^-134.
"""
import numpy as np
import pytest
import torch

from gpu_util import f32, u8
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import few_binding as FB
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L
from oracle import few as OF

pytestmark = pytest.mark.gpu
BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(autouse=True)
def built():
    B.lib(build_if_missing=True)


def held(w, bits):
    if bits == 4:
        return L.mx4_quantize(w)
    c = L.mx_quantize_experts(w[None], colwise=False)
    return L.MxExpertWeights(c.q_row[0], c.e8_row, None, None)


def values(w):
    q, e8, bits = L._held(w)
    return OF.mx_weight(u8(q), u8(e8), bits)


def inputs(M, N, K, bits, seed=0):
    rng = np.random.default_rng(seed + 7 * M + 11 * N + 13 * K + bits)
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).bfloat16().cuda()
    w = torch.from_numpy((0.02 * rng.standard_normal((N, K))).astype(np.float32)).bfloat16().cuda()
    return x, held(w, bits)


def check(y, x, w, floor=0.0):
    W, xd = values(w), f32(x).astype(np.float64)
    K = xd.shape[1]
    want = xd @ W.T
    top = np.repeat(np.abs(xd).reshape(len(xd), -1, 32).max(axis=2), 32, axis=1)
    bound = BF16 * np.abs(want) + 2.0 ** -134 + 1.01 * (K * 2.0 ** -23 * (np.abs(xd) @ np.abs(W).T) + 2.0 ** -21 * (top @ np.abs(W).T)) + floor
    assert (np.abs(f32(y) - want) <= bound).all(), float((np.abs(f32(y) - want) / np.maximum(bound, 1e-300)).max())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 32), (1, 17, 64), (2, 300, 16384), (1, 130, 16416), (3, 2100, 128), (2, 40000, 4096), (1, 2048, 2048), (2, 33, 96), (3, 100, 416), (5, 257, 2080), (7, 64, 1056), (8, 160, 512),
    (9, 31, 160), (13, 130, 4128), (16, 512, 256), (17, 48, 992), (24, 65, 2048), (25, 129, 320), (31, 1000, 544),
    (32, 1, 32), (32, 640, 1024), (1, 5, 16384), (4, 3, 33024), (32, 7, 20000 // 32 * 32),
])
def test_against_64_bits(M, N, K, bits):
    x, w = inputs(M, N, K, bits)
    check(L.mx_linear_few(x, w), x, w)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", range(1, 33))
def test_every_token_count(M, bits):
    x, w = inputs(M, 80, 736, bits)
    check(L.mx_linear_few(x, w), x, w)


@pytest.mark.parametrize("bits", [4, 8])
def test_large(bits):
    x, w = inputs(6, 8192, 5120, bits)
    check(L.mx_linear_few(x, w), x, w)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [1, 8, 20])
def test_magnitudes_far_apart(M, bits):
    """Tokens and blocks from 2^-100 to 2^60, zeros, a lone huge element, subnormals."""
    rng = np.random.default_rng(M)
    K, N = 1024, 96
    x = rng.standard_normal((M, K)) * np.exp2(rng.integers(-100, 61, (M, K // 32))).repeat(32, axis=1)
    x[:, 64:128] = 0
    x[:, 200] = 2.0 ** 70
    x[M - 1] = rng.standard_normal(K) * 2.0 ** -130  # bf16 subnormals
    x = torch.from_numpy(x).bfloat16().cuda()
    w = held(torch.from_numpy(rng.standard_normal((N, K)) * np.exp2(rng.integers(-20, 21, (N, 1)))).bfloat16().cuda(), bits)
    # sums of subnormal products may lose what is below the smallest fp32
    check(L.mx_linear_few(x, w), x, w, floor=K * 2.0 ** -149)


@pytest.mark.parametrize("bits", [4, 8])
def test_scales_of_every_byte(bits):
    K = 32 * 256
    x = torch.zeros(3, K, dtype=torch.bfloat16, device="cuda")
    x[0, ::32], x[1, 5::32], x[2, :32 * 40] = 1.0, -2.0 ** -9, 2.0 ** 100
    codes = {4: torch.full((2, K // 2), 0x12, dtype=torch.uint8), 8: torch.full((2, K), 0x38, dtype=torch.uint8)}[bits].cuda()
    for lo, hi in ((0, 200), (30, 227)):  # up to sums that stay finite
        e8 = torch.zeros(2, 256, dtype=torch.uint8, device="cuda")
        e8[:, lo:hi] = torch.arange(lo, hi, dtype=torch.uint8, device="cuda")
        w = L.Mx4Weights(codes, e8) if bits == 4 else L.MxExpertWeights(codes, e8, None, None)
        check(L.mx_linear_few(x, w), x, w, floor=K * 2.0 ** -140)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [3, 12, 32])
def test_nan_and_infinity_stay_in_their_rows_and_columns(M, bits):
    x, w = inputs(M, 75, 608, bits)
    want = L.mx_linear_few(x, w)
    x[1, 77], x[2, 300] = float("nan"), float("inf")
    y = L.mx_linear_few(x, w)
    assert bool(torch.isnan(y[[1, 2]]).all())
    rest = [t for t in range(M) if t not in (1, 2)]
    assert torch.equal(y[rest], want[rest])
    e8 = L._held(w)[1]
    e8[20, 3] = 255
    y = L.mx_linear_few(x, w)
    assert bool(torch.isnan(y[:, 20]).all())
    others = [n for n in range(75) if n != 20]
    assert torch.equal(y[rest][:, others], want[rest][:, others])


def test_e4m3_nan_code():
    x, w = inputs(2, 40, 128, 8)
    w.q_row[7, 100] = 0x7F
    w.q_row[9, 1] = 0xFF
    y = L.mx_linear_few(x, w)
    assert torch.isnan(y).any(dim=0).nonzero().ravel().tolist() == [7, 9] and bool(torch.isnan(y[:, [7, 9]]).all())


def test_zero_tokens_give_zero():
    x, w = inputs(4, 50, 96, 4)
    assert not L.mx_linear_few(torch.zeros_like(x), w).any()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M,N,K", [(1, 300, 2048), (7, 2048, 2048), (32, 513, 1600)])
def test_calls_repeat_bit_for_bit_on_two_streams_at_once(M, N, K, bits):
    x, w = inputs(M, N, K, bits)
    want = L.mx_linear_few(x, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(L.mx_linear_few(x, w))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("M,N,K", [(2, 33, 96), (32, 70, 1056)])
def test_nothing_is_written_behind_the_result(M, N, K):
    x, w = inputs(M, N, K, 4)
    buf = torch.full((M * N + 512,), 3.0, dtype=torch.bfloat16, device="cuda")
    n = FB.mx_few_linear_workspace_bytes(M, N, K)
    for fill in (0x00, 0xFF):  # whatever was in the workspace before
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device="cuda")
        FB.mx_few_linear(x, w.q, w.e8, 4, buf[:M * N].view(M, N), ws[:n] if n else None)
        assert bool((buf[M * N:] == 3.0).all()) and bool((ws[n:] == fill).all())
        check(buf[:M * N].view(M, N), x, w)


def test_captured_and_replayed_with_new_tokens():
    x, w = inputs(5, 400, 1024, 4)
    L.mx_linear_few(x, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = L.mx_linear_few(x, w)
    for seed in (1, 2):
        x.copy_(inputs(5, 400, 1024, 4, seed)[0])
        g.replay()
        torch.cuda.synchronize()
        check(y, x, w)


def test_on_a_stream_of_its_own():
    """The result and the workspace are the stream's: what the current stream allocates meanwhile is other memory."""
    cases = [inputs(M, 3000, 4096, 4) for M in (1, 9, 32)]
    want = [L.mx_linear_few(x, w) for x, w in cases]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        for (x, w), expected in zip(cases, want):
            got, junk = [], []
            for _ in range(20):
                got.append(L.mx_linear_few(x, w, stream=stream))
                junk.append(torch.full((1 << 16,), 7.0, device="cuda"))
                junk = junk[-2:]
            torch.cuda.synchronize()
            assert all(torch.equal(g, expected) for g in got)
    w = torch.randn(96, 160, device="cuda").bfloat16()
    torch.cuda.synchronize()
    q = L.mx4_quantize(w, stream=side)
    wide = L.mx4_widen(q, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(q.q, L.mx4_quantize(w).q) and torch.equal(wide.q_row, L.mx4_widen(q).q_row)


@pytest.mark.parametrize("M,N,K", [(1, 140, 256), (4, 300, 1024), (32, 70, 640)])
def test_codes_at_every_16th_byte(M, N, K):
    """Rows of whole chunks whose codes start 16 bytes past what TMA spreads out."""
    x, w = inputs(M, N, K, 4)
    room = torch.empty(w.q.numel() + 64, dtype=torch.uint8, device="cuda")
    want = L.mx_linear_few(x, w)
    for at in (0, 16, 32, 48):
        q = room[at:at + w.q.numel()].view(w.q.shape)
        q.copy_(w.q)
        got = L.mx_linear_few(x, L.Mx4Weights(q, w.e8))
        check(got, x, w)
        assert torch.equal(got, want)
    with pytest.raises(B.Fp8bwError):
        L.mx_linear_few(x, L.Mx4Weights(room[8:8 + w.q.numel()].view(w.q.shape), w.e8))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M,N,K", [(1, 500, 12320), (2, 200, 16352), (2, 130, 4064), (1, 129, 32), (1, 4608, 12288), (2, 4500, 12256),
                                   (2, 4609, 12288), (1, 640, 7680), (2, 1000, 10752), (1, 36865, 128), (1, 36864, 1536)])
def test_one_or_two_tokens(M, N, K, bits):
    """Around the lengths and heights up to which the product brings the tokens into parts itself."""
    x, w = inputs(M, N, K, bits)
    check(L.mx_linear_few(x, w), x, w)


@pytest.mark.parametrize("Ms", [(1, 1, 1, 1), (2, 3, 2, 9), (32, 32, 1, 32), (17, 1, 5, 2)])
def test_one_behind_the_other(Ms):
    """Each call reads what the one before wrote, and weights and tokens are written over right after a call: a kernel starts
    under the one before, and none may read or write too early."""
    rng = np.random.default_rng(3)
    weights = [[held(torch.from_numpy((0.05 * rng.standard_normal((512, 512))).astype(np.float32)).bfloat16().cuda(), bits)
                for bits in (4, 8)] for _ in range(2)]
    x0 = torch.from_numpy(rng.standard_normal((32, 512)).astype(np.float32)).bfloat16().cuda()

    def walk(wait):
        x, out = x0.clone(), []
        w = [L.Mx4Weights(weights[0][0].q.clone(), weights[0][0].e8.clone()), weights[0][1]]
        for step in range(12):
            M = Ms[step % len(Ms)]
            y = L.mx_linear_few(x[:M], w[step % 2])
            wait()
            x[:M].copy_(y)
            wait()
            w[0].q.copy_(weights[(step + 1) % 2][0].q), w[0].e8.copy_(weights[(step + 1) % 2][0].e8)
            wait()
            if step % 3 == 2:  # codes written by a kernel right before they are read
                w[0] = L.mx4_quantize((x[:, :, None].expand(32, 512, 16).permute(0, 2, 1).reshape(512, 512) * 0.05).contiguous())
                wait()
            out.append(y.clone())
            wait()
        return out

    want = walk(torch.cuda.synchronize)
    for _ in range(5):
        got = walk(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_refusals_on_the_device():
    x, w = inputs(4, 50, 96, 4)
    for bad, error in ((x.t().contiguous().t(), ValueError), (x.float(), TypeError), (x[:, :64], ValueError),
                       (x[:, :64].contiguous(), ValueError), (torch.cat([x] * 9), B.Fp8bwError)):
        with pytest.raises(error):
            L.mx_linear_few(bad, w)
    two = L.Mx4Weights(torch.stack([w.q] * 2), torch.cat([w.e8] * 2))
    with pytest.raises(ValueError):
        L.mx_linear_few(x, two)
    one = L.Mx4Weights(w.q[None], w.e8)
    assert torch.equal(L.mx_linear_few(x, one), L.mx_linear_few(x, w))


def test_past_2_to_the_31_bytes():
    N, K = 65664, 65536  # 2^32 weights and more in 4 bits
    x = torch.randn(2, K, device="cuda").bfloat16()
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda")
    e8 = torch.randint(118, 123, (N, K // 32), dtype=torch.uint8, device="cuda")
    y = L.mx_linear_few(x, L.Mx4Weights(q, e8))
    rows = [0, 1, 32767, 32768, 65535, 65536, N - 1]
    check(y[:, rows], x, L.Mx4Weights(q[rows], e8[rows]))
