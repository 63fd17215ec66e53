"""GPU parity of dispatch (gather + MX codes), combine and their gradients."""
import numpy as np
import pytest
import torch

from gpu_util import adversarial_bf16, f32, lib, u8
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import moe
from mxfp8_precision_gemms_fp8bw_gb300 import moe_binding as MB
from oracle import moe as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = 2.0 ** -8      # bf16 rounds within half a unit of its 8th significant bit


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


def setup(M, E, k, seed, dropped=0.0):
    r = np.random.default_rng(seed)
    ex = np.argsort(r.standard_normal((M, E)) + r.standard_normal(E), axis=1)[:, :k].astype(np.int32)
    ex[r.uniform(size=(M, k)) < dropped] = -1
    p = moe.plan(torch.from_numpy(np.ascontiguousarray(ex)).cuda(), E)
    w = torch.from_numpy(r.uniform(0.05, 1.0, size=(M, k)).astype(np.float32)).cuda()
    return r, p, w


def normal(r, *shape, std=1.0):
    return torch.from_numpy((r.standard_normal(shape) * std).astype(np.float32)).bfloat16().cuda()


def same_codes(got, want):
    for a, b in zip((got.q, got.e8, got.qT, got.e8T), want):
        if a is not None:
            assert np.array_equal(u8(a), b)


SHAPES = [(1, 1, 1, 32), (1, 8, 2, 96), (17, 64, 4, 160), (100, 4, 3, 32), (130, 8, 2, 256), (65, 3, 2, 416), (300, 16, 4, 64),
          (257, 5, 5, 1056)]


@pytest.mark.parametrize("mode", [B.MX_RCEIL, B.MX_FLOOR])
@pytest.mark.parametrize("M,E,k,C", SHAPES)
def test_dispatch_is_bit_exact(M, E, k, C, mode):
    r, p, w = setup(M, E, k, seed=M + C, dropped=0.1)
    x = adversarial_bf16(M, C, seed=C, block=32).cuda()
    got = moe.dispatch(x, p, mode=mode)
    B.fp8bw_sync_status()
    same_codes(got, O.moe_gather_quant(f32(x), u8(p.src_of), k, mode=mode))
    rows = moe.dispatch(x, p, colwise=False, mode=mode)
    assert rows.qT is None and torch.equal(rows.q, got.q) and torch.equal(rows.e8, got.e8)


@pytest.mark.parametrize("mode", [B.MX_RCEIL, B.MX_FLOOR])
@pytest.mark.parametrize("M,E,k,C", SHAPES)
def test_combine_backward(M, E, k, C, mode):
    r, p, w = setup(M, E, k, seed=M + C, dropped=0.1)
    dout, y = adversarial_bf16(M, C, seed=C + 1, block=32).cuda(), normal(r, p.rows, C)
    w[0, 0] = 0.0
    dy, dw = moe.combine_backward(dout, y, w, p, mode=mode)
    B.fp8bw_sync_status()
    # one fp32 product and the codes of it: exact
    same_codes(dy, O.moe_gather_quant(f32(dout), u8(p.src_of), k, w.cpu().numpy(), mode=mode))
    a, b, row = np.abs(f32(dout)).astype(np.float64), np.abs(f32(y)).astype(np.float64), u8(p.row_of)
    # an fp32 sum of C products in any order
    bound = C * U * O.moe_combine_dweights(a, b, row)
    assert np.all(np.abs(dw.cpu().numpy() - O.moe_combine_dweights(f32(dout), f32(y), row)) <= bound)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("based", [False, True])
@pytest.mark.parametrize("M,E,k,C", SHAPES + [(33, 40, 32, 8), (40, 8, 8, 24), (1000, 8, 2, 72)])
def test_combine(M, E, k, C, weighted, based):
    r, p, w = setup(M, E, k, seed=M + C, dropped=0.2)
    y, base = normal(r, p.rows, C), normal(r, M, C) if based else None
    wn = w.cpu().numpy() if weighted else None
    out = moe.combine(y, w if weighted else None, p, base)
    B.fp8bw_sync_status()
    ref = O.moe_combine(f32(y), u8(p.row_of), wn, f32(base) if based else None)
    size = O.moe_combine(np.abs(f32(y)), u8(p.row_of), wn, np.abs(f32(base)) if based else None)
    assert np.all(np.abs(f32(out) - ref) <= BF * np.abs(ref) + (k + 2) * U * size * (1 + BF))
    if based:   # base may be the output itself
        MB.fp8bw_moe_combine(y, w if weighted else None, p.row_of, base, base)
        assert torch.equal(base, out)


def test_rows_without_entries_do_not_reach_the_tokens():
    """NaN and infinity in rows and weights that no token has: combine and the weights' gradient do not touch them."""
    r, p, w = setup(50, 8, 2, seed=9, dropped=0.3)
    y, dout = normal(r, p.rows, 64), normal(r, 50, 64)
    out = moe.combine(y, w, p)
    dw = moe.combine_backward(dout, y, w, p)[1]
    y[p.src_of < 0] = float("nan")
    w2 = w.clone()
    w2[p.row_of < 0] = float("inf")
    assert torch.equal(moe.combine(y, w2, p), out)
    dy, dw2 = moe.combine_backward(dout, y, w2, p)
    assert torch.equal(dw2, dw) and torch.all(dw[p.row_of < 0] == 0)
    same_codes(dy, O.moe_gather_quant(f32(dout), u8(p.src_of), 2, w.cpu().numpy()))
    B.fp8bw_sync_status()


def test_nan_and_infinity_stay_visible_in_the_codes():
    r, p, _ = setup(40, 2, 1, seed=1)
    x = normal(r, 40, 64)
    x[3, 5], x[7, 40] = float("nan"), float("inf")
    q = moe.dispatch(x, p)
    B.fp8bw_sync_status()
    row3, row7 = int(p.row_of[3, 0]), int(p.row_of[7, 0])
    assert int(q.q[row3, 5]) & 0x7F == 0x7F and int(q.e8[row3, 0]) == 247
    assert int(q.qT[5, row3]) & 0x7F == 0x7F
    assert int(q.q[row7, 40]) == 0x7E and int(q.e8[row7, 1]) == 247     # saturated, largest scale
    clean = x.clone()
    clean[3, :32], clean[7, 32:] = 0, 0
    other = moe.dispatch(clean, p)
    keep = torch.ones_like(q.q, dtype=torch.bool)
    keep[row3, :32] = keep[row7, 32:] = False
    assert torch.equal(q.q[keep], other.q[keep])


def test_indices_out_of_range_are_skipped_and_reported():
    r, p, w = setup(60, 4, 2, seed=5)
    x, y = normal(r, 60, 96), normal(r, p.rows, 96)
    bad = moe.Plan(p.group_end, p.counts, p.row_of.clone(), p.src_of.clone())
    row, src = int(p.row_of[10, 1]), int(p.src_of[0])
    bad.row_of[10, 1], bad.src_of[0] = p.rows, 120
    good = moe.Plan(p.group_end, p.counts, p.row_of.clone(), p.src_of.clone())
    good.row_of[10, 1], good.src_of[0] = -1, -1
    B.fp8bw_sync_status()
    for call in (lambda q: moe.dispatch(x, q).q, lambda q: moe.combine(y, w, q),
                 lambda q: moe.combine_backward(x, y, w, q)[1]):
        got = call(bad)
        with pytest.raises(B.Fp8bwError) as e:
            B.fp8bw_sync_status()
        assert e.value.code == B.ERR_SHAPE
        assert torch.equal(got, call(good))
    B.fp8bw_sync_status()
    assert row >= 0 and src >= 0


@pytest.mark.parametrize("M,k,C", [(8200, 1, 256), (9001, 2, 544)])
def test_many_rows(M, k, C):
    """More tiles than the GPU holds at once; codes against the framework's own quantizers of gathered rows."""
    r, p, w = setup(M, 8, k, seed=M)
    x = torch.randn(M, C, device="cuda").bfloat16()
    got = moe.dispatch(x, p)
    rows = torch.where((p.src_of >= 0)[:, None], x[p.src_of.clamp(min=0).long() // k], 0)
    q, e8 = B.alloc_mx_row(rows)
    B.mxfp8_quant_1x32_row(rows, q, e8)
    qT, e8T = B.alloc_mx_col(rows)
    B.mxfp8_quant_1x32_col(rows, qT, e8T)
    B.fp8bw_sync_status()
    for a, b in zip((got.q, got.e8, got.qT, got.e8T), (q, e8, qT, e8T)):
        assert torch.equal(a, b)
    y = torch.randn(p.rows, C, device="cuda").bfloat16()
    picked = y[p.row_of.clamp(min=0).long()].double()
    ref = (picked * w[..., None].double()).sum(1)
    size = (picked.abs() * w[..., None].double()).sum(1)
    assert bool(((moe.combine(y, w, p).double() - ref).abs() <= BF * ref.abs() + (k + 2) * U * size * (1 + BF)).all())
    dw = moe.combine_backward(x, y, w, p)[1].double()
    prod = picked * x[:, None].double()
    assert bool(((dw - prod.sum(2)).abs() <= C * U * prod.abs().sum(2)).all())


def test_past_2_to_the_31_elements():
    """Rows whose flat offsets leave the int32 range, in the codes of both layouts and in the rows combined."""
    M, k, C = 1048960, 1, 2080
    x = torch.empty(M, C, dtype=torch.bfloat16, device="cuda").normal_()
    p = moe.plan(torch.zeros(M, 1, dtype=torch.int32, device="cuda"), 1)
    assert p.rows * C > 2 ** 31
    got = moe.dispatch(x, p)
    B.fp8bw_sync_status()
    last = x[-64:]
    lo = M - 64
    assert lo % 32 == 0 and torch.equal(p.row_of[-64:, 0].cpu(), torch.arange(lo, M, dtype=torch.int32))
    q, e8 = B.alloc_mx_row(last)
    B.mxfp8_quant_1x32_row(last.contiguous(), q, e8)
    qT, e8T = B.alloc_mx_col(last)
    B.mxfp8_quant_1x32_col(last.contiguous(), qT, e8T)
    assert torch.equal(got.q[lo:M], q) and torch.equal(got.e8[lo:M], e8)
    assert torch.equal(got.qT[:, lo:M], qT) and torch.equal(got.e8T[:, lo // 32:M // 32], e8T)
    out = moe.combine(x, None, p)
    assert torch.equal(out[-64:], last) and torch.equal(out[:64], x[:64])
    dw = moe.combine_backward(out, x, torch.ones(M, 1, device="cuda"), p)[1]
    ref = last.double().square().sum(1)
    assert bool(((dw[-64:, 0].double() - ref).abs() <= C * U * ref).all())


def test_calls_follow_their_stream_and_replay_in_graphs():
    r, p, w = setup(500, 8, 2, seed=4)
    x, y = normal(r, 500, 128), normal(r, p.rows, 128)
    ref = moe.dispatch(x, p), moe.combine(y, w, p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a, b = moe.dispatch(x, p), moe.combine(y, w, p)
    side.synchronize()
    assert torch.equal(a.qT, ref[0].qT) and torch.equal(b, ref[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c, d = moe.dispatch(x, p), moe.combine(y, w, p)
        dy, dw = moe.combine_backward(x, y, w, p)
    x.copy_(normal(r, 500, 128))
    g.replay()
    torch.cuda.synchronize()
    same_codes(c, O.moe_gather_quant(f32(x), u8(p.src_of), 2))
    same_codes(dy, O.moe_gather_quant(f32(x), u8(p.src_of), 2, w.cpu().numpy()))
    assert torch.equal(d, ref[1])


def test_first_call_of_a_thread():
    """A thread that has not used the GPU yet, as autograd's backward thread may be, on a stream it is handed."""
    import threading

    r, p, w = setup(200, 4, 2, seed=8)
    x = normal(r, 200, 160)
    ref = moe.dispatch(x, p)
    out, stream, errors = moe._mx_rows(p.rows, 160, x.device), torch.cuda.current_stream().cuda_stream, []

    def work():
        try:
            MB.mxfp8_moe_gather_quant(x, None, p.src_of, 2, out.q, out.e8, out.qT, out.e8T, stream=stream)
        except Exception as e:
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    B.fp8bw_sync_status()
    assert not errors and torch.equal(out.q, ref.q) and torch.equal(out.qT, ref.qT) and torch.equal(out.e8T, ref.e8T)


def test_outputs_stay_in_bounds():
    """Canaries on both sides of every output."""
    r, p, w = setup(45, 8, 2, seed=6)
    x, y = normal(r, 45, 96), normal(r, p.rows, 96)
    guards = []

    def guarded(shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        guards.append((raw, n))
        return raw[4096:4096 + n].view(dtype).view(shape)

    P = p.rows
    codes = lambda: [guarded(s, torch.uint8) for s in ((P, 96), (P, 3), (96, P), (96, P // 32))]  # noqa: E731
    MB.mxfp8_moe_gather_quant(x, None, p.src_of, 2, *codes())
    MB.mxfp8_moe_gather_quant(x, w, p.src_of, 2, *codes())
    MB.fp8bw_moe_combine(y, w, p.row_of, None, guarded((45, 96), torch.bfloat16))
    MB.fp8bw_moe_combine_dweights(x, y, p.row_of, guarded((45, 2), torch.float32))
    logits = torch.randn(45, 70, device="cuda")
    ex = guarded((45, 3), torch.int32)
    MB.fp8bw_moe_route(logits, None, 3, ex, guarded((45, 3), torch.float32))
    MB.fp8bw_moe_route_bwd(torch.ones(45, 3, device="cuda"), logits, ex, guarded((45, 70), torch.float32))
    n = MB.fp8bw_moe_plan_workspace_bytes(45, 70, 3)
    MB.fp8bw_moe_plan(ex, 70, guarded((70,), torch.int32), guarded((70,), torch.int32), guarded((45, 3), torch.int32),
                      guarded((MB.fp8bw_moe_plan_rows(45, 70, 3),), torch.int32), guarded((n,), torch.uint8))
    h = normal(r, 32, 192)
    hq, he = guarded((32, 192), torch.uint8), guarded((32, 6), torch.uint8)
    MB.mxfp8_swiglu(h, *[guarded(s, torch.uint8) for s in ((32, 96), (32, 3), (96, 32), (96, 1))], hq, he)
    MB.mxfp8_swiglu_bwd(normal(r, 32, 96), hq, he,
                        *[guarded(s, torch.uint8) for s in ((32, 192), (32, 6), (192, 32), (192, 1))])
    B.fp8bw_sync_status()
    for raw, n in guards:
        raw = raw.cpu().numpy()
        assert np.all(raw[:4096] == 0xA5) and np.all(raw[4096 + n:] == 0xA5)
