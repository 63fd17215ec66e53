"""The mixture-of-experts layer for a few tokens, against the formulas in 64 bits (oracle.few has its error bound)."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from gpu_util import f32, u8
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L
from mxfp8_precision_gemms_fp8bw_gb300 import moe
from oracle import few as OF
from oracle.moe import moe_keys, moe_route

pytestmark = pytest.mark.gpu
BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(autouse=True)
def built():
    B.lib(build_if_missing=True)


def values(w, shape):
    q, e8, bits = L._held(w)
    return OF.mx_weight(u8(q).reshape(shape[0] * shape[1], -1), u8(e8), bits).reshape(shape)


def clear_choice(rng, M, C, router, bias, top_k, how):
    """Tokens whose choice no fp32 rounding can change: other experts are chosen neither with keys moved by 1e-4 up or down."""
    x = np.empty((M, C), np.float32)
    t = 0
    while t < M:
        row = torch.from_numpy(rng.standard_normal((1, C)).astype(np.float32)).bfloat16().float().numpy()
        logits = row.astype(np.float64) @ router.astype(np.float64).T
        first = moe_route(logits, top_k, bias=bias, **how)[0]
        near = [moe_route(logits + 1e-4 * rng.standard_normal(logits.shape), top_k, bias=bias, **how)[0] for _ in range(8)]
        if all(np.array_equal(np.sort(first), np.sort(n)) for n in near):
            x[t] = row
            t += 1
    return x


class Case:
    def __init__(self, M, E, k, C, F, bits, bias=None, seed=0, **how):
        self.M, self.E, self.k, self.C, self.F, self.bits, self.how = M, E, k, C, F, bits, how
        rng = np.random.default_rng(seed + 3 * M + 5 * E + 7 * k + 11 * C + 13 * F + bits)
        self.router = (1.5 / np.sqrt(C) * rng.standard_normal((E, C))).astype(np.float32)
        self.bias = None if bias is None else np.round(rng.standard_normal(E) * 20).astype(np.float32) * np.float32(1e-3)
        if bias == "off":
            self.bias[rng.permutation(E)[:max(1, E // 3)]] = -np.inf
        self.x = clear_choice(rng, M, C, self.router, self.bias, k, how)
        dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        self.tx, self.trouter, self.tbias = dev(self.x).bfloat16(), dev(self.router), dev(self.bias)
        w = [torch.from_numpy((0.05 * rng.standard_normal(s)).astype(np.float32)).bfloat16().cuda()
             for s in ((E, 2 * F, C), (E, C, F))]
        make = L.mx4_quantize if bits == 4 else lambda t: L.mx_quantize_experts(t, colwise=False)
        self.w13, self.w2 = make(w[0]), make(w[1])

    def run(self, x=None, **other):
        x = self.tx if x is None else x
        return moe.ffn_few(x, self.trouter, self.w13, self.w2, self.k, bias=self.tbias, **{**self.how, **other})

    def want(self):
        return OF.few_layer(self.x, self.router, values(self.w13, (self.E, 2 * self.F, self.C)),
                            values(self.w2, (self.E, self.C, self.F)), self.k, bias=self.bias, **self.how)

    def check(self, y, rows=slice(None)):
        want, bound, _ = self.want()
        off = np.abs(f32(y) - want)[rows]
        most = (1.01 * bound + BF16 * (np.abs(want) + bound) + 1e-37)[rows]
        assert (off <= most).all(), float((off / most).max())
        norm = np.linalg.norm(want[rows])  # and as a whole, one rounding of bf16
        assert np.linalg.norm(off) <= BF16 * norm + 1e-37


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M,E,k,C,F", [
    (1, 1, 1, 32, 32), (1, 8, 2, 64, 96), (1, 64, 4, 256, 160), (2, 5, 5, 96, 64), (3, 12, 3, 416, 224), (7, 64, 8, 160, 96),
    (8, 8, 2, 512, 256), (9, 8, 1, 96, 544), (16, 4, 4, 128, 64), (17, 64, 4, 256, 128), (31, 9, 2, 64, 1056), (32, 8, 2, 256, 512),
    (32, 1, 1, 64, 64), (32, 128, 8, 64, 32), (32, 3, 3, 32, 32),
])
def test_against_64_bits(M, E, k, C, F, bits):
    c = Case(M, E, k, C, F, bits)
    c.check(c.run())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M,E,k,C,F", [(16, 32, 4, 128, 1056), (32, 32, 4, 96, 1056), (27, 48, 2, 160, 704), (17, 16, 4, 384, 2048)])
def test_more_tiles_than_blocks(M, E, k, C, F, bits):
    """Enough experts and rows for blocks to take one tile after the other."""
    c = Case(M, E, k, C, F, bits)
    c.check(c.run())


def test_as_many_choices_as_there_may_be():
    c = Case(32, 1024, 32, 32, 32, 4, score="sigmoid")
    c.check(c.run())


@pytest.mark.parametrize("M", [1, 3, 9, 32])
def test_choice_by_the_router_s_last_bit(M):
    """Experts whose logits differ by one unit in the last place of fp32: tokens with one element other than zero."""
    E, C, F = 40, 96, 32
    c = Case(M, E, 1, C, F, 4)
    rng = np.random.default_rng(M)
    router = np.ones((E, C), np.float32)
    best = rng.integers(0, E, C)
    router[best, np.arange(C)] = 1 + np.float32(2.0 ** -23)
    x = np.zeros((M, C), np.float32)
    at = rng.integers(0, C, M)
    x[np.arange(M), at] = 1.0
    c.x, c.router = x, router
    c.tx, c.trouter = torch.from_numpy(x).bfloat16().cuda(), torch.from_numpy(router).cuda()
    assert (c.want()[2][:, 0] == best[at]).all()
    c.check(c.run(renormalize=True))


@pytest.mark.parametrize("M", range(1, 33))
def test_every_token_count(M):
    c = Case(M, 6, 2, 96, 128, 4 if M % 2 else 8)
    c.check(c.run())


@pytest.mark.parametrize("how", [
    dict(score="sigmoid"), dict(score="sigmoid", renormalize=False, scale=2.5), dict(renormalize=False),
    dict(groups=4, groups_kept=2), dict(groups=4, groups_kept=1, group_top=2, score="sigmoid"),
    dict(groups=8, groups_kept=3, group_top=2, scale=0.5),
])
@pytest.mark.parametrize("bias", [None, "on", "off"])
@pytest.mark.parametrize("M,E", [(1, 32), (11, 32), (20, 64)])
def test_ways_of_choosing(M, E, bias, how):
    c = Case(M, E, 3, 128, 96, 4, bias=bias, **how)
    c.check(c.run())


@pytest.mark.parametrize("M", [1, 4, 18])
def test_more_choices_than_experts_left(M):
    """Five experts of eight are off: the fourth choice has no expert."""
    c = Case(M, 8, 3, 64, 64, 4)
    bias = np.zeros(8, np.float32)
    bias[[0, 1, 2, 4, 5, 6]] = -np.inf
    c.bias, c.tbias = bias, torch.from_numpy(bias).cuda()
    c.check(c.run())
    assert (c.want()[2] == -1).any()


@pytest.mark.parametrize("M", [1, 6, 32])
def test_no_expert_left_gives_zero(M):
    c = Case(M, 8, 2, 64, 64, 8)
    y = moe.ffn_few(c.tx, c.trouter, c.w13, c.w2, 2, bias=torch.full((8,), float("-inf"), device="cuda"))
    assert y.shape == (M, 64) and not y.any()


@pytest.mark.parametrize("E,k,top", [(1024, 32, 1), (300, 10, 1), (513, 7, 1), (256, 32, 2)])
def test_many_experts_and_choices(E, k, top):
    c = Case(5, E, k, 64, 32, 4, groups=1 if top == 1 else 8, groups_kept=1 if top == 1 else 4, group_top=top)
    c.check(c.run())


def test_all_tokens_choose_the_same_experts():
    c = Case(32, 16, 2, 128, 96, 4)
    bias = np.zeros(16, np.float32)
    bias[[3, 9]] = 5.0
    c.bias, c.tbias = bias, torch.from_numpy(bias).cuda()
    assert set(np.unique(c.want()[2])) == {3, 9}
    c.check(c.run())


@pytest.mark.parametrize("M", [3, 14])
def test_nan_and_infinity_stay_in_their_tokens(M):
    c = Case(M, 8, 2, 96, 64, 4)
    x = c.tx.clone()
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    y = c.run(x)
    assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[2]).all())
    c.check(y, rows=[t for t in range(M) if t not in (1, 2)])


@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** 30])
def test_tokens_far_from_one(size):
    c = Case(4, 4, 2, 64, 64, 8)
    c.x = (c.x * np.float32(size)).astype(np.float32)
    c.router = (c.router / np.float32(size)).astype(np.float32)
    c.tx, c.trouter = torch.from_numpy(c.x).bfloat16().cuda(), torch.from_numpy(c.router).cuda()
    c.check(c.run())


@pytest.mark.parametrize("M", [1, 8, 32])
def test_calls_repeat_bit_for_bit_on_two_streams_at_once(M):
    c = Case(M, 16, 4, 256, 160, 4)
    want = c.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(8):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(c.run())
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("Ms", [(1, 1, 1), (5, 1, 32), (32, 17, 2)])
def test_one_behind_the_other(Ms):
    """Layers and linears that read what the call before wrote, none waited for, as a decoder's step runs them."""
    c = [Case(M, 16, 4, 256, F, bits) for M, F, bits in zip((4, 4, 4), (160, 512, 1056), (4, 8, 4))]
    x0 = Case(32, 16, 4, 256, 32, 4).tx
    proj = L.mx4_quantize((torch.randn(256, 256, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) * 0.06).bfloat16())

    def walk(wait):
        x, out = x0.clone(), []
        for step in range(12):
            M, case = Ms[step % len(Ms)], c[step % 3]
            h = L.mx_linear_few(x[:M], proj)
            wait()
            y = case.run(h)
            wait()
            z = case.run(y)  # right behind, with a workspace that may be the same memory
            wait()
            x[:M].copy_(z / z.float().norm(dim=1, keepdim=True).clamp_min(1e-3) * 16)
            wait()
            out += [h.clone(), y.clone(), z.clone()]
            wait()
        return out

    want = walk(torch.cuda.synchronize)
    assert all(bool(torch.isfinite(w).all()) for w in want) and bool(want[-1].any())
    for _ in range(5):
        got = walk(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_tokens_one_at_a_time():
    c = Case(8, 16, 4, 256, 160, 4)
    c.check(torch.cat([c.run(c.tx[t:t + 1]) for t in range(8)]))


def test_captured_in_two_graphs_and_replayed_with_new_tokens():
    c, d = Case(3, 8, 2, 128, 96, 4), Case(19, 8, 2, 128, 96, 8)
    c.run(), d.run()
    torch.cuda.synchronize()
    graphs = []
    for case in (c, d):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = case.run()
        graphs.append((g, y))
    new = [Case(c.M, 8, 2, 128, 96, 4, seed=100), Case(d.M, 8, 2, 128, 96, 8, seed=100)]
    side = torch.cuda.Stream()
    for _ in range(3):
        for case in (c, d):
            case.tx.copy_(torch.from_numpy(case.x).cuda())
        torch.cuda.synchronize()
        graphs[0][0].replay()
        with torch.cuda.stream(side):  # both at once
            graphs[1][0].replay()
        torch.cuda.synchronize()
        c.check(graphs[0][1])
        d.check(graphs[1][1])
    for case, n, (g, y) in zip((c, d), new, graphs):
        want = moe.ffn_few(n.tx, case.trouter, case.w13, case.w2, 2)
        case.tx.copy_(n.tx)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_threads_with_streams_of_their_own():
    cases = [Case(M, 16, 4, 256, 160, bits) for M, bits in ((1, 4), (9, 8), (32, 4), (2, 8))]
    proj = [L.mx4_quantize((torch.randn(300, 256, device="cuda") * 0.06).bfloat16()) for _ in cases]
    want = [(c.run(), L.mx_linear_few(c.tx, w)) for c, w in zip(cases, proj)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                got = (cases[i].run(), L.mx_linear_few(cases[i].tx, proj[i]))
            torch.cuda.current_stream().synchronize()
        if not all(torch.equal(g, w) for g, w in zip(got, want[i])):
            wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    [t.start() for t in threads], [t.join() for t in threads]
    assert wrong == []


FIRST_CALL = """
import sys, torch
sys.path.insert(0, {root!r})
from mxfp8_precision_gemms_fp8bw_gb300 import linear as L, moe
g = torch.Generator("cuda").manual_seed(2)
new = lambda *s: (torch.randn(s, device="cuda", generator=g) * 0.1).bfloat16()
x, r, w = new(5, 256), new(8, 256).float(), [new(8, 256, 256), new(8, 256, 128), new(300, 256)]
w13, w2, w1 = map(L.mx4_quantize, w)  # the library's first call is eager; the products' first ones are captured
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
def step():
    return moe.ffn_few(x, r, w13, w2, 2), L.mx_linear_few(x, w1), L.mx_linear_few(x[:1], w1)
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step())), "captured and eager differ"
"""


def test_first_call_under_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=root)], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_rows_behind_the_result_and_the_workspace_stay():
    from mxfp8_precision_gemms_fp8bw_gb300 import few_binding as FB
    c = Case(5, 8, 2, 96, 64, 4)
    want = c.run()
    y = torch.full((7, 96), 3.0, dtype=torch.bfloat16, device="cuda")
    n = FB.mx_few_moe_workspace_bytes(5, 8, 2, 96, 64)
    for fill in (0x00, 0xFF, 0x7F):  # whatever was there before
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device="cuda")
        FB.mx_few_moe(c.tx, c.trouter, None, c.w13.q, c.w13.e8, c.w2.q, c.w2.e8, 4, 2, y[:5], ws[:n])
        torch.cuda.synchronize()
        assert torch.equal(y[:5], want) and bool((y[5:] == 3.0).all()) and bool((ws[n:] == fill).all())


def test_refusals_on_the_device():
    c = Case(4, 8, 2, 96, 64, 4)
    with pytest.raises(ValueError, match="contiguous"):
        c.run(c.tx.t().contiguous().t())
    with pytest.raises(TypeError):
        c.run(c.tx.float())
    with pytest.raises(ValueError, match="router"):
        moe.ffn_few(c.tx, c.trouter[:4], c.w13, c.w2, 2)
    with pytest.raises(ValueError, match="w2"):
        moe.ffn_few(c.tx, c.trouter, c.w13, L.Mx4Weights(c.w2.q[:4], c.w2.e8), 2)
    with pytest.raises(B.Fp8bwError):
        c.run(torch.cat([c.tx] * 9))
    with pytest.raises(B.Fp8bwError):
        c.run(groups=3)
    with pytest.raises(ValueError, match="score"):
        c.run(score="tanh")


# ------------------------------------------------------------------ through the layer

def layer_of(dim=256, hidden=512, E=8, k=2, **how):
    torch.manual_seed(5)
    return moe.MxMoEFFN(dim, hidden, E, k, device="cuda", **how)


@pytest.mark.parametrize("bits", [4, 8])
def test_prompt_then_tokens(bits):
    """As a decoder runs: a prompt through forward, then tokens one by one and in batches through decode, same codes."""
    layer = layer_of(score="sigmoid", groups=4, groups_kept=2, group_top=2)
    rng = np.random.default_rng(9)
    how = dict(score="sigmoid", groups=4, groups_kept=2, group_top=2)
    x = clear_choice(rng, 40, 256, f32(layer.router), np.zeros(8, np.float32), 2, how)
    tx = torch.from_numpy(x).bfloat16().cuda()
    codes = layer.weight_codes(colwise=False, bits=bits)
    w13, w2 = values(codes[0], (8, 1024, 256)), values(codes[1], (8, 256, 512))
    want, bound, _ = OF.few_layer(x, f32(layer.router), w13, w2, 2, bias=np.zeros(8, np.float32), **how)
    with torch.no_grad():
        prompt = layer(tx, codes)
        together = layer.decode(tx[:32], codes)
        alone = torch.cat([layer.decode(tx[i:i + 1], codes) for i in range(4)])
    for got, ref, b in ((together, want[:32], bound[:32]), (alone, want[:4], bound[:4])):
        assert (np.abs(f32(got) - ref) <= 1.01 * b + BF16 * (np.abs(ref) + b)).all()
    # forward rounds tokens and then activations to e4m3, at most 2^-4 of each element: the same layer, a few percent off
    assert np.linalg.norm(f32(prompt) - want) <= 2.0 ** -3 * np.linalg.norm(want)
    assert together.grad_fn is None


def test_four_bit_codes_through_forward_equal_their_widened_ones():
    layer = layer_of()
    codes = layer.weight_codes(bits=4)
    x = torch.randn(70, 256, device="cuda").bfloat16()
    with torch.no_grad():
        assert torch.equal(layer(x, codes), layer(x, tuple(L.mx4_widen(c) for c in codes)))


def test_decode_leaves_the_layer_as_it_was():
    layer = layer_of()
    layer.train()
    x = torch.randn(9, 256, device="cuda").bfloat16()
    layer(x)
    counts = layer.counts.clone()
    layer.decode(x[:3], layer.weight_codes(bits=4))
    assert torch.equal(layer.counts, counts)
    layer.update_balance()
    assert layer.decode(x[:0], layer.weight_codes()).shape == (0, 256)
    with pytest.raises(B.Fp8bwError, match="32"):
        layer.decode(torch.cat([x] * 4), layer.weight_codes())


def test_balance_shifts_the_choice():
    layer = layer_of()
    codes = layer.weight_codes(bits=8)
    x = torch.randn(4, 256, device="cuda").bfloat16()
    before = layer.decode(x, codes)
    layer.balance[:4] = -float("inf")
    after = layer.decode(x, codes)
    keys = moe_keys(f32(x).astype(np.float64) @ f32(layer.router).astype(np.float64).T, "softmax", f32(layer.balance))
    assert (keys[:, :4] == -np.inf).all() and not torch.equal(before, after)
