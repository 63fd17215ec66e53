"""GPU parity of routing, its gradient and the plan against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from gpu_util import lib
from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import moe
from mxfp8_precision_gemms_fp8bw_gb300 import moe_binding as MB
from oracle import moe as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NINF, LOWEST = -np.inf, float(np.finfo(np.float32).min)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


def coarse_logits(M, E, seed):
    """Logits on a grid of 1/8 in [-4, 4] (exact in bf16): equal ones tie exactly, different ones are far apart."""
    return np.random.default_rng(seed).integers(-32, 33, size=(M, E)).astype(np.float32) / 8


def coarse_bias(E, seed):
    return np.random.default_rng(seed + 1).integers(-40, 41, size=E).astype(np.float32) / 1000


def weight_bound(logits, k):
    """Relative error of a weight: exp of a rounded difference (|x| u, and 2 ulp of exp itself), a division, a sum by
    halves over at most 1024 (10 roundings), the sum of the chosen (k), the division by it and the scale; for both the
    score and the normaliser."""
    x = np.abs(logits[np.isfinite(logits) & (np.abs(logits) < 1e3)])
    return (2 * (2 * float(x.max(initial=0.0)) + 4 + 2 + 10) + k + 4) * U


def apart(logits, bias, score, groups, group_top):
    """The rows in which no two keys, and no two group scores, that differ are within the rounding of fp32 of each other."""
    s, keys = O.moe_scores(logits, score), O.moe_keys(logits, score, bias)
    best = np.sort(keys.reshape(len(keys), groups, -1), axis=2)[:, :, -group_top:].sum(axis=2)
    near = lambda v: (np.diff(np.sort(v, axis=1)) > 0) & (np.diff(np.sort(v, axis=1)) < 40 * U * (1 + s.max()))  # noqa: E731
    return logits[~(near(keys).any(axis=1) | near(best).any(axis=1))]


CASES = [
    # M, E, k, how
    (1, 1, 1, {}), (1, 64, 4, {}), (5, 8, 2, {}), (33, 8, 8, {}), (7, 3, 2, dict(score="sigmoid")),
    (130, 16, 3, dict(scale=2.5)), (65, 33, 5, {}), (9, 160, 6, dict(renormalize=False)),
    (257, 64, 8, dict(score="sigmoid", renormalize=False)), (11, 200, 32, {}), (3, 1024, 32, {}), (5, 777, 9, {}),
    (12, 512, 4, dict(score="sigmoid")),
    (40, 64, 6, dict(groups=8, groups_kept=3)), (40, 60, 4, dict(groups=4, groups_kept=2, group_top=2, score="sigmoid")),
    (16, 32, 2, dict(groups=32, groups_kept=5, group_top=2)), (10, 1024, 16, dict(groups=32, groups_kept=4, group_top=2)),
    (10, 12, 6, dict(groups=2, groups_kept=1, group_top=2, score="sigmoid")),
    (10, 12, 12, dict(groups=2, groups_kept=2, group_top=1)),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("M,E,k,how", CASES)
def test_route_and_gradient(M, E, k, how, dtype):
    logits = coarse_logits(M, E, seed=M + E)
    group_kw = {n: v for n, v in how.items() if n.startswith("group")}
    grad_kw = {n: v for n, v in how.items() if not n.startswith("group")}
    ref_e, ref_w = O.moe_route(logits, k, **how)
    x = torch.from_numpy(logits).to(dtype).cuda()
    experts, weights = moe.route(x, k, **grad_kw, **group_kw)
    B.fp8bw_sync_status()
    assert np.array_equal(experts.cpu().numpy(), ref_e)
    tol = weight_bound(logits, k)
    assert np.all(np.abs(weights.cpu().numpy() - ref_w) <= tol * ref_w)

    dw = np.random.default_rng(E).standard_normal((M, k)).astype(np.float32)
    dlogits = moe.route_backward(torch.from_numpy(dw).cuda(), x, experts, **grad_kw)
    B.fp8bw_sync_status()
    assert dlogits.dtype == dtype
    ref = O.moe_route_bwd(dw, logits, ref_e, **grad_kw)
    # every term is at most s_e (|ds_e| + sum |ds_i| s_i); each carries the relative error of a weight a few times over
    s = O.moe_scores(logits, grad_kw.get("score", "softmax"))
    c = np.take_along_axis(s, ref_e.astype(np.int64), axis=1)
    D = c.sum(axis=1, keepdims=True) if grad_kw.get("renormalize", True) else np.ones((M, 1))
    size = np.abs(dw) * grad_kw.get("scale", 1.0)
    size = size / D + (size * c).sum(axis=1, keepdims=True) / D ** 2
    full = np.zeros_like(s)
    np.put_along_axis(full, ref_e.astype(np.int64), size, axis=1)
    bound = 4 * (tol + 2 * k * U) * s * (full + (size * c).sum(axis=1, keepdims=True))
    out_u = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    assert np.all(np.abs(dlogits.float().cpu().numpy() - ref) <= bound + out_u * np.abs(ref) + 1e-40)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,k,groups,kept,top", [(50, 64, 6, 8, 3, 2), (50, 20, 4, 1, 1, 1), (20, 160, 8, 5, 2, 2)])
def test_route_with_bias(M, E, k, groups, kept, top, score):
    bias = coarse_bias(E, seed=7)
    logits = apart(coarse_logits(8 * M, E, seed=7), bias, score, groups, top)[:M]
    assert len(logits) == M
    how = dict(score=score, groups=groups, groups_kept=kept, group_top=top)
    ref_e, ref_w = O.moe_route(logits, k, bias=bias, **how)
    experts, weights = moe.route(torch.from_numpy(logits).cuda(), k, bias=torch.from_numpy(bias).cuda(), **how)
    B.fp8bw_sync_status()
    assert np.array_equal(experts.cpu().numpy(), ref_e)
    assert np.all(np.abs(weights.cpu().numpy() - ref_w) <= weight_bound(logits, k) * ref_w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(8, 1), (8, 4), (70, 1), (70, 7), (160, 5)])
def test_masked_rows(E, groups, score, dtype):
    """Rows with all, all but one, and half of the experts masked by -inf, and masks of the type's lowest value."""
    logits = coarse_logits(8, E, seed=E)
    lowest = float(torch.finfo(dtype).min)
    logits[0] = NINF
    logits[1] = NINF
    logits[1, E - 1] = 0.5
    logits[2, ::2] = NINF
    logits[3] = lowest
    logits[4, 1:] = lowest
    logits[5, : E // 2] = lowest
    logits[6] = NINF
    logits[6, : E // groups] = 1.0       # one whole group
    k = min(6, 2 * (E // groups))
    how = dict(score=score, groups=groups, groups_kept=min(2, groups), group_top=2 if groups > 1 else 1)
    ref_e, ref_w = O.moe_route(logits, k, **how)
    x = torch.from_numpy(logits).to(dtype).cuda()
    experts, weights = moe.route(x, k, **how)
    dw = torch.ones(8, k, device="cuda")
    dlogits = moe.route_backward(dw, x, experts, score=score)
    B.fp8bw_sync_status()
    assert np.array_equal(experts.cpu().numpy(), ref_e)
    assert np.all(experts[0].cpu().numpy() == -1) and np.all(weights[0].cpu().numpy() == 0)
    assert experts[1].cpu().tolist() == [E - 1] + [-1] * (k - 1)
    assert np.all(np.abs(weights.cpu().numpy() - ref_w) <= weight_bound(logits, k) * ref_w + 1e-30)
    d = dlogits.float().cpu().numpy()
    assert np.all(np.isfinite(d)) and np.all(d[0] == 0) and np.all(d[np.isneginf(logits)] == 0)


def test_bias_masks_and_lowest_biases():
    E, k = 16, 4
    logits = coarse_logits(6, E, seed=2)
    bias = np.zeros(E, np.float32)
    bias[::2] = NINF
    bias[1] = LOWEST
    for groups in (1, 4):
        how = dict(groups=groups, groups_kept=min(groups, 3), group_top=1 if groups == 1 else 2)
        ref_e, _ = O.moe_route(logits, k, bias=bias, **how)
        experts, _ = moe.route(torch.from_numpy(logits).cuda(), k, bias=torch.from_numpy(bias).cuda(), **how)
        B.fp8bw_sync_status()
        assert np.array_equal(experts.cpu().numpy(), ref_e)
        assert not np.any(experts.cpu().numpy() % 2 == 0)
    # two lowest biases overflow a group's sum: the group counts as the lowest, not as masked
    bias = np.full(4, LOWEST, np.float32)
    experts, _ = moe.route(torch.zeros(1, 4, device="cuda"), 2, bias=torch.from_numpy(bias).cuda(), groups=2,
                           groups_kept=1, group_top=2)
    assert experts.cpu().tolist() == [[0, 1]]


def test_nan_and_infinity_show_in_the_weights():
    x = torch.zeros(4, 8, device="cuda")
    x[0, 3] = float("nan")
    x[1, 3] = float("inf")
    x[2, 3] = float("nan")
    x[2, 5] = float("-inf")
    experts, weights = moe.route(x, 2, score="sigmoid")
    e, w = experts.cpu().numpy(), weights.cpu().numpy()
    assert e[0, 0] == 3 and np.isnan(w[0, 0]) and e[1, 0] == 3 and np.isfinite(w[1]).all() and e[2, 0] == 3
    experts, weights = moe.route(x, 2)
    w = weights.cpu().numpy()
    assert np.isnan(w[0]).all() and np.isnan(w[1]).all() and np.isnan(w[2]).all() and np.isfinite(w[3]).all()
    assert 5 not in experts.cpu().numpy()[2]
    B.fp8bw_sync_status()


def test_route_bwd_skips_and_reports_experts_out_of_range():
    x, dw = torch.randn(3, 8, device="cuda"), torch.ones(3, 2, device="cuda")
    experts, _ = moe.route(x, 2)
    good = moe.route_backward(dw, x, experts, renormalize=False)
    bad = experts.clone()
    bad[1, 1] = 8
    skipped = experts.clone()
    skipped[1, 1] = -1
    B.fp8bw_sync_status()
    got = moe.route_backward(dw, x, bad, renormalize=False)
    with pytest.raises(B.Fp8bwError) as e:
        B.fp8bw_sync_status()
    assert e.value.code == B.ERR_SHAPE
    want = moe.route_backward(dw, x, skipped, renormalize=False)
    assert torch.equal(got, want) and torch.equal(got[0], good[0])


# ------------------------------------------------------------------ plan

def check_plan(experts, E, P=None):
    ex = torch.from_numpy(experts).cuda()
    M, k = experts.shape
    if P is None:
        p = moe.plan(ex, E)
        P = p.rows
        assert P == MB.fp8bw_moe_plan_rows(M, E, k)
    else:
        i32 = lambda *s: torch.full(s, 7, dtype=torch.int32, device="cuda")  # noqa: E731
        p = moe.Plan(i32(E), i32(E), i32(M, k), i32(P))
        ws = torch.empty(MB.fp8bw_moe_plan_workspace_bytes(M, E, k), dtype=torch.uint8, device="cuda")
        MB.fp8bw_moe_plan(ex, E, p.group_end, p.counts, p.row_of, p.src_of, ws)
    B.fp8bw_sync_status()
    for got, want in zip((p.group_end, p.counts, p.row_of, p.src_of), O.moe_plan(experts, E, P)):
        assert np.array_equal(got.cpu().numpy(), want)


def random_experts(M, E, k, seed, dropped=0.0):
    r = np.random.default_rng(seed)
    ex = np.argsort(r.standard_normal((M, E)) + r.standard_normal(E), axis=1)[:, :k].astype(np.int32)
    ex[r.uniform(size=M) < dropped] = -1
    return np.ascontiguousarray(ex)


@pytest.mark.parametrize("M,E,k,dropped", [
    (1, 1, 1, 0.0), (1, 8, 2, 0.0), (17, 64, 4, 0.0), (31, 8, 1, 0.0), (32, 8, 1, 0.0), (33, 4, 4, 0.3), (511, 8, 2, 0.0),
    (1000, 5, 3, 0.1), (4099, 160, 6, 0.02), (2048, 1024, 8, 0.0), (5, 1024, 32, 0.0), (20011, 64, 8, 0.05),
    (65536, 8, 2, 0.0), (50001, 128, 4, 0.0), (30000, 1000, 3, 0.0),
])
def test_plan(M, E, k, dropped):
    check_plan(random_experts(M, E, k, seed=M, dropped=dropped), E)


@pytest.mark.parametrize("fill", [-1, 0, 6, 7])
@pytest.mark.parametrize("M", [1, 100, 9000])
def test_plan_of_one_expert_or_none(fill, M):
    check_plan(np.full((M, 1), fill, np.int32), 8)


def test_plan_with_more_rows_than_needed():
    check_plan(random_experts(100, 8, 2, seed=1), 8, P=1024)
    check_plan(random_experts(9000, 8, 2, seed=1), 8, P=32768)


def test_plan_skips_and_reports_experts_out_of_range():
    ex = random_experts(300, 8, 2, seed=3)
    bad = ex.copy()
    bad[5, 0], bad[77, 1] = 8, -2
    ex[5, 0] = ex[77, 1] = -1
    B.fp8bw_sync_status()
    got = moe.plan(torch.from_numpy(bad).cuda(), 8)
    with pytest.raises(B.Fp8bwError) as e:
        B.fp8bw_sync_status()
    assert e.value.code == B.ERR_SHAPE
    want = moe.plan(torch.from_numpy(ex).cuda(), 8)
    for n in ("group_end", "counts", "row_of", "src_of"):
        assert torch.equal(getattr(got, n), getattr(want, n))


def test_plan_on_a_reused_workspace_and_in_a_graph():
    """A workspace holding another call's leftovers, and replays of a captured call on new experts."""
    E, k = 64, 4
    ex = torch.from_numpy(random_experts(20000, E, k, seed=1)).cuda()
    p = moe.plan(ex, E)
    ws = torch.full((MB.fp8bw_moe_plan_workspace_bytes(20000, E, k),), 0xFF, dtype=torch.uint8, device="cuda")
    call = lambda: MB.fp8bw_moe_plan(ex, E, p.group_end, p.counts, p.row_of, p.src_of, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (2, 3):
        new = random_experts(20000, E, k, seed=seed, dropped=0.1)
        ex.copy_(torch.from_numpy(new))
        g.replay()
        B.fp8bw_sync_status()
        for got, want in zip((p.group_end, p.counts, p.row_of, p.src_of), O.moe_plan(new, E, p.rows)):
            assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("E,k", [(160, 4), (160, 8), (64, 1), (256, 8), (200, 7), (24, 8)])
def test_rows_of_every_spread(E, k, dtype):
    """Rows whose best experts share one lane, many ties at the smallest chosen key, keys spread over all magnitudes down
    to underflow, and masked experts in between: equal to the oracle where keys tie exactly or lie far apart."""
    r = np.random.default_rng(E + k)
    M = 64
    logits = coarse_logits(M, E, seed=E)
    logits[0:8] = -4
    logits[0:8, 0::8] = 1 + np.arange(len(range(0, E, 8))) / 8          # the best are all 8 apart
    logits[8:16] = 0.5                                                 # everything ties
    logits[16:24] = np.where(r.uniform(size=(8, E)) < 0.5, 2.0, -1.0)  # half of the experts tie at the top
    logits[24:32] = -np.arange(E) * 4.0                                # spread down to underflow
    logits[32:40][r.uniform(size=(8, E)) < 0.9] = NINF                 # few left
    logits[40, :] = NINF
    logits[40, E // 2:E // 2 + k + 3] = 3.0
    logits = logits[r.permutation(M)]
    ref_e, ref_w = O.moe_route(logits, k)
    # spread rows: keys that underflow to the same value tie in fp32 and not in 64 bits
    s = O.moe_scores(logits, "softmax").astype(np.float32)
    keep = np.array([len(np.unique(s[t][s[t] > 1e-37])) >= k or (s[t] > 1e-37).sum() >= k or np.isneginf(logits[t]).any()
                     for t in range(M)])
    x = torch.from_numpy(logits).to(dtype).cuda()
    experts, weights = moe.route(x, k)
    B.fp8bw_sync_status()
    assert keep.sum() > M // 2 and np.array_equal(experts.cpu().numpy()[keep], ref_e[keep])
    assert np.all(np.abs(weights.cpu().numpy() - ref_w)[keep] <= (weight_bound(logits, k) * ref_w + 1e-37)[keep])


@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E", [16, 64, 160, 600])
def test_nan_is_chosen_first_at_every_width(E, biased, groups):
    """A NaN logit comes before every number, masked experts never, whatever path the width takes."""
    x = torch.randn(9, E, device="cuda")
    at = [0, 1, 7, 8, E // 2, E - 2, E - 1, 3, 5]
    for t, e in enumerate(at):
        x[t, e] = float("nan")
        x[t, (e + 2) % E] = float("-inf")
    bias = torch.randn(E, device="cuda") * 0.01 if biased else None
    how = dict(bias=bias, groups=groups, groups_kept=min(groups, 2), group_top=1)
    experts, weights = moe.route(x, 3, score="sigmoid", **how)
    assert experts[:, 0].tolist() == at and bool(weights[:, 0].isnan().all())
    experts, weights = moe.route(x, 3, **how)       # a softmax row with a NaN has nothing else
    assert bool(weights.isnan().all())
    assert not bool((experts == torch.tensor([(e + 2) % E for e in at], device="cuda")[:, None]).any())
    B.fp8bw_sync_status()


@pytest.mark.parametrize("bits", [0x7FC00000, -0x400000, -1, 0x7F800001])
@pytest.mark.parametrize("E", [8, 16, 64, 160, 600])
def test_a_nan_counts_whatever_its_sign_and_payload(E, bits):
    x = torch.randn(5, E, device="cuda")
    at = [0, 7, E // 2, E - 1, 3]
    for t, e in enumerate(at):
        x[t].view(torch.int32)[e] = bits
    assert int(x.isnan().sum()) == 5
    experts, weights = moe.route(x, 2, score="sigmoid")
    assert experts[:, 0].tolist() == at and bool(weights.isnan().all())
    experts, weights = moe.route(x, 2)       # every score is NaN: the lowest places
    assert experts.tolist() == [[0, 1]] * 5 and bool(weights.isnan().all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [8, 16, 64, 160, 600])
def test_infinite_logits(E, dtype):
    x = torch.randn(4, E, device="cuda").to(dtype)
    x[:, E - 3] = float("inf")
    x[1, 2] = float("-inf")
    x[2] = float("-inf")
    experts, weights = moe.route(x, 2, score="sigmoid", renormalize=False)
    assert experts[:, 0].tolist() == [E - 3, E - 3, -1, E - 3]
    assert weights[:, 0].tolist() == [1, 1, 0, 1] and experts[2].tolist() == [-1, -1]
    experts, weights = moe.route(x, 2, renormalize=False)  # inf - inf: the softmax of the row is NaN
    assert bool(weights[[0, 1, 3]].isnan().all()) and weights[2].tolist() == [0, 0]
    assert experts.tolist() == [[0, 1], [0, 1], [-1, -1], [0, 1]]
