"""Pins of the 64-bit oracle of routing, dispatch, combine and the gated
activation: hand-worked cases, invariants, and gradients against differences."""
import numpy as np
import pytest

from oracle import moe as O

RNG = np.random.default_rng


def test_route_hand_case():
    # softmax of (ln 1, ln 2, ln 5) = (1, 2, 5) / 8; the best two are experts 2 and 1
    logits = np.log(np.array([[1.0, 2.0, 5.0]]))
    experts, w = O.moe_route(logits, 2, renormalize=False)
    assert experts.tolist() == [[2, 1]] and np.allclose(w, [[5 / 8, 2 / 8]])
    _, w = O.moe_route(logits, 2, scale=2.0)
    assert np.allclose(w, [[2 * 5 / 7, 2 * 2 / 7]])


def test_bias_chooses_and_does_not_weigh():
    logits = np.log(np.array([[1.0, 2.0, 5.0]]))
    experts, w = O.moe_route(logits, 1, bias=[1.0, 0.0, 0.0], renormalize=False)
    assert experts.tolist() == [[0]] and np.allclose(w, [[1 / 8]])


def test_ties_masks_and_empty_rows():
    ninf = -np.inf
    logits = np.array([[0.0, 0.0, 0.0, 0.0], [ninf, 1.0, ninf, 1.0], [ninf] * 4, [ninf, ninf, 0.0, ninf]])
    experts, w = O.moe_route(logits, 2)
    assert experts.tolist() == [[0, 1], [1, 3], [-1, -1], [2, -1]]
    assert np.allclose(w, [[0.5, 0.5], [0.5, 0.5], [0, 0], [1, 0]])


def test_groups_hand_case():
    # runs {0, 1}, {2, 3}, {4, 5}: sums of the two largest 0.9, 1.0, 0.8; the single best key is in run 0
    s = np.array([[0.85, 0.05, 0.5, 0.5, 0.4, 0.4]])
    logits = np.log(s / (1 - s))
    experts, _ = O.moe_route(logits, 2, score="sigmoid", groups=3, groups_kept=1, group_top=2)
    assert experts.tolist() == [[2, 3]]
    experts, _ = O.moe_route(logits, 2, score="sigmoid", groups=3, groups_kept=1, group_top=1)
    assert experts.tolist() == [[0, 1]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_against_differences(score, renormalize):
    r = RNG(3)
    logits, dw = r.normal(size=(5, 9)), r.normal(size=(5, 3))
    experts, _ = O.moe_route(logits, 3, score=score)
    experts[1, 2] = experts[4, 1] = -1
    how = dict(score=score, renormalize=renormalize, scale=1.7)
    got = O.moe_route_bwd(dw, logits, experts, **how)
    d = 1e-6
    for t in range(5):
        for e in range(9):
            up, down = logits.copy(), logits.copy()
            up[t, e] += d
            down[t, e] -= d
            slope = (dw * (O.moe_weights(up, experts, **how) - O.moe_weights(down, experts, **how))).sum() / (2 * d)
            # central differences: d^2 / 6 times a third derivative of order 1, and 2^-53 / d of rounding
            assert abs(got[t, e] - slope) < 1e-8


def test_swiglu_gradient_against_differences():
    r = RNG(4)
    h, da = r.normal(size=(3, 8)), r.normal(size=(3, 4))
    got = O.swiglu_bwd(da, h)
    d = 1e-6
    for i in np.ndindex(*h.shape):
        up, down = h.copy(), h.copy()
        up[i] += d
        down[i] -= d
        assert abs(got[i] - (da * (O.swiglu(up) - O.swiglu(down))).sum() / (2 * d)) < 1e-8


def test_combine_is_the_transpose_of_gather():
    r = RNG(5)
    experts = np.array([[0, 2], [2, -1], [1, 0], [-1, -1]], np.int32)
    group_end, counts, row_of, src_of = O.moe_plan(experts, 3, 128)
    assert group_end.tolist() == [32, 64, 128] and counts.tolist() == [2, 1, 2]
    assert row_of.tolist() == [[0, 64], [65, -1], [32, 1], [-1, -1]]
    x, y = r.normal(size=(4, 32)), r.normal(size=(128, 32))
    rows = O.moe_gather(x, src_of, 2)
    assert np.all(rows[src_of < 0] == 0)
    # <gather(x), y> = <x, combine(y)>, up to the rounding of x to fp32
    assert abs((rows * y).sum() - (x * O.moe_combine(y, row_of)).sum()) < 1e-4
    w = r.uniform(size=(4, 2)).astype(np.float32)
    d = 1e-6
    dout = r.normal(size=(4, 32))
    dw = O.moe_combine_dweights(dout, y, row_of)
    for t, j in np.ndindex(4, 2):
        up = w.astype(np.float64)
        up[t, j] += d
        slope = (dout * (O.moe_combine(y, row_of, up) - O.moe_combine(y, row_of, w.astype(np.float64)))).sum() / d
        assert abs(dw[t, j] - slope) < 1e-6
