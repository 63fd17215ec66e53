"""Test infrastructure: the operators around the experts' products, plain and in 64 bits.

Only tests may import this module.  Definitions as in ``include/fp8bw_moe.h``;
each function is the formula written out, with loops where they are clearer.
"""
from __future__ import annotations

import numpy as np

from .mx import RCEIL, mx_quant_1x32_col, mx_quant_1x32_row

EPS = 1e-20
LOWEST = -float(np.finfo(np.float32).max)


def moe_scores(logits: np.ndarray, score: str) -> np.ndarray:
    """float64 scores [M, E]; a softmax row of nothing but -inf has scores 0."""
    x = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        top = x.max(axis=1, keepdims=True)
        e = np.exp(x - np.where(top == -np.inf, 0.0, top))
        total = e.sum(axis=1, keepdims=True)
        return np.where(total == 0, 0.0, e / np.where(total == 0, 1.0, total))


def _best(keys, count):
    """Indices of the `count` largest unmasked (> -inf) keys: NaN above all, the lowest index first among equals."""
    order = sorted((i for i, v in enumerate(keys) if v != -np.inf),
                   key=lambda i: (0, 0.0, i) if np.isnan(keys[i]) else (1, -keys[i], i))
    return order[:count]


def moe_keys(logits, score, bias=None):
    """float64 keys [M, E], -inf where masked."""
    x = np.asarray(logits, np.float64)
    b = np.zeros(x.shape[1]) if bias is None else np.asarray(bias, np.float64)
    with np.errstate(invalid="ignore"):
        return np.where((x == -np.inf) | (b == -np.inf), -np.inf, moe_scores(x, score) + b)


def moe_route(logits, top_k, bias=None, score="softmax", renormalize=True, scale=1.0, groups=1, groups_kept=1,
              group_top=1):
    """experts int32 [M, top_k] and float64 weights [M, top_k]."""
    M, E = np.asarray(logits).shape
    s, keys = moe_scores(logits, score), moe_keys(logits, score, bias)
    experts, weights = np.full((M, top_k), -1, np.int32), np.zeros((M, top_k))
    size = E // groups
    for t in range(M):
        key = keys[t].copy()
        if groups > 1:
            total = []
            for g in range(groups):
                best = _best(key[g * size:(g + 1) * size], group_top)
                v = sum(key[g * size + i] for i in best)
                total.append(np.nan if np.isnan(v) else max(v, LOWEST) if best else -np.inf)
            kept = _best(total, groups_kept)
            for g in range(groups):
                if g not in kept:
                    key[g * size:(g + 1) * size] = -np.inf
        best = _best(key, top_k)
        chosen = s[t, best]
        experts[t, :len(best)] = best
        weights[t, :len(best)] = scale * (chosen / (chosen.sum() + EPS) if renormalize else chosen)
    return experts, weights


def moe_weights(logits, experts, score="softmax", renormalize=True, scale=1.0):
    """float64 weights of given experts."""
    s = moe_scores(logits, score)
    chosen = np.where(experts >= 0, np.take_along_axis(s, np.maximum(experts, 0).astype(np.int64), axis=1), 0.0)
    return scale * (chosen / (chosen.sum(axis=1, keepdims=True) + EPS) if renormalize else chosen)


def moe_route_bwd(dweights, logits, experts, score="softmax", renormalize=True, scale=1.0):
    """float64 dlogits [M, E]."""
    s = moe_scores(logits, score)
    dlogits = np.zeros_like(s)
    for t in range(s.shape[0]):
        live = [j for j, e in enumerate(experts[t]) if e >= 0]
        if not live:
            continue
        idx = experts[t, live].astype(np.int64)
        c = s[t, idx]
        ds = scale * np.asarray(dweights, np.float64)[t, live]
        if renormalize:
            D = c.sum() + EPS
            ds = (ds - (ds * c).sum() / D) / D
        full = np.zeros(s.shape[1])
        full[idx] = ds
        dlogits[t] = full * s[t] * (1 - s[t]) if score == "sigmoid" else s[t] * (full - (ds * c).sum())
    return dlogits


def moe_plan(experts, E, P):
    """group_end, counts, row_of, src_of by walking the entries one after another."""
    experts = np.asarray(experts)
    flat = experts.reshape(-1)
    counts = np.array([(flat == e).sum() for e in range(E)], np.int32)
    end = np.cumsum((counts + 31) // 32 * 32)
    at = end - (counts + 31) // 32 * 32
    row_of, src_of = np.full(flat.size, -1, np.int32), np.full(P, -1, np.int32)
    for i, e in enumerate(flat):
        if e >= 0:
            row_of[i] = at[e]
            src_of[at[e]] = i
            at[e] += 1
    group_end = end.astype(np.int32)
    group_end[-1] = P
    return group_end, counts, row_of.reshape(experts.shape), src_of


def moe_gather(x, src_of, top_k, weights=None):
    """float32 rows [P, C]; the product with the weight is one fp32 product."""
    x = np.asarray(x, np.float32)
    rows = x[np.maximum(src_of, 0) // top_k]
    if weights is not None:
        rows = rows * np.asarray(weights, np.float32).reshape(-1)[np.maximum(src_of, 0)][:, None]
    return np.where((src_of >= 0)[:, None], rows, np.float32(0)).astype(np.float32)


def moe_gather_quant(x, src_of, top_k, weights=None, mode=RCEIL):
    """q, e8, qT, e8T of the gathered rows."""
    rows = moe_gather(x, src_of, top_k, weights)
    return (*mx_quant_1x32_row(rows, mode), *mx_quant_1x32_col(rows, mode))


def moe_combine(y, row_of, weights=None, base=None):
    """float64 out [M, C]."""
    y = np.asarray(y, np.float64)
    out = np.zeros((row_of.shape[0], y.shape[1])) if base is None else np.asarray(base, np.float64).copy()
    for t in range(row_of.shape[0]):
        for j, r in enumerate(row_of[t]):
            if r >= 0:
                out[t] += y[r] * (1.0 if weights is None else float(weights[t, j]))
    return out


def moe_combine_dweights(dout, y, row_of):
    """float64 dweights [M, top_k]."""
    dots = np.einsum("tc,tjc->tj", np.asarray(dout, np.float64), np.asarray(y, np.float64)[np.maximum(row_of, 0)])
    return np.where(row_of >= 0, dots, 0.0)


def swiglu(h):
    """float64 a [R, F] of h = [gate | up]."""
    h = np.asarray(h, np.float64)
    F = h.shape[1] // 2
    with np.errstate(over="ignore"):
        return h[:, :F] / (1.0 + np.exp(-h[:, :F])) * h[:, F:]


def swiglu_bwd(da, h):
    """float64 gradient of h (the values the kept codes stand for)."""
    h, da = np.asarray(h, np.float64), np.asarray(da, np.float64)
    F = h.shape[1] // 2
    gate, up = h[:, :F], h[:, F:]
    with np.errstate(over="ignore"):
        sig = 1.0 / (1.0 + np.exp(-gate))
    return np.concatenate([da * up * sig * (1 + gate * (1 - sig)), da * gate * sig], axis=1)
