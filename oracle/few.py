"""Test infrastructure: MXFP4 weights and the products of a few tokens, plain and in 64 bits.

Only tests may import this module.  Definitions as in ``include/fp8bw_few.h``.
"""
from __future__ import annotations

import numpy as np

from .e4m3 import e4m3_encode
from .moe import moe_route
from .mx import E8M0_BIAS, FLOOR, MX_BLOCK, RCEIL, mx_dequant_row

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e2m1_decode(codes) -> np.ndarray:
    c = np.asarray(codes, np.uint8)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def e2m1_encode(v) -> np.ndarray:
    """Nearest of the 16 values, ties to the even code, saturating."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    code = np.zeros(v.shape, np.uint8)
    for i in range(7):
        middle = (E2M1[i] + E2M1[i + 1]) / 2
        code += (a > middle) | ((a == middle) & (i % 2 == 1))
    return code | np.where(np.signbit(v), 8, 0).astype(np.uint8)


def e2m1_exponent(amax, mode: int = RCEIL) -> np.ndarray:
    """Unbiased exponent of a block of finite weights."""
    a = np.asarray(amax, np.float64)
    safe = np.where(a > 0, a, 1.0)
    _, ex = np.frexp(safe)
    E = ex.astype(np.int64) - 1 - 2                     # floor(log2 amax) - 2
    if mode == RCEIL:
        E = np.where(6 * np.ldexp(1.0, E) >= safe, E, E + 1)
    elif mode != FLOOR:
        raise ValueError("mode must be RCEIL (0) or FLOOR (1)")
    return np.clip(np.where(a > 0, E, -E8M0_BIAS), -E8M0_BIAS, E8M0_BIAS)


def mx4_quant_row(w, mode: int = RCEIL):
    """Packed codes [R, C/2] and E8M0 bytes [R][C/32] of finite fp32 w."""
    w = np.asarray(w)
    blocks = w.reshape(w.shape[0], -1, MX_BLOCK).astype(np.float64)
    E = e2m1_exponent(np.abs(blocks).max(axis=2), mode)
    c = e2m1_encode(blocks * np.ldexp(1.0, -E)[:, :, None]).reshape(w.shape)
    return c[:, 0::2] | (c[:, 1::2] << 4), (E + E8M0_BIAS).astype(np.uint8)


def mx4_unpack(q) -> np.ndarray:
    """Codes [..., C] of packed ones [..., C/2]."""
    return np.stack((q & 15, q >> 4), axis=-1).reshape(*q.shape[:-1], -1)


def mx4_widen(q) -> np.ndarray:
    """e4m3 codes of packed e2m1 codes."""
    return e4m3_encode(e2m1_decode(mx4_unpack(q)))


def mx_weight(q, e8, bits: int) -> np.ndarray:
    """float64 values of MX weights [R, C]."""
    e8 = np.asarray(e8)
    if bits == 8:
        w = mx_dequant_row(q, e8)
    else:
        w = e2m1_decode(mx4_unpack(q)) * np.ldexp(1.0, np.repeat(e8.astype(np.int64) - E8M0_BIAS, MX_BLOCK, axis=-1))
    return np.where(np.repeat(e8 == 255, MX_BLOCK, axis=-1), np.nan, w)


def few_layer(x, router, w13, w2, top_k, bias=None, **how):
    """y, and what its error bounds are made of, from float64 weights w13 [E, 2F, C] and w2 [E, C, F]."""
    x = np.asarray(x, np.float64)
    experts, weights = moe_route(x @ np.asarray(router, np.float64).T, top_k, bias=bias, **how)
    y, bound = np.zeros_like(x), np.zeros_like(x)
    F, C = w2.shape[2], x.shape[1]
    # Sums of n terms in fp32, products exact: at most n roundings of at most 2^-23 of the sum of magnitudes.  Tokens are held to
    # 2^-21 of a block's largest element, activations, in five parts, to 2^-36 of it.
    sums = lambda n: n * 2.0 ** -23  # noqa: E731
    for t in range(x.shape[0]):
        dlogit = sums(C) * float((np.abs(x[t]) * np.abs(np.asarray(router, np.float64))).sum(axis=1).max())
        for e, w in zip(experts[t], weights[t]):
            if e < 0:
                continue
            h = w13[e] @ x[t]
            dh = sums(C) * (np.abs(w13[e]) @ np.abs(x[t])) + 2.0 ** -21 * np.abs(x[t]).max() * np.abs(w13[e]).sum(axis=1)
            gate, up, dg, du = h[:F], h[F:], dh[:F], dh[F:]
            with np.errstate(over="ignore"):
                silu = gate / (1 + np.exp(-gate))
            a = silu * up
            # |silu'| < 1.1; the sigmoid in fp32 is off by a few ulp and |gate| roundings of its argument
            da = 1.1 * dg * (np.abs(up) + du) + np.abs(silu) * du + np.abs(a) * (8 + np.abs(gate)) * 2.0 ** -23
            da += 2.0 ** -36 * np.abs(a).max()
            part = w2[e] @ a
            dpart = np.abs(w2[e]) @ da + sums(F * len(experts[t])) * (np.abs(w2[e]) @ np.abs(a))
            y[t] += w * part
            bound[t] += w * dpart + (4 * dlogit + 2.0 ** -20) * np.abs(w * part)
    return y, bound, experts
