"""Pins of the oracle's MXFP4 (no GPU): against torch's arithmetic and by brute force."""
import numpy as np
import pytest

import oracle
from oracle import few as OF


def test_values_are_the_format_s():
    for c in range(16):
        s, e, m = c >> 3, (c >> 1) & 3, c & 1
        v = m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
        assert OF.e2m1_decode(np.array([c]))[0] == (-v if s else v)


def test_encode_is_the_nearest_with_ties_to_the_even_code():
    v = np.linspace(-7, 7, 14 * 512 + 1)  # every tie is among them
    codes = OF.e2m1_encode(v)
    for x, c in zip(v, codes):
        far = np.abs(OF.E2M1 - min(abs(x), 6.0))
        best = np.flatnonzero(far == far.min())
        want = best[0] if len(best) == 1 else [b for b in best if b % 2 == 0][0]
        assert (c & 7) == want and bool(c & 8) == bool(np.signbit(x))


@pytest.mark.parametrize("mode", [oracle.RCEIL, oracle.FLOOR])
def test_exponent_by_brute_force(mode):
    bits = np.arange(0, 0x7F80, dtype=np.uint32) << 16  # every finite bf16 magnitude
    amax = bits.view(np.float32).astype(np.float64)
    E = OF.e2m1_exponent(amax, mode)
    for a, e in zip(amax[1:], E[1:]):
        if mode == oracle.RCEIL:
            assert 6 * 2.0 ** e >= a and (e == -127 or 6 * 2.0 ** (e - 1) < a)
        else:
            assert e == max(int(np.floor(np.log2(a))) - 2, -127)
    assert E[0] == -127


def test_widened_values_are_the_same():
    q = np.arange(256, dtype=np.uint8)
    assert np.array_equal(oracle.e4m3_decode(OF.mx4_widen(q)), OF.e2m1_decode(OF.mx4_unpack(q)))


def test_packing_order():
    w = np.zeros((1, 32), np.float32)
    w[0, 0], w[0, 1] = 6.0, -1.5
    q, e8 = OF.mx4_quant_row(w)
    assert e8[0, 0] == 127 and q[0, 0] == 7 | (11 << 4) and not q[0, 1:].any()
