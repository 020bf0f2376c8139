"""How far a rotary table's entries may be off, from the arithmetic of its kernel replayed in numpy (CPU):
the angle p f / 2 pi and its reduction in float64, the series of the eighth of a turn in fp32."""
from __future__ import annotations

import numpy as np
import pytest

TWO_PI = 6.283185307179586476925286766559


def fma(a, b, c):
    """fp32 a * b + c rounded once (the product is exact in float64; a second rounding moves it by 2^-53 of it)."""
    return (a.astype(np.float64) * b.astype(np.float64) + np.float64(c)).astype(np.float32)


def series(y):
    f = np.float32
    z = y * y
    s = fma(z, np.full_like(z, f(1 / 362880)), f(-1 / 5040))
    s = fma(z, s, f(1 / 120))
    s = fma(z, s, f(-1 / 6))
    s = fma(y * z, s, y)
    c = fma(z, np.full_like(z, f(-1 / 3628800)), f(1 / 40320))
    c = fma(z, c, f(-1 / 720))
    c = fma(z, c, f(1 / 24))
    c = fma(z, c, f(-0.5))
    return s, fma(z, c, f(1))


def table(p, f):
    """The kernel's cosines and sines of the positions p (float64 integers) at the frequency f, m = 1."""
    a = p * (np.float64(f) / TWO_PI)
    q4 = np.rint(4.0 * a)
    s, c = series((TWO_PI * (a - 0.25 * q4)).astype(np.float32))
    q = q4.astype(np.int64) & 3
    sn, cs = np.where(q & 1, c, s), np.where(q & 1, s, c)
    return np.where((q == 1) | (q == 2), -cs, cs).astype(np.float64), np.where(q & 2, -sn, sn).astype(np.float64)


def off(p, f):
    """The largest error against 80-bit floats, f taken for exact."""
    c, s = table(p, f)
    a = p.astype(np.longdouble) * np.longdouble(f)
    return float(max(np.abs(c - np.cos(a)).max(), np.abs(s - np.sin(a)).max()))


def rows(end, n=200000):
    return np.arange(end - n, end, dtype=np.float64)


@pytest.mark.parametrize("f", [1.0, 0.8, 0.3])
def test_two_ulp_up_to_angles_of_2_24(f):
    assert np.finfo(np.longdouble).eps < 2.0 ** -60
    for end in (200000, 1 << 20, 1 << 24):
        # the fp32 part stays within 3/4 of an ulp of 1; the rest of the 2 is the angle's
        assert off(rows(end), f) <= 2.0 ** -22
    assert off(rows(200000), f) <= 2.0 ** -23


def test_far_angles_follow_the_stated_growth():
    """2^-49 p f more beyond angles of 2^24; and 2 ulp alone do not hold up to the last position."""
    for end in (1 << 27, 1 << 29, (1 << 31) - 1):
        for f in (1.0, 0.8, 0.3):
            assert off(rows(end), f) <= 2.0 ** -22 + 2.0 ** -49 * end * f
    assert off(rows((1 << 31) - 1), 1.0) > 2.0 ** -22
