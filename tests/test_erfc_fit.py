"""How far the gelu epilogue's complementary error function is off, replayed from the constants in its source (CPU)."""
from __future__ import annotations

import pathlib
import re

import numpy as np
import pytest

special = pytest.importorskip("scipy.special")

SOURCE = pathlib.Path(__file__).resolve().parent.parent / "weight_only_int4_awq_amd" / "csrc" / "linear_act.hip"


@pytest.fixture(scope="module")
def coefficients():
    text = SOURCE.read_text()
    body = text[text.index("float erfc_tail("):text.index("float activate(")]
    first = re.search(r"float q = (-?[\d.]+)f;", body).group(1)
    rest = re.findall(r"q = __builtin_fmaf\(q, t, (-?[\d.]+)f\);", body)
    assert len(rest) == 9
    return [np.float32(c) for c in (first, *rest)]


def fma(a, b, c):
    """fp32 a * b + c rounded once (the product is exact in float64; a second rounding moves it by 2^-53 of it)."""
    return (a.astype(np.float64) * b.astype(np.float64) + np.float64(c)).astype(np.float32)


def test_polynomial(coefficients):
    """The fp32 coefficients in exact arithmetic, over the range of the fit."""
    x = np.linspace(0, 14.6, 400001)
    t = 1 / (1 + 0.5 * x)
    q = np.zeros_like(t)
    for c in coefficients:
        q = q * t + np.float64(c)
    assert np.abs(q - np.log(special.erfcx(x) / t)).max() <= 1.2e-7


@pytest.mark.parametrize("last,off", [(5.0, 3e-6), (9.2, 8e-6)])
def test_complementary_error_function(coefficients, last, off):
    """Every step rounded to fp32, the reciprocal and the exponential correctly: the hardware's unit in the
    last place of each, 2^-23, is what the stated figures leave beside it."""
    x = np.linspace(0, last, 400001).astype(np.float32)
    t = np.float32(1) / fma(x, np.full_like(x, 0.5), 1)
    q = np.full_like(t, coefficients[0])
    for c in coefficients[1:]:
        q = fma(q, t, c)
    e = (q.astype(np.float64) - x.astype(np.float64) ** 2).astype(np.float32)
    y = t * np.exp2((e * np.float32(1.4426950408889634)).astype(np.float64)).astype(np.float32)
    assert np.abs(y / special.erfc(x.astype(np.float64)) - 1).max() <= off - 2 * 2.0 ** -23
