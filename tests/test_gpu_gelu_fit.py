"""The polynomial of gelu's normal distribution as it stands in the source: its error as
fp32 constants, and the error of the whole tail with each step rounded to fp32, are what
the comment beside it states. (The device function itself is held to 2^-18 by the
gated block's GPU tests.)"""
import os
import re

import numpy as np
import pytest
from scipy.special import erfcx, log_ndtr

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_precision_weight_amd", "csrc",
                   "owq_act.h")
F = np.float32


@pytest.fixture(scope="module")
def coefficients():
    s = open(SRC).read()
    first = re.search(r"float q = (-?[\d.]+)f;", s).group(1)
    c = [F(v) for v in [first] + re.findall(r"q = __builtin_fmaf\(q, t, (-?[\d.]+)f\);", s)]
    assert len(c) == 10
    return c


def _fma(a, b, c):
    """One rounding to fp32: the product of fp32 values is exact in fp64."""
    return (np.float64(1) * a * np.float64(1) * np.asarray(b, np.float64) + np.asarray(c, np.float64)).astype(F)


def test_fit(coefficients):
    x = np.concatenate([np.linspace(0, 200, 400001), np.linspace(0, 16, 400001)])
    t = 1 / (1 + x / 4)
    q = np.zeros_like(x)
    for c in coefficients:
        q = q * t + np.float64(c)
    assert np.abs(q * t / (0.5 * erfcx(x / np.sqrt(2.0))) - 1).max() <= 2.0 ** -23.5


def test_tail(coefficients):
    x = np.linspace(0, 16, 800001).astype(F)
    t = (1 / _fma(x, F(0.25), F(1)).astype(np.float64)).astype(F)
    q = np.full_like(x, coefficients[0])
    for c in coefficients[1:]:
        q = _fma(q, t, c)
    hi = F(0.72134752)
    lo = F(0.72134752044448170368 - np.float64(hi))
    s = x * x
    ds = _fma(x, x, -s)
    y = s * hi
    dy = _fma(ds, hi, _fma(s, lo, _fma(s, hi, -y)))
    e0 = np.exp2(-y.astype(np.float64)).astype(F)
    e0[e0 < 2.0 ** -126] = 0
    e = _fma(e0 * F(-0.69314718), dy, e0)
    tail = q * t * e
    p = np.exp(log_ndtr(-x.astype(np.float64)))
    near = x <= 13.1
    assert np.abs(tail[near] / p[near] - 1).max() <= 2.0 ** -20.5
    assert p[~near & (tail == 0)].max() < 2.0 ** -131 and not tail[x >= 13.22].any()
