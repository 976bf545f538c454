"""The cap of attention scores: the kernels' two forms of tanh, evaluated in fp32
as csrc/kv8_attention.h writes them, against the bound that include/w4a16.h states
(host-only; the exponential and the reciprocal are taken to be off by 1 ulp)."""

import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = np.float32


def source(*path):
    with open(os.path.join(ROOT, *path)) as f:
        return f.read()


KERNEL = source("bit_weight_only_gemm_amd", "csrc", "kv8_attention.h")
HEADER = re.sub(r"\s*\n \*\s*", " ", source("include", "w4a16.h"))


def fma(a, b, c):
    """Rounded once (up to a double rounding of 2^-29 ulp)."""
    return (np.asarray(a, np.float64) * np.asarray(b, np.float64) + np.asarray(c, np.float64)).astype(F)


def number(name):
    return float(re.search(name + r" = ([0-9.e+-]+)f", KERNEL).group(1))


def near(x):
    """x P(x^2)"""
    body = KERNEL[KERNEL.index("float tanh_near(float x) {"):]
    body = body[:body.index("}")]
    c = [F(v) for v in re.findall(r"(-?\d\.\d+)f", body)]
    assert len(c) == 5
    y = (x * x).astype(F)
    p = fma(y, c[0], c[1])
    for v in c[2:]:
        p = fma(y, p, v)
    return (x * p).astype(F)


def far(z, ulps):
    """1 - 2 / (1 + 2^z), the exponential and the reciprocal each off by some ulp."""
    with np.errstate(over="ignore"):
        e = np.exp2(z.astype(np.float64)).astype(F)
        e = np.where(np.isfinite(e), e * F(1 + ulps[0] * 2.0 ** -23), e).astype(F)
        d = (F(1) + e).astype(F)
        r = (1.0 / d.astype(np.float64)).astype(F)
    r = (r * F(1 + ulps[1] * 2.0 ** -23)).astype(F)
    return fma(F(-2), r, F(1))


def stated():
    m = re.search(r"the cap is off by 2\^(-\d+) softcap up to (\d+), by 2\^(-\d+) of the score beyond", HEADER)
    assert m, "the header states the cap's bound"
    return 2.0 ** int(m.group(1)), float(m.group(2)), 2.0 ** int(m.group(3))


def test_small_scores():
    absolute, _, relative = stated()
    bend = number("kBend")
    x = np.concatenate([np.linspace(1e-6, bend, 2_000_001), np.geomspace(1e-30, 1e-3, 100_000)]).astype(F)
    exact = np.tanh(x.astype(np.float64))
    err = np.abs(near(x).astype(np.float64) - exact)
    # and one product more, that with the cap: 2^-24 of the score
    assert np.max(err + 2.0 ** -24 * exact) <= absolute
    assert np.max(err / exact) + 2.0 ** -24 <= relative
    assert np.array_equal(near(-x), -near(x))


@pytest.mark.parametrize("ulps", [(a, b) for a in (-1, 0, 1) for b in (-1, 0, 1)])
def test_any_score_under_a_cap(ulps):
    """Up to the stated cap the error is a part of the cap."""
    absolute, most, _ = stated()
    assert most <= number("kWideCap") / np.log2(np.e)
    x = np.concatenate([np.linspace(-12, 12, 1_000_001), [-200, 200]]).astype(F)
    z = (x * F(2 * np.log2(np.e))).astype(F)
    err = np.abs(far(z, ulps).astype(np.float64) - np.tanh(x.astype(np.float64)))
    assert np.max(err) + 2.0 ** -24 <= absolute


@pytest.mark.parametrize("ulps", [(a, b) for a in (-1, 0, 1) for b in (-1, 0, 1)])
def test_large_scores_under_a_wide_cap(ulps):
    """Beyond it scores below kBend of the cap take the polynomial: the error of the
    rest is a part of the score."""
    _, _, relative = stated()
    x = np.linspace(number("kBend"), 12, 1_000_001).astype(F)
    z = (x * F(2 * np.log2(np.e))).astype(F)
    exact = np.tanh(x.astype(np.float64))
    assert np.max(np.abs(far(z, ulps).astype(np.float64) - exact) / exact) + 2.0 ** -24 <= relative
