"""8-bit integer product with token and channel scales, in 64 bits."""

import numpy as np


def quantize(x):
    """Rows of x [M, K] -> (codes int64 [M, K], scales float64 [M])."""
    x = np.asarray(x, np.float64)
    s = np.abs(x).max(axis=1) / 127.0
    s[s == 0] = 1.0
    return np.clip(np.rint(x / s[:, None]), -127, 127).astype(np.int64), s


def product(xq, xs, wq, ws, bias=None):
    """(y, sum of the magnitudes of y's terms) in 64 bits, integer sums exact."""
    acc = xq.astype(np.int64) @ wq.astype(np.int64).T
    y = acc * (np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64)[None, :])
    mag = np.abs(y)
    if bias is not None:
        b = np.asarray(bias, np.float64)
        y, mag = y + b, mag + np.abs(b)
    return y, mag


def product_bound(y, mag, dtype):
    """How far a correctly rounded fp32 evaluation may be from y: the sum's
    conversion, two products and an addition in fp32 (each half an ulp, 2^-24;
    a fifth for second-order terms), then half an ulp of the 16-bit type (or of
    its smallest subnormal)."""
    u, tiny = (2.0 ** -11, 2.0 ** -25) if dtype == "f16" else (2.0 ** -8, 2.0 ** -134)
    return u * np.abs(y) * (1 + 2.0 ** -10) + 5 * 2.0 ** -24 * mag + tiny


def gated(xq, xs, wq, ws, bias, act):
    """act(gate) * up of the rows of wq [2 F, K] in 64 bits, and what bounds it:
    (y, g, u, act(g), magnitudes of g's and u's terms).  The integer sums are
    below 2^53, so exact."""
    from scipy.special import expit, ndtr
    acc = xq.astype(np.float64) @ wq.astype(np.float64).T
    v = acc * (np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64)[None, :])
    mag = np.abs(v)
    if bias is not None:
        b = np.asarray(bias, np.float64)
        v, mag = v + b, mag + np.abs(b)
    F = v.shape[1] // 2
    g, u = v[:, :F], v[:, F:]
    a = {"silu": lambda: g * expit(g), "gelu": lambda: g * ndtr(g),
         "gelu_tanh": lambda: g * expit(2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3))}[act]()
    return a * u, g, u, a, mag[:, :F], mag[:, F:]


def gated_bound(y, g, u, a, mag_g, mag_u, act, dtype):
    """g and u are off by 4 2^-24 of their terms (product_bound's, without the
    rounding to 16 bits).  An activation's slope is at most 1.13, so the first
    moves act(g) by 1.13 times that; the activation itself is off by 2^-19 of
    itself (a reciprocal and an exponential of 1 ulp, five roundings, for gelu a
    fit that is 7e-7 off: 2^-20 and a half), and by the exponential's argument,
    itself off by 4 roundings: 2^-22 for each unit of it.  Where the exponential
    leaves fp32 act(g) is 0: at most |g| 2^-126.  Then the 16-bit rounding."""
    u16, tiny = (2.0 ** -11, 2.0 ** -25) if dtype == "f16" else (2.0 ** -8, 2.0 ** -134)
    arg = {"silu": np.abs(g), "gelu": g * g / 2, "gelu_tanh": 1.6 * np.abs(g) * (1 + 0.0448 * g * g)}[act]
    dg, du = 5 * 2.0 ** -24 * mag_g, 5 * 2.0 ** -24 * mag_u
    da = 1.13 * dg + np.abs(a) * (2.0 ** -19 + 2.0 ** -22 * arg) + np.abs(g) * 2.0 ** -126
    err = da * np.abs(u) + (np.abs(a) + da) * du
    return err * (1 + u16) + u16 * np.abs(y) * (1 + 2.0 ** -10) + tiny
