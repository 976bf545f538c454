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
