"""Paged 8-bit cache: append with rotation, read-back, attention, in 64 bits.

A cache is dict(k [P, Hkv, T, D], v [P, Hkv, T/16, D, 16] codes, k_scale,
v_scale [P, Hkv]); here it is handled as tokens: rows(cache) gives k and v as
signed codes [P, Hkv, T, D].
"""

import numpy as np


def rows_k(k):
    return k.astype(np.int64) - 128


def rows_v(v):
    P, H, S, D, _ = v.shape
    return v.astype(np.int64).transpose(0, 1, 2, 4, 3).reshape(P, H, S * 16, D) - 128


def rotate(x, cos, sin, pos, interleaved):
    """Rows x [n, H, D] at positions pos [n], pairs turned by the table's angles."""
    x = np.array(x, np.float64)
    half = cos.shape[1]
    a = np.arange(half) * 2 if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    c, s = (np.asarray(t, np.float64)[pos][:, None, :] for t in (cos, sin))
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def append_pages(table, lens, cu, T):
    """(sequence, page, first row, end row, first new token) of each touched page."""
    got = []
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        old = lens[b] - n
        for p in range(max(old, 0) // T, -(-lens[b] // T) if n else 0):
            lo, hi = max(p * T, old, 0), min((p + 1) * T, lens[b])
            if hi > lo:
                got.append((b, table[b][p], lo - p * T, hi - p * T, cu[b] + lo - old))
    return got


def attention(q, k, v, table, lens, cu, T, scale, causal):
    """(out, sum p |v|, lse, score error scale) for q [tokens, H, D] and the
    cache's values k, v [P, Hkv, T, D]; a row that sees nothing is 0, lse -inf.
    The last is scale sum |q||k| at its largest over the visible keys."""
    tokens, H, D = q.shape
    G = H // k.shape[1]
    out, mass = np.zeros((tokens, H, D)), np.zeros((tokens, H, D))
    lse, work = np.full((tokens, H), -np.inf), np.zeros((tokens, H))
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        if lens[b] <= 0:
            continue
        pages = [table[b][p] for p in range(-(-lens[b] // T))]
        kk = k[pages].transpose(1, 0, 2, 3).reshape(k.shape[1], -1, D)[:, :lens[b]]
        vv = v[pages].transpose(1, 0, 2, 3).reshape(k.shape[1], -1, D)[:, :lens[b]]
        for j in range(n):
            seen = min(lens[b], lens[b] - n + j + 1) if causal else lens[b]
            if seen <= 0:
                continue
            for h in range(H):
                x = q[cu[b] + j, h].astype(np.float64)
                keys, vals = kk[h // G, :seen], vv[h // G, :seen]
                s = keys @ x * scale
                m = s.max()
                p = np.exp(s - m)
                z = p.sum()
                out[cu[b] + j, h] = p @ vals / z
                mass[cu[b] + j, h] = p @ np.abs(vals) / z
                lse[cu[b] + j, h] = m + np.log(z)
                work[cu[b] + j, h] = (np.abs(keys) @ np.abs(x)).max() * abs(scale)
    return out, mass, lse, work


def attention_bounds(out, mass, work, tokens_seen, D, dtype):
    """Bounds of |out - exact| and |lse - exact|.

    A score is a sum of D exact products in fp32, each addition off by at most
    2^-23 of the terms' magnitudes, then two products and a subtraction: d =
    (D + 4) 2^-23 work absolute.  The exponential and its argument add 2^-20.
    Probabilities are off by that relative amount, and by 2^-11 where they
    enter the second product in fp16 (2^-24 of the largest, absolutely, below
    fp16's normal range); its sums over 64 tokens and then over units add
    (64 + units) 2^-23; numerator and denominator together twice the first.
    Then one rounding to the output's type."""
    u, tiny = (2.0 ** -11, 2.0 ** -25) if dtype == "f16" else (2.0 ** -8, 2.0 ** -134)
    d = ((D + 4) * 2.0 ** -23 * work + 2.0 ** -20)[..., None]
    rel = 2 * d + 2.0 ** -11 + (80 + tokens_seen / 64) * 2.0 ** -22 + tokens_seen * 2.0 ** -24
    return rel * mass + u * np.abs(out) * 1.01 + tiny, d[..., 0] + 2.0 ** -18
