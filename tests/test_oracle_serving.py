"""Pins for oracle/w8a8.py and oracle/kv8.py: exact rational arithmetic, closed
forms, and an independent library routine."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import kv8, w8a8


# ------------------------------------------------------------- 8-bit product

def test_quantize_closed_form():
    x = np.array([[127.0, -63.5, 1.0, 0.49], [0.0, 0.0, 0.0, 0.0], [-2.54, 1.27, 0.02, 0.0]])
    c, s = w8a8.quantize(x)
    assert np.allclose(s, [1.0, 1.0, 0.02], rtol=1e-15)
    assert c.tolist() == [[127, -64, 1, 0], [0, 0, 0, 0], [-127, 64, 1, 0]]      # half to even


def test_quantize_is_the_nearest_code():
    x = np.random.default_rng(1).standard_normal((5, 200))
    c, s = w8a8.quantize(x)
    assert np.abs(c).max(axis=1).tolist() == [127] * 5
    assert np.all(np.abs(c * s[:, None] - x) <= s[:, None] * (0.5 + 1e-12))


def test_product_in_rationals():
    r = np.random.default_rng(2)
    xq, wq = r.integers(-127, 128, (3, 20)), r.integers(-127, 128, (4, 20))
    xs, ws, b = r.random(3), r.random(4), r.standard_normal(4)
    y, mag = w8a8.product(xq, xs, wq, ws, b)
    for m in range(3):
        for n in range(4):
            acc = sum(int(p) * int(q) for p, q in zip(xq[m], wq[n]))
            term = acc * Fraction(float(xs[m])) * Fraction(float(ws[n]))
            want = term + Fraction(float(b[n]))
            assert abs(Fraction(float(y[m, n])) - want) <= Fraction(float(mag[m, n])) * Fraction(1, 2 ** 50)
            assert mag[m, n] >= abs(float(want)) * (1 - 1e-14)


def test_product_bound_holds_for_a_float32_evaluation():
    r = np.random.default_rng(3)
    xq, wq = r.integers(-127, 128, (40, 512)), r.integers(-127, 128, (30, 512))
    xs, ws = r.random(40).astype(np.float32), r.random(30).astype(np.float32)
    b = r.standard_normal(30).astype(np.float32)
    y, mag = w8a8.product(xq, xs, wq, ws, b)
    f = (xq @ wq.T).astype(np.float32) * (xs[:, None] * ws[None]) + b
    for name, t in (("f16", torch.float16), ("bf16", torch.bfloat16)):
        got = torch.from_numpy(f / 64).to(t).double().numpy()
        assert np.all(np.abs(got - y / 64) <= w8a8.product_bound(y / 64, mag / 64, name))
        assert np.any(np.abs(got - y / 64) > 0.5 * w8a8.product_bound(y / 64, mag / 64, name))


# --------------------------------------------------------------- 8-bit cache

def test_cache_orders():
    k = np.arange(2 * 3 * 16 * 4).reshape(2, 3, 16, 4) % 256
    assert np.array_equal(kv8.rows_k(k.astype(np.uint8)), k - 128)
    v = np.zeros((1, 1, 2, 4, 16), np.uint8)            # [page, head, 16s of tokens, channel, token]
    v[0, 0, 1, 2, 5] = 200
    rows = kv8.rows_v(v)
    assert rows.shape == (1, 1, 32, 4) and rows[0, 0, 21, 2] == 72
    assert (rows == -128).sum() == rows.size - 1


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_complex_multiplication(interleaved):
    r = np.random.default_rng(4)
    x, pos = r.standard_normal((5, 2, 12)), np.array([0, 3, 9, 2, 9])
    a = r.random((10, 4)) * 6                            # 8 of 12 channels turned
    y = kv8.rotate(x, np.cos(a), np.sin(a), pos, interleaved)
    pair = (lambda t: (t[..., 0:8:2], t[..., 1:8:2])) if interleaved else (
        lambda t: (t[..., :4], t[..., 4:8]))
    re, im = pair(x)
    z = (re + 1j * im) * np.exp(1j * a[pos])[:, None]
    assert np.allclose(pair(y)[0], z.real) and np.allclose(pair(y)[1], z.imag)
    assert np.array_equal(y[..., 8:], x[..., 8:])


def test_pages_of_an_append():
    # 10 tokens after 5 and 3 after 16 in pages of 8, then none
    table, lens, cu = [[7, 4], [1, 2, 3], [0]], [15, 19, 4], [0, 10, 13, 13]
    assert kv8.append_pages(table, lens, cu, 8) == [
        (0, 7, 5, 8, 0), (0, 4, 0, 7, 3), (1, 3, 0, 3, 10)]


@pytest.mark.parametrize("causal", [False, True])
def test_attention_against_a_library_routine(causal):
    r = np.random.default_rng(5)
    T, Hkv, H, D, lens, news = 16, 2, 6, 8, [37, 3, 16], [5, 3, 1]
    table = [[4, 0, 2], [1, -1, -1], [3, -1, -1]]
    k, v = r.standard_normal((2, 5, Hkv, T, D))
    cu = np.concatenate([[0], np.cumsum(news)])
    q = r.standard_normal((sum(news), H, D))
    out, mass, lse, work = kv8.attention(q, k, v, table, lens, cu, T, 0.3, causal)
    for b, n in enumerate(lens):
        pages = table[b][:-(-n // T)]
        kk = torch.from_numpy(np.concatenate([k[p] for p in pages], axis=1)[:, :n]).repeat_interleave(3, 0)
        vv = torch.from_numpy(np.concatenate([v[p] for p in pages], axis=1)[:, :n]).repeat_interleave(3, 0)
        qq = torch.from_numpy(q[cu[b]:cu[b + 1]]).transpose(0, 1)
        see = torch.ones(news[b], n, dtype=torch.bool)
        if causal:
            see = see.tril(n - news[b])
        want = torch.nn.functional.scaled_dot_product_attention(qq, kk, vv, attn_mask=see, scale=0.3)
        assert np.allclose(out[cu[b]:cu[b + 1]], want.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-13)
        s = (qq @ kk.transpose(1, 2) * 0.3).masked_fill(~see, -np.inf)
        assert np.allclose(lse[cu[b]:cu[b + 1]], s.logsumexp(-1).T.numpy(), rtol=1e-12)
    assert np.all(mass >= np.abs(out) - 1e-12) and np.all(work > 0)


def test_attention_of_rows_that_see_nothing():
    q, k = np.ones((3, 1, 4)), np.ones((1, 1, 16, 4))
    out, _, lse, _ = kv8.attention(q, k, k, [[0]], [2], [0, 3], 16, 1.0, True)
    assert np.all(out[0] == 0) and lse[0, 0] == -np.inf      # 3 new tokens in a length of 2
    assert np.allclose(out[1:], 1)
