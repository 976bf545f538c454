"""Appends of many sequences at once, a few long ones among short and empty
ones: each sequence gets the same codes, scales and queries as in a call of its
own, whatever bound of one sequence's new tokens is given."""

import numpy as np
import pytest
import torch

import bit_weight_only_gemm_amd as w4
from gpu_util import DEV, TDT, say

pytestmark = pytest.mark.gpu


def _many(B, longest, Hkv, H, D, T, dtype, tokens=None):
    r = np.random.RandomState(B + longest + T)
    news = np.where(r.rand(B) < 0.1, r.randint(1, longest + 1, B), r.randint(0, 4, B))
    news[r.randint(B)] = longest
    if tokens is not None:
        news[-1] += tokens - news.sum()
    lens = news + r.randint(0, 3 * T, B)
    counts = -(-lens // T)
    table = np.full((B, max(counts.max(), 1)), -1, np.int32)
    order = r.permutation(int(counts.sum()) + 1)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    cache = w4.kv8_cache(len(order), T, Hkv, D, DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(news.sum()))
    for n in ("k", "v"):
        cache[n].copy_(torch.randint(1, 256, cache[n].shape, generator=g, device=DEV, dtype=torch.uint8))
        cache[n + "_scale"].copy_(torch.rand(cache[n + "_scale"].shape, generator=g, device=DEV) * 0.03)
    n = int(news.sum())
    mk = lambda h: torch.randn(n, h, D, generator=g, device=DEV).to(TDT[dtype])  # noqa: E731
    a = torch.rand(int(lens.max()) + 1, D // 2, generator=g, device=DEV) * 6
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(DEV)  # noqa: E731
    return cache, mk(H), mk(Hkv), mk(Hkv), a.cos(), a.sin(), table, lens, np.concatenate([[0], news.cumsum()]), dev


@pytest.mark.parametrize("B,longest,Hkv,H,D,T,dtype", [
    (1, 200, 2, 4, 64, 16, "f16"), (3, 150, 1, 1, 128, 32, "bf16"), (64, 90, 2, 6, 64, 16, "bf16"),
    (65, 300, 4, 4, 128, 128, "f16"), (300, 70, 1, 2, 64, 32, "f16"), (129, 257, 2, 2, 128, 64, "bf16")])
def test_a_sequence_alone_and_among_many(B, longest, Hkv, H, D, T, dtype):
    say("append of many", B, longest, Hkv, H, D, T, dtype)
    cache, q, k, v, cos, sin, table, lens, cu, dev = _many(B, longest, Hkv, H, D, T, dtype)
    alone = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in cache.items()}
    bound = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in cache.items()}
    got = w4.kv8_append(cache, k, v, dev(table), dev(lens), dev(cu), q=q, cos=cos, sin=sin)
    also = w4.kv8_append(bound, k, v, dev(table), dev(lens), dev(cu), max_new=int(np.diff(cu).max()),
                         q=q, cos=cos, sin=sin)
    assert torch.equal(got, also)
    for b in range(B):
        t = slice(int(cu[b]), int(cu[b + 1]))
        n = t.stop - t.start
        if n:
            one = w4.kv8_append(alone, k[t], v[t], dev(table[b:b + 1]), dev(lens[b:b + 1]), dev([0, n]),
                                max_new=n, q=q[t], cos=cos, sin=sin)
            assert torch.equal(got[t], one)
    for n in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(cache[n], alone[n]) and torch.equal(cache[n], bound[n])


def test_65536_tokens_of_256_sequences_without_a_bound():
    """What would be 2^32 work-items with room for all tokens in each sequence."""
    B, Hkv, D, T = 256, 8, 64, 16
    cache, _, k, v, _, _, table, lens, cu, dev = _many(B, 2000, Hkv, Hkv, D, T, "f16", tokens=65536)
    parts = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in cache.items()}
    assert len(k) == 65536
    w4.kv8_append(cache, k, v, dev(table), dev(lens), dev(cu))
    for b in range(0, B, 32):
        t = slice(int(cu[b]), int(cu[b + 32]))
        w4.kv8_append(parts, k[t], v[t], dev(table[b:b + 32]), dev(lens[b:b + 32]), dev(cu[b:b + 33] - cu[b]),
                      max_new=int(np.diff(cu[b:b + 33]).max()))
    for n in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(cache[n], parts[n])
