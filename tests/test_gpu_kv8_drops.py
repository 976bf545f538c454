"""Drafted tokens that are appended, dropped and followed by accepted ones
(kv8_reserve above and below 0 around kv8_append): which codes and scales a page is
left with, what a NaN among the drafted rows does, and drafting on a fork, which
leaves the row as it was."""

import numpy as np
import pytest
import torch

import bit_weight_only_gemm_amd as w4
from gpu_util import DEV, TDT, say
from oracle import kv8

pytestmark = pytest.mark.gpu
INV = np.float32(1) / np.float32(127)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Pages:
    """The append's definition on signed codes [page][head][T][D] and scales, keys
    and values alike (no rotation)."""

    def __init__(self, pages, T, Hkv, D):
        self.T, self.codes, self.scale = T, np.zeros((pages, Hkv, T, D), np.int64), np.zeros((pages, Hkv), np.float32)

    def append(self, table, length, rows):
        """rows [n][Hkv][D] behind the first `length` tokens."""
        t = 0
        while t < len(rows):
            page, lo = table[(length + t) // self.T], (length + t) % self.T
            n = min(self.T - lo, len(rows) - t)
            x = rows[t:t + n].transpose(1, 0, 2)
            old = self.scale[page] if lo else np.zeros_like(self.scale[page])
            s = np.maximum(old, np.abs(x).max((1, 2)) * INV)
            ratio = (old / s)[:, None, None]
            was = self.codes[page][:, :lo]
            self.codes[page][:, :lo] = np.where(ratio == 1, was, np.clip(np.rint(was.astype(np.float32) * ratio), -128, 127))
            self.codes[page][:, lo:lo + n] = np.clip(np.rint(x / s[:, None, None]), -127, 127)
            self.scale[page] = s
            t += n

    def check(self, cache, table, length, dtype):
        """Every cached token of a row, codes, scales and read back."""
        for i in range(-(-length // self.T)):
            page, n = table[i], min(self.T, length - i * self.T)
            k, v = (f(cache[n_].cpu().numpy())[page] for f, n_ in ((kv8.rows_k, "k"), (kv8.rows_v, "v")))
            assert np.array_equal(k[:, :n], self.codes[page][:, :n]) and np.array_equal(v[:, :n], self.codes[page][:, :n])
            assert np.array_equal(cache["k_scale"][page].cpu().numpy(), self.scale[page])
            want = self.codes[page].astype(np.float32) * self.scale[page][:, None, None]
            for got in w4.kv8_dequant(cache, ints([page]), TDT[dtype]):
                assert torch.equal(got[0, :, :n].cpu(), torch.from_numpy(want[:, :n]).to(TDT[dtype]))


def rows_of(r, n, Hkv, D, dtype, size=1.0):
    return torch.from_numpy(size * r.randn(n, Hkv, D)).to(TDT[dtype])


@pytest.mark.parametrize("T,Hkv,D,dtype", [(16, 2, 64, "f16"), (32, 1, 128, "bf16"), (64, 3, 64, "bf16"), (128, 2, 128, "f16")])
def test_drafts_leave_the_scale_and_codes_they_made(T, Hkv, D, dtype):
    """Lengths that end inside a page, at its end and pages back; drafts larger and
    smaller than what is there."""
    say("drops", T, Hkv, D, dtype)
    r = np.random.RandomState(T + D)
    cache, refs = w4.kv8_cache(12, T, Hkv, D, DEV), w4.kv8_refs(12)
    table, lens = torch.full((1, 6), -1, dtype=torch.int32, device=DEV), ints([0])
    want, length = Pages(12, T, Hkv, D), 0

    def grow(n, size):
        nonlocal length
        assert w4.kv8_reserve(refs, table, lens, ints([n]), T).tolist() == [0]
        x = rows_of(r, n, Hkv, D, dtype, size)
        w4.kv8_append(cache, x.to(DEV), x.to(DEV), table, lens, ints([0, n]), n)
        want.append(table[0].tolist(), length, x.float().numpy())
        length += n

    def drop(n):
        nonlocal length
        assert w4.kv8_reserve(refs, table, lens, ints([-n]), T).tolist() == [0]
        length -= n

    for kept, size, drafted, big, back in ((T // 2 + 1, 1.0, 3, 9.0, 3), (5, 1.0, T, 30.0, T), (T, 2.0, 2, 0.1, 1),
                                           (2 * T - length % T, 1.0, 7, 50.0, 7), (3, 1.0, 4, 200.0, 2)):
        grow(kept, size)
        want.check(cache, table[0].tolist(), length, dtype)
        before = want.scale.copy()
        grow(drafted, big)
        drop(back)
        # the page that the row ends in keeps the drafts' scale, its rows their coarser codes
        want.check(cache, table[0].tolist(), length, dtype)
        page = table[0].tolist()[max(length - 1, 0) // T]
        if big > size and length % T:
            assert np.all(want.scale[page] >= before[page])
        assert lens.tolist() == [length]


def test_a_drafted_nan_stays_with_its_page():
    T, Hkv, D = 16, 2, 64
    r = np.random.RandomState(3)
    cache, refs = w4.kv8_cache(4, T, Hkv, D, DEV), w4.kv8_refs(4)
    table, lens = torch.full((1, 3), -1, dtype=torch.int32, device=DEV), ints([0])

    def grow(x):
        assert w4.kv8_reserve(refs, table, lens, ints([len(x)]), T).tolist() == [0]
        w4.kv8_append(cache, x.to(DEV), x.to(DEV), table, lens, ints([0, len(x)]), len(x))

    grow(rows_of(r, 20, Hkv, D, "f16"))
    bad = rows_of(r, 14, Hkv, D, "f16")     # to token 34: the second page's rest and a third page
    bad[2, 1, 5] = float("nan")
    grow(bad)
    assert w4.kv8_reserve(refs, table, lens, ints([-14]), T).tolist() == [0]
    grow(rows_of(r, 1, Hkv, D, "f16"))
    k, _ = w4.kv8_dequant(cache, table[0, :2].contiguous(), torch.float16)
    assert torch.isfinite(k[0]).all() and torch.isfinite(k[1, 0, :5]).all() and torch.isnan(k[1, 1, :5]).all()
    # dropped to the page's beginning, it begins anew
    assert w4.kv8_reserve(refs, table, lens, ints([-5]), T).tolist() == [0]
    grow(rows_of(r, 3, Hkv, D, "f16"))
    k, _ = w4.kv8_dequant(cache, table[0, :2].contiguous(), torch.float16)
    assert torch.isfinite(k[0]).all() and torch.isfinite(k[1, :, :3]).all()


def test_drafts_on_a_fork_leave_the_row_as_it_was():
    T, Hkv, D = 16, 2, 64
    r = np.random.RandomState(4)
    caches, refs = [w4.kv8_cache(9, T, Hkv, D, DEV) for _ in range(2)], w4.kv8_refs(9)
    table, lens = torch.full((2, 4), -1, dtype=torch.int32, device=DEV), ints([0, 0])
    assert w4.kv8_reserve(refs, table, lens, ints([21, 0]), T).tolist() == [0]
    x = rows_of(r, 21, Hkv, D, "f16").to(DEV)
    for c in caches:
        w4.kv8_append(c, x, x, table[:1], lens[:1], ints([0, 21]), 21)
    pages = table[0, :2].tolist()
    was = [{n: c[n][pages].clone() for n in ("k", "v", "k_scale", "v_scale")} for c in caches]
    assert w4.kv8_fork(caches, refs, table, lens, ints([0]), ints([1])).tolist() == [0]
    assert w4.kv8_reserve(refs, table, lens, ints([0, 13]), T).tolist() == [0]
    x = rows_of(r, 13, Hkv, D, "f16", 40.0).to(DEV)
    x[1, 0, 0] = float("nan")
    for c in caches:
        w4.kv8_append(c, x, x, table, lens, ints([0, 0, 13]), 13)
    w4.kv8_free(refs, table, lens, ints([1]), T)
    assert lens.tolist() == [21, 0] and refs.sum().item() == 2
    for c, w in zip(caches, was):
        assert all(torch.equal(c[n][pages], t) for n, t in w.items())
