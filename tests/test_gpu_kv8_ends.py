"""Attention over the paged 8-bit cache where each query's keys have an end:
documents that share a sequence, seen both ways or up to a prefix, against 64
bits; ends in any order, rows that see nothing, and pages that ends hide."""

import numpy as np
import pytest
import torch

import bit_weight_only_gemm_amd as w4
from gpu_util import DEV, TDT, say
from oracle import kv8

pytestmark = pytest.mark.gpu


def case(seed, lens, news, H, Hkv, D, T, dtype, size=1.0):
    r = np.random.RandomState(seed)
    counts = [max(1, -(-L // T)) for L in lens]
    pages, width = sum(counts) + 2, max(counts) + 1
    order, at = r.permutation(pages), 0
    table = np.where(r.rand(len(lens), width) < 0.5, -1, 1 << 29).astype(np.int32)
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    cache = w4.kv8_cache(pages, T, Hkv, D, DEV)
    for n in ("k", "v"):
        cache[n].copy_(torch.from_numpy(r.randint(1, 256, cache[n].shape).astype(np.uint8)))
    for n in ("k_scale", "v_scale"):
        cache[n].copy_(torch.from_numpy((r.rand(pages, Hkv) * 0.02 + 0.005).astype(np.float32)))
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    q = torch.from_numpy(size * r.randn(int(cu[-1]), H, D)).to(TDT[dtype]).to(DEV)
    return {"cache": cache, "table": table, "lens": list(lens), "cu": cu, "q": q, "T": T, "D": D, "H": H, "r": r,
            "dtype": dtype, "one": all(n == 1 for n in news), "max_new": max(news), "scale": D ** -0.5, "causal": True}


def ints(v):
    return torch.tensor(np.asarray(v, np.int64).astype(np.int32), device=DEV)


def call(c, **more):
    tokens, H, D = c["q"].shape
    lse = torch.full((tokens, H), 7.0, device=DEV)
    kw = dict(cu_seqlens=None if c["one"] else ints(c["cu"]), max_new=None if c["one"] else c["max_new"],
              max_len=max(c["lens"]), scale=c["scale"], causal=c["causal"], lse=lse)
    kw.update({n: ints(t) if n in ("first", "end", "prefix") and t is not None else t for n, t in more.items()})
    return w4.kv8_attention_scored(c["q"], c["cache"], ints(c["table"]), ints(c["lens"]), **kw), lse


def check(c, softcap=0.0, slopes=None, first=None, prefix=None, end=None):
    f32 = None if slopes is None else np.asarray(slopes, np.float32)
    o, lse = call(c, softcap=softcap, slopes=None if f32 is None else torch.from_numpy(f32).to(DEV), first=first,
                  prefix=prefix, end=end)
    cache = c["cache"]
    k = kv8.rows_k(cache["k"].cpu().numpy()) * cache["k_scale"].cpu().numpy().astype(np.float64)[:, :, None, None]
    v = kv8.rows_v(cache["v"].cpu().numpy()) * cache["v_scale"].cpu().numpy().astype(np.float64)[:, :, None, None]
    want, wlse, bound, lb = kv8.attention_scored(
        c["q"].double().cpu().numpy(), k, v, c["table"].tolist(), c["lens"], c["cu"], c["T"], c["scale"], c["causal"],
        softcap, None if f32 is None else f32.astype(np.float64), first, prefix, (0.025 / 0.005), end)
    bound = kv8.rounded_bound(bound, want, c["dtype"])
    err = np.abs(o.double().cpu().numpy() - want)
    assert np.all(err <= bound), (np.max(err / bound), np.argwhere(~(err <= bound))[:4])
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), np.isneginf(wlse))
    fine = np.isfinite(wlse)
    err = np.abs(got[fine] - wlse[fine])
    assert np.all(err <= lb[fine]), np.max(err / lb[fine])
    return o, lse


def slopes_of(H, top=0.5):
    return top * 2.0 ** (-8.0 * np.arange(H) / H)


def documents(c, mean):
    """Starts and ends of documents of random lengths, for every new token."""
    first, end = [], []
    for L, n in zip(c["lens"], np.diff(c["cu"])):
        cuts = [0]
        while cuts[-1] < L:
            cuts.append(cuts[-1] + 1 + int(c["r"].rand() * 2 * mean))
        for p in range(L - n, L):
            i = max(j for j, s in enumerate(cuts) if s <= max(p, 0))
            first.append(cuts[i])
            end.append(cuts[i + 1] if i + 1 < len(cuts) else L)
    return first, end


SHAPES = [
    # lens, new tokens, H, Hkv, D, T
    ([1], [1], 1, 1, 64, 16),
    ([16, 17, 63], [1, 1, 1], 4, 2, 128, 16),
    ([2000, 1, 900], [1, 1, 1], 8, 4, 64, 32),              # keys split over workgroups
    ([40, 129, 7], [5, 3, 0], 8, 8, 64, 32),
    ([300, 61], [11, 9], 6, 2, 128, 128),
    ([2500, 61], [16, 16], 4, 2, 64, 64),
    ([70, 200, 64, 0], [70, 5, 64, 0], 12, 4, 128, 64),      # prompts
    ([333, 120], [150, 33], 5, 1, 64, 16),
    ([1500], [140], 2, 1, 128, 128),                         # prompts, keys split
    ([700, 650], [131, 650], 4, 2, 64, 64),
    ([900, 300], [900, 300], 2, 1, 128, 32),
]


@pytest.mark.parametrize("mode", ["prefix", "both ways", "all"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_documents(i, mode):
    lens, news, H, Hkv, D, T = SHAPES[i]
    dtype = ("f16", "bf16")[(i + len(mode)) % 2]
    say("documents", lens, news, H, Hkv, D, T, mode, dtype)
    c = case(i, lens, news, H, Hkv, D, T, dtype, size=2.0)
    c["causal"] = mode != "both ways"
    first, end = documents(c, (40, 200)[i % 2])
    some = [L - n + int(0.6 * n) for L, n in zip(lens, news)]
    check(c, first=first, end=end, prefix=None if mode == "both ways" else some,
          softcap=15.0 if mode == "all" else 0.0, slopes=slopes_of(H) if mode == "all" else None)


@pytest.mark.parametrize("news,lens", [([1, 1, 1], [30, 200, 1]), ([6, 16, 3], [30, 200, 2]), ([70, 60, 90], [130, 200, 90])])
def test_ends_in_any_order(news, lens):
    """Before the first key, at it, far out; of rows in one tile without order; all of one sequence hidden."""
    c = case(22, lens, news, 4, 1, 128, 16, "f16")
    n = int(c["cu"][-1])
    end = [[5, 10 ** 9, -5, 29, 0, 2 ** 31 - 1, -(2 ** 31), 17, 1][t % 9] for t in range(n)]
    first = [[0, 3, 20, 29, 10 ** 6][t % 5] for t in range(n)]
    for causal in (True, False):
        c["causal"] = causal
        check(c, end=end)
        check(c, end=end, first=first, slopes=slopes_of(4), softcap=20.0)
        check(c, end=end, prefix=[25, 64, 7])
        hidden = list(end)
        hidden[c["cu"][1]:c["cu"][2]] = [-1] * int(news[1])
        o, lse = check(c, end=hidden, first=first)
        rows = slice(int(c["cu"][1]), int(c["cu"][2]))
        assert not o[rows].any() and torch.isneginf(lse[rows]).all()


@pytest.mark.parametrize("new", [1, 16, 130])
def test_an_end_past_the_keys_changes_no_bit(new):
    for T in (16, 64):
        c = case(23, [900, 333], [new, new], 4, 2, 64, T, "bf16")
        first = [100] * (2 * new)
        for kw in (dict(), dict(first=first, prefix=[890, 0], softcap=9.0, slopes=torch.full((4,), 0.01, device=DEV))):
            a, la = call(c, **kw)
            b, lb = call(c, **kw, end=[900] * new + [2 ** 31 - 1] * new)
            assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("news", [[1, 1], [5, 5], [90, 170]])
@pytest.mark.parametrize("T", [16, 64])
def test_hidden_pages_do_not_matter(news, T):
    """NaN and infinite scales of pages from every query's end on."""
    c = case(25, [450, 333], news, 8, 2, 64, T, "f16")
    c["causal"] = False
    end = [200] * news[0] + [147] * news[1]        # in the middle of units
    slopes = torch.from_numpy(slopes_of(8).astype(np.float32)).to(DEV)
    kw = dict(end=end, slopes=slopes, softcap=9.0)
    a, la = call(c, **kw)
    for b, e in ((0, 200), (1, 147)):
        for p in c["table"][b, -(-e // T):-(-c["lens"][b] // T)]:
            c["cache"]["k_scale"][int(p)] = float("nan") if p % 2 else float("inf")
            c["cache"]["v_scale"][int(p)] = float("nan") if p % 3 else float("inf")
    o, lse = call(c, **kw)
    assert torch.equal(o, a) and torch.equal(lse, la)


def test_documents_are_apart():
    """Keys and values of other documents change no bit of a document's rows."""
    c = case(26, [640], [640], 4, 2, 64, 64, "f16")
    cuts = [0, 100, 320, 640]
    doc = np.searchsorted(cuts, np.arange(640), side="right") - 1
    first, end = [cuts[d] for d in doc], [cuts[d + 1] for d in doc]
    for kw in (dict(prefix=[500]), dict(causal=False)):
        c["causal"] = kw.get("causal", True)
        more = dict(first=first, end=end, prefix=kw.get("prefix"))
        a, _ = call(c, **more)
        saved = {n: c["cache"][n].clone() for n in ("k", "v")}
        for p in range(5, 10):                     # the last document's pages
            page = int(c["table"][0, p])
            c["cache"]["k"][page] = 255
            c["cache"]["v"][page] = 1
        b, _ = call(c, **more)
        assert torch.equal(a[:320], b[:320]) and not torch.equal(a[320:], b[320:])
        for n, t in saved.items():
            c["cache"][n].copy_(t)


@pytest.mark.parametrize("new", [1, 130])
def test_captured_in_a_graph(new):
    c = case(32, [1500, 900], [new, new], 4, 1, 64, 32, "bf16")
    q, table, lens, cu = c["q"], ints(c["table"]), ints(c["lens"]), ints(c["cu"])
    first, end = (ints(t) for t in documents(c, 300))
    space = w4.workspace(w4.kv8_attention_workspace_bytes(2 * new, 2, new, 1500, 4, 1, 64), DEV)
    kw = dict(cu_seqlens=cu, max_new=new, max_len=1500, causal=False, first=first, end=end)
    out = torch.empty_like(q)
    w4.kv8_attention_scored(q, c["cache"], table, lens, out=out, workspace=space, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.kv8_attention_scored(q, c["cache"], table, lens, out=out, workspace=space, **kw)
    for i in range(4):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(i)))
        first += 3
        end -= 5
        want = w4.kv8_attention_scored(q, c["cache"], table, lens, **kw)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals():
    c = case(34, [20, 30], [1, 1], 4, 2, 64, 16, "f16")
    q, cache, table, lens = c["q"], c["cache"], ints(c["table"]), ints(c["lens"])
    with pytest.raises(ValueError):
        w4.kv8_attention_scored(q, cache, table, lens, end=ints([0]))
    with pytest.raises(TypeError):
        w4.kv8_attention_scored(q, cache, table, lens, end=torch.zeros(2, dtype=torch.int64, device=DEV))
    with pytest.raises(TypeError):
        w4.kv8_attention_scored(q, cache, table, lens, end=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(w4.W4A16Error, match="status 1"):
        w4.kv8_attention_scored(q, cache, table, lens, end=ints([1, 1]), softcap=-1.0)
    none = q[:0]
    assert w4.kv8_attention_scored(none, cache, table[:0], lens[:0], end=ints([])).shape == (0, 4, 64)
