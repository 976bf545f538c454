"""Attention over the paged 8-bit cache with capped scores, distance bias,
document and prefix masks, against 64 bits: single tokens, drafted ones and
prompts, split and whole, rows that see nothing, and what masks hide."""

import math

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


def call(c, fn=None, **more):
    tokens, H, D = c["q"].shape
    lse = torch.full((tokens, H), 7.0, device=DEV)
    kw = dict(cu_seqlens=None if c["one"] else ints(c["cu"]), max_new=None if c["one"] else c["max_new"],
              max_len=max(c["lens"]), scale=c["scale"], causal=c["causal"], lse=lse, **more)
    o = (fn or w4.kv8_attention_scored)(c["q"], c["cache"], ints(c["table"]), ints(c["lens"]), **kw)
    return o, lse


def check(c, softcap=0.0, slopes=None, first=None, prefix=None):
    f32 = None if slopes is None else np.asarray(slopes, np.float32)
    o, lse = call(c, softcap=softcap, slopes=None if slopes is None else torch.from_numpy(f32).to(DEV),
                  first=None if first is None else ints(first), prefix=None if prefix is None else ints(prefix))
    cache = c["cache"]
    k = kv8.rows_k(cache["k"].cpu().numpy()) * cache["k_scale"].cpu().numpy().astype(np.float64)[:, :, None, None]
    v = kv8.rows_v(cache["v"].cpu().numpy()) * cache["v_scale"].cpu().numpy().astype(np.float64)[:, :, None, None]
    want, wlse, bound, lb = kv8.attention_scored(
        c["q"].double().cpu().numpy(), k, v, c["table"].tolist(), c["lens"], c["cu"], c["T"], c["scale"], c["causal"],
        softcap, None if f32 is None else f32.astype(np.float64), first, prefix, (0.025 / 0.005))
    bound = kv8.rounded_bound(bound, want, c["dtype"])
    err = np.abs(o.double().cpu().numpy() - want)
    assert np.all(err <= bound), (np.max(err / bound), np.argwhere(~(err <= bound))[:4], softcap)
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), np.isneginf(wlse))
    fine = np.isfinite(wlse)
    err = np.abs(got[fine] - wlse[fine])
    assert np.all(err <= lb[fine]), np.max(err / lb[fine])
    return o


def slopes_of(H, top=0.5):
    return top * 2.0 ** (-8.0 * np.arange(H) / H)


def starts(c, mean):
    """Starts of documents of random lengths, for every new token."""
    got = []
    for L, n in zip(c["lens"], np.diff(c["cu"])):
        cuts = [0]
        while cuts[-1] < L:
            cuts.append(cuts[-1] + 1 + int(c["r"].rand() * 2 * mean))
        got += [max(s for s in cuts if s <= max(p, 0)) for p in range(L - n, L)]
    return got


SHAPES = [
    # lens, new tokens, H, Hkv, D, T
    ([1], [1], 1, 1, 64, 16),
    ([16, 17, 63], [1, 1, 1], 4, 2, 128, 16),
    ([5, 64, 65, 700], [1, 1, 1, 1], 10, 2, 128, 64),
    ([2000, 1, 900], [1, 1, 1], 8, 4, 64, 32),              # keys split over workgroups
    ([40, 129, 7], [5, 3, 0], 8, 8, 64, 32),
    ([300, 61], [11, 9], 6, 2, 128, 128),
    ([70, 200, 64, 0], [70, 5, 64, 0], 12, 4, 128, 64),      # prompts
    ([333, 120], [150, 33], 5, 1, 64, 16),
    ([1500], [140], 2, 1, 128, 128),                         # prompts, keys split
    ([700, 650], [131, 129], 4, 2, 64, 64),
]
MODES = ["cap", "slopes", "documents", "prefix", "all"]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_every_shape(i, mode):
    lens, news, H, Hkv, D, T = SHAPES[i]
    dtype = ("f16", "bf16")[(i + MODES.index(mode)) % 2]
    say("scored", lens, news, H, Hkv, D, T, mode, dtype)
    c = case(i, lens, news, H, Hkv, D, T, dtype, size=2.0)
    some = [L - n + int(0.6 * n) for L, n in zip(lens, news)]
    check(c, softcap=15.0 if mode in ("cap", "all") else 0.0, slopes=slopes_of(H) if mode in ("slopes", "all") else None,
          first=starts(c, 40) if mode in ("documents", "all") else None, prefix=some if mode in ("prefix", "all") else None)


@pytest.mark.parametrize("softcap", [1e-3, 0.5, 30.0, 349.0, 400.0, 5e3, 1e6, 1e30])
def test_caps(softcap):
    for shape, dtype in (([90, 200], [1, 1], 4, 2, 64, 16), "f16"), (([260], [140], 2, 2, 128, 64), "bf16"):
        c = case(20, *shape, dtype, size=4.0)
        check(c, softcap=softcap)
        c["q"] *= 20
        check(c, softcap=softcap)


@pytest.mark.parametrize("causal", [True, False])
def test_slopes_up_and_down(causal):
    """Steep, negative and absent slopes, both ways and far back."""
    for shape in (([3000, 40], [1, 1], 4, 2, 64, 32), ([600, 31], [150, 31], 4, 2, 64, 64)):
        c = case(21, *shape, "f16")
        c["causal"] = causal
        check(c, slopes=[2.0, 0.0, -0.01, 0.03])
        check(c, slopes=[8.0, 1e-4, 0.25, -0.02], softcap=5.0, prefix=[shape[0][0] // 2, 40])


def test_rows_that_see_nothing():
    for news, lens in (([1, 1, 1], [30, 200, 1]), ([6, 40, 3], [30, 200, 2]), ([70, 60, 90], [130, 200, 90])):
        c = case(22, lens, news, 4, 1, 128, 16, "f16")
        n = int(c["cu"][-1])
        # from the query on, after it, past everything, before everything; all of the second sequence hidden
        first = [[0, 10 ** 9, -5, 29, 31, 2 ** 31 - 1, -(2 ** 31)][t % 7] for t in range(n)]
        first[c["cu"][1]:c["cu"][2]] = [10 ** 6] * int(news[1])
        check(c, first=first, slopes=slopes_of(4), softcap=20.0)
        c["causal"] = False
        check(c, first=first)


def test_prefixes_of_any_length():
    c = case(23, [100, 64, 200, 5], [50, 64, 3, 5], 4, 2, 64, 32, "bf16")
    for prefix in ([0, 1, 199, 5], [-7, 64, 1000, 2], [75, 32, 198, 2 ** 31 - 1]):
        check(c, prefix=prefix)
        check(c, prefix=prefix, first=starts(c, 30), slopes=slopes_of(4))


@pytest.mark.parametrize("new", [1, 7, 80])
def test_more_new_tokens_than_the_sequence_has(new):
    """Tokens at negative positions see nothing, with a prefix too."""
    c = case(24, [max(new - 3, 0), new + 20], [new, new], 2, 2, 64, 16, "f16")
    check(c, prefix=[50, 5], first=[0] * (2 * new), slopes=slopes_of(2))


@pytest.mark.parametrize("news", [[1, 1], [5, 5], [90, 70]])
def test_hidden_pages_do_not_matter(news):
    """NaN and infinite scales of pages that no query sees."""
    T = 16
    c = case(25, [250, 333], news, 8, 2, 64, T, "f16")
    first = [100] * news[0] + [147] * news[1]      # in the middle of pages and units
    a = check(c, first=first, slopes=slopes_of(8), softcap=9.0)
    for b, f in ((0, 100), (1, 147)):
        for p in c["table"][b, :f // T]:
            c["cache"]["k_scale"][int(p)] = float("nan") if p % 2 else float("inf")
            c["cache"]["v_scale"][int(p)] = float("nan") if p % 3 else float("inf")
    o, _ = call(c, first=ints(first), slopes=torch.from_numpy(slopes_of(8).astype(np.float32)).to(DEV), softcap=9.0)
    assert torch.equal(o, a)


def test_windows_over_a_long_context():
    """Only what is seen is read: splits follow it."""
    c = case(26, [20000, 9000], [1, 1], 8, 1, 128, 64, "bf16")
    check(c, first=[20000 - 1024, 9000 - 100], softcap=30.0)
    check(c, first=[0, 8999])
    c = case(27, [4000], [130], 2, 1, 64, 64, "f16")
    check(c, first=[p - 255 for p in range(3870, 4000)])


def test_scores_far_out():
    """Large scores and bias: the maximum leaves the range of one fma."""
    c = case(28, [500, 77], [1, 1], 4, 2, 64, 32, "f16", size=300.0)
    check(c, slopes=slopes_of(4, 30.0))
    c = case(29, [300], [130], 2, 2, 128, 64, "bf16", size=1000.0)
    check(c, slopes=[5.0, 100.0])
    check(c, slopes=[5.0, 100.0], softcap=1e5)


@pytest.mark.parametrize("news", [[1, 1, 1], [4, 1, 9], [140, 1, 60]])
def test_nothing_set_is_plain_attention(news):
    c = case(30, [300, 50, 777], news, 8, 2, 128, 64, "f16")
    o, lse = call(c)
    p, plse = call(c, w4.kv8_attention)
    # both are within the same bounds of the exact result; probabilities are formed alike but for one rounding
    assert torch.allclose(o.float(), p.float(), rtol=2e-3, atol=2e-3) and torch.allclose(lse, plse, rtol=1e-5, atol=1e-5)
    again, _ = call(c)
    assert torch.equal(o, again)


def test_max_new_and_rows_behind():
    """Rows past max_new and rows of no sequence keep what they hold."""
    c = case(31, [90, 40], [6, 3], 4, 2, 64, 16, "f16")
    q = torch.cat([c["q"], c["q"][:4]])
    out, lse = torch.full_like(q, 5.0), torch.full((13, 4), 5.0, device=DEV)
    kw = dict(cu_seqlens=ints(c["cu"]), max_new=4, max_len=90, softcap=10.0, first=ints([3] * 13))
    w4.kv8_attention_scored(q, c["cache"], ints(c["table"]), ints(c["lens"]), out=out, lse=lse, **kw)
    rows = [4, 5, 9, 10, 11, 12]
    assert (out[rows] == 5).all() and (lse[rows] == 5).all()
    assert (out[[0, 1, 2, 3, 6, 7, 8]] != 5).any(-1).all()


@pytest.mark.parametrize("new", [1, 130])
def test_captured_in_a_graph(new):
    c = case(32, [1500, 900], [new, new], 4, 1, 64, 32, "bf16")
    q, table, lens, cu = c["q"], ints(c["table"]), ints(c["lens"]), ints(c["cu"])
    first, prefix = ints(starts(c, 300)), ints([1450, 0])
    slopes = torch.from_numpy(slopes_of(4).astype(np.float32)).to(DEV)
    space = w4.workspace(w4.kv8_attention_workspace_bytes(2 * new, 2, new, 1500, 4, 1, 64), DEV)
    assert space is not None
    kw = dict(cu_seqlens=cu, max_new=new, max_len=1500, softcap=20.0, slopes=slopes, first=first, prefix=prefix)
    out = torch.empty_like(q)
    w4.kv8_attention_scored(q, c["cache"], table, lens, out=out, workspace=space, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.kv8_attention_scored(q, c["cache"], table, lens, out=out, workspace=space, **kw)
    for i in range(4):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(i)))
        first += 3
        lens -= 1
        want = w4.kv8_attention_scored(q, c["cache"], table, lens, **kw)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_on_another_stream_and_strided_rows():
    c = case(33, [200, 90], [1, 1], 4, 2, 128, 64, "f16")
    rows = torch.zeros(2, 8, 128, dtype=torch.float16, device=DEV)
    rows[:, 2:6] = c["q"]
    table, lens, first = ints(c["table"]), ints(c["lens"]), ints([17, 60])
    out = torch.zeros(2, 6, 128, dtype=torch.float16, device=DEV)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    w4.kv8_attention_scored(rows[:, 2:6], c["cache"], table, lens, first=first, softcap=3.0, out=out[:, 1:5], stream=st)
    st.synchronize()
    want = w4.kv8_attention_scored(c["q"], c["cache"], table, lens, first=first, softcap=3.0)
    assert torch.equal(out[:, 1:5], want) and not out[:, 0].any() and not out[:, 5].any()


def test_refusals():
    c = case(34, [20, 30], [1, 1], 4, 2, 64, 16, "f16")
    q, cache, table, lens = c["q"], c["cache"], ints(c["table"]), ints(c["lens"])
    for bad in (-1.0, 1e-9, 1e31, float("inf"), float("nan")):
        with pytest.raises(w4.W4A16Error, match="status 1"):
            w4.kv8_attention_scored(q, cache, table, lens, softcap=bad)
    with pytest.raises(ValueError):
        w4.kv8_attention_scored(q, cache, table, lens, slopes=torch.zeros(3, device=DEV))
    with pytest.raises(TypeError):
        w4.kv8_attention_scored(q, cache, table, lens, slopes=torch.zeros(4, device=DEV).half())
    with pytest.raises(ValueError):
        w4.kv8_attention_scored(q, cache, table, lens, first=ints([0]))
    with pytest.raises(TypeError):
        w4.kv8_attention_scored(q, cache, table, lens, first=torch.zeros(2, dtype=torch.int64, device=DEV))
    with pytest.raises(TypeError):
        w4.kv8_attention_scored(q, cache, table, lens, prefix=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        w4.kv8_attention_scored(q, cache, table, lens, prefix=ints([0, 1, 2]))
    with pytest.raises(ValueError):
        w4.kv8_attention_scored(q[:, :, :32], cache, table, lens)
    with pytest.raises(ValueError):
        w4.kv8_attention_scored(q[0], cache, table, lens)
    with pytest.raises(TypeError):
        w4.kv8_attention_scored(q, cache, table, lens.tolist())
    none = q[:0]
    assert w4.kv8_attention_scored(none, cache, table[:0], lens[:0], softcap=3.0).shape == (0, 4, 64)
    assert math.isfinite(w4.kv8_attention_scored(q, cache, table, lens, softcap=None).float().sum().item())


def test_workspace_of_both_attentions():
    """One workspace for plain and scored calls in turn, split and not."""
    space = None
    for seed, (lens, news) in enumerate((([3000], [1]), ([2500, 100], [1, 1]), ([1500], [140]), ([2000], [3]))):
        c = case(40 + seed, lens, news, 4, 1, 64, 32, "f16")
        tokens = int(c["cu"][-1])
        need = w4.kv8_attention_workspace_bytes(tokens, len(lens), max(news), max(lens), 4, 1, 64)
        if space is None or space.numel() * 4 < need:
            space = w4.workspace(max(need, 1 << 22), DEV)
        slopes = torch.from_numpy(slopes_of(4).astype(np.float32)).to(DEV)
        for _ in range(2):
            a, _ = call(c, workspace=space, softcap=9.0, slopes=slopes)
            p, _ = call(c, w4.kv8_attention, workspace=space)
        assert torch.equal(a, call(c, softcap=9.0, slopes=slopes)[0])
        assert torch.equal(p, call(c, w4.kv8_attention)[0])


def test_two_streams_at_once():
    c = case(50, [3000, 900], [1, 1], 8, 2, 128, 64, "bf16")
    q, table, lens = c["q"], ints(c["table"]), ints(c["lens"])
    want = [w4.kv8_attention_scored(q * (i + 1), c["cache"], table, lens, softcap=10.0 + i) for i in range(2)]
    streams, xs = [torch.cuda.Stream() for _ in range(2)], [q * (i + 1) for i in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            got[i].append(w4.kv8_attention_scored(xs[i], c["cache"], table, lens, softcap=10.0 + i, stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])


@pytest.mark.parametrize("lens,news", [([201, 77], [1, 1]), ([201, 330], [140, 1])])
def test_unused_rows_of_a_page_do_not_show(lens, news):
    """Codes past a sequence's end, and before every query's first key, change no bit."""
    for T in (16, 64):
        c = case(60, lens, news, 4, 2, 64, T, "f16", size=0.5)
        first = [70] * int(c["cu"][-1])
        kw = dict(softcap=20.0, first=ints(first))
        a, lse = call(c, **kw)
        for b, L in enumerate(lens):
            for p in range(-(-L // T)):
                page = int(c["table"][b, p])
                rows = [t for t in range(T) if not 70 <= p * T + t < L]
                c["cache"]["k"][page][:, rows] = 255          # large scores, if they were seen
                for t in rows:
                    c["cache"]["v"][page][:, t // 16, :, t % 16] = 255
        b, lse2 = call(c, **kw)
        assert torch.equal(a, b) and torch.equal(lse, lse2)
