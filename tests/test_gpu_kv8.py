"""The paged 8-bit cache on the GPU: append with rotation and read-back
against the formula (bit for bit in fp32, and in 64 bits), attention against
64-bit softmax over the cache's values, at the sizes and masks where it can go
wrong."""

import math

import numpy as np
import pytest
import torch

import bit_weight_only_gemm_amd as w4
from oracle import kv8
from gpu_util import DEV, TDT, say

pytestmark = pytest.mark.gpu
INV = np.float32(1 / 127)


def _case(seed, lens, news, H, Hkv, D, T, dtype, spare=2):
    """Sequences over a shuffled page pool; unused table entries are -1 or far
    out of range."""
    r = np.random.RandomState(seed)
    counts = [max(1, -(-L // T)) for L in lens]
    pages, width = sum(counts) + spare, max(counts) + 1
    order = r.permutation(pages)
    table = np.where(r.rand(len(lens), width) < 0.5, -1, 1 << 29).astype(np.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    cache = w4.kv8_cache(pages, T, Hkv, D, DEV)
    cache["k"].copy_(torch.from_numpy(r.randint(0, 256, cache["k"].shape).astype(np.uint8)))
    cache["v"].copy_(torch.from_numpy(r.randint(0, 256, cache["v"].shape).astype(np.uint8)))
    cache["k_scale"].copy_(torch.from_numpy((r.rand(pages, Hkv) * 0.02 + 0.005).astype(np.float32)))
    cache["v_scale"].copy_(torch.from_numpy((r.rand(pages, Hkv) * 0.02 + 0.005).astype(np.float32)))
    tokens = sum(news)
    mk = lambda h: torch.from_numpy(r.randn(tokens, h, D)).to(TDT[dtype]).to(DEV)  # noqa: E731
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    return {"cache": cache, "table": table, "lens": list(lens), "cu": cu, "q": mk(H), "k": mk(Hkv),
            "v": mk(Hkv), "T": T, "r": r,
            "dev": {"table": torch.from_numpy(table).to(DEV), "cu": torch.from_numpy(cu).to(DEV),
                    "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}}


def _rope(positions, dim):
    a = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, dim, 2) / dim)
    return (torch.from_numpy(f(a).astype(np.float32)).to(DEV) for f in (np.cos, np.sin))


def _np(c):
    cache = c["cache"]
    return {"k": kv8.rows_k(cache["k"].cpu().numpy()), "v": kv8.rows_v(cache["v"].cpu().numpy()),
            "ks": cache["k_scale"].cpu().numpy().copy(), "vs": cache["v_scale"].cpu().numpy().copy()}


def _rotate32(x, cos, sin, pos, interleaved):
    """The kernel's fp32 operations, each rounded once."""
    half = cos.shape[1]
    a = np.arange(half) * 2 if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    c, s = cos[pos][:, None, :], sin[pos][:, None, :]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _positions(c):
    return np.concatenate([np.arange(L - n, L) for L, n in zip(c["lens"], np.diff(c["cu"]))])


APPENDS = [
    # lens (after), new tokens, H, Hkv, D, T
    ([1], [1], 1, 1, 64, 16),
    ([16, 17, 33], [1, 1, 1], 4, 2, 128, 16),
    ([5, 64, 65, 200], [1, 1, 1, 1], 10, 2, 128, 64),
    ([40, 129, 7], [40, 3, 0], 8, 8, 64, 32),
    ([100, 300], [37, 299], 5, 1, 128, 128),
    ([70, 200, 64, 0], [70, 5, 64, 0], 8, 4, 128, 64),
    ([31, 47], [16, 31], 16, 2, 64, 128),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,news,H,Hkv,D,T", APPENDS)
@pytest.mark.parametrize("form", ["half", "pairs", "part", "none"])
def test_append(lens, news, H, Hkv, D, T, dtype, form):
    say("append", lens, news, H, Hkv, D, T, dtype, form)
    c = _case(len(lens) + T, lens, news, H, Hkv, D, T, dtype)
    before = _np(c)
    dim = {"half": D, "pairs": D, "part": D // 2, "none": D}[form]
    cos, sin = _rope(max(lens) + 3, dim)
    inter = form == "pairs"
    rope = {} if form == "none" else {"cos": cos, "sin": sin, "interleaved": inter}
    one = all(n == 1 for n in news)
    args = dict(cu_seqlens=None if one else c["dev"]["cu"], max_new=max(news), **rope)
    # rows of one fused buffer
    qkv = torch.cat([c["q"], c["k"], c["v"]], 1).flatten(1)
    q, k, v = (t.view(len(qkv), -1, D) for t in qkv.split([H * D, Hkv * D, Hkv * D], 1))
    got_q = w4.kv8_append(c["cache"], k, v, c["dev"]["table"], c["dev"]["lens"], q=q, **args)
    after = _np(c)
    pos = _positions(c)
    cn, sn = cos.cpu().numpy(), sin.cpu().numpy()
    f = {n: c[n].float().cpu().numpy() for n in "qkv"}
    if form != "none":
        want_q = torch.from_numpy(_rotate32(f["q"], cn, sn, pos, inter)).to(TDT[dtype])
        assert torch.equal(got_q.cpu(), want_q)
        k32 = _rotate32(f["k"], cn, sn, pos, inter)
        k64 = kv8.rotate(f["k"], cn, sn, pos, inter)
    else:
        assert torch.equal(got_q, c["q"])
        k32, k64 = f["k"], f["k"].astype(np.float64)
    untouched = {n: np.ones(before[n].shape[:1], bool) for n in ("k", "v")}
    for b, page, lo, hi, t0 in kv8.append_pages(c["table"], c["lens"], c["cu"], T):
        for name, x32, x64 in (("k", k32, k64), ("v", f["v"], f["v"].astype(np.float64))):
            untouched[name][page] = False
            rows32 = x32[t0:t0 + hi - lo].transpose(1, 0, 2)
            rows64 = x64[t0:t0 + hi - lo].transpose(1, 0, 2)
            old = before[name + "s"][page] if lo else np.zeros(Hkv, np.float32)
            s = np.maximum(old, np.abs(rows32).max((1, 2)) * INV)
            assert np.array_equal(after[name + "s"][page], s)
            codes = after[name][page]
            want = np.clip(np.rint(rows32 / s[:, None, None]), -127, 127)
            assert np.array_equal(codes[:, lo:hi], want)
            # 64 bits: half a step, and what the fp32 rotation, scale and quotient are off by
            s64 = np.maximum(old.astype(np.float64), np.abs(rows64).max((1, 2)) / 127)
            assert np.all(np.abs(rows64 / s64[:, None, None] - codes[:, lo:hi]) <= 0.5 + 2.0 ** -13)
            assert np.array_equal(codes[:, hi:], before[name][page][:, hi:])
            ratio = (old / s)[:, None, None]
            want = before[name][page][:, :lo]
            want = np.where(ratio == 1, want, np.clip(np.rint(want.astype(np.float32) * ratio), -128, 127))
            assert np.array_equal(codes[:, :lo], want)
    for name in ("k", "v"):
        assert np.array_equal(after[name][untouched[name]], before[name][untouched[name]])
        assert np.array_equal(after[name + "s"][untouched[name]], before[name + "s"][untouched[name]])
    # the same rows again change nothing
    w4.kv8_append(c["cache"], k, v, c["dev"]["table"], c["dev"]["lens"], **args)
    again = _np(c)
    assert all(np.array_equal(again[n], after[n]) for n in again)


def test_append_grows_a_page_token_by_token_and_reads_back():
    """A page filled one token at a time with growing rows: every step's
    older rows are requantized, and the values stay within a step of the rows
    for each time the scale grew."""
    T, D, Hkv = 32, 64, 2
    cache = w4.kv8_cache(3, T, Hkv, D, DEV)
    r = np.random.RandomState(0)
    x = torch.from_numpy(r.randn(T, Hkv, D) * np.linspace(0.1, 3, T)[:, None, None]).half().to(DEV)
    table = torch.tensor([[2]], dtype=torch.int32, device=DEV)
    grew, last = torch.zeros(Hkv, device=DEV), torch.zeros(Hkv, device=DEV)
    for t in range(T):
        w4.kv8_append(cache, x[t:t + 1], x[t:t + 1], table,
                      torch.tensor([t + 1], dtype=torch.int32, device=DEV))
        grew += (cache["k_scale"][2] > last).float()
        last = cache["k_scale"][2].clone()
    k, v = w4.kv8_dequant(cache, torch.tensor([2], dtype=torch.int32, device=DEV), torch.float16)
    assert torch.equal(k, v) and torch.equal(cache["k_scale"], cache["v_scale"])
    err = (k[0].float() - x.transpose(0, 1).float()).abs().amax((1, 2))
    step = cache["k_scale"][2]
    # each quantization is half a step of its time off, and no step is above the last
    assert torch.all(err <= 0.5 * (grew + 1) * step + 2.0 ** -10 * 127 * step)
    full = (x.float().abs().amax((0, 2)) * INV)
    assert torch.equal(step, full)


def test_append_zeros_nonfinite_and_reused_pages():
    T, D = 16, 64
    cache = w4.kv8_cache(4, T, 1, D, DEV)
    lens = lambda n: torch.tensor([n], dtype=torch.int32, device=DEV)  # noqa: E731
    table = torch.tensor([[1, 3]], dtype=torch.int32, device=DEV)
    zero = torch.zeros(1, 1, D, dtype=torch.bfloat16, device=DEV)
    row = torch.linspace(-1, 1, D, device=DEV).bfloat16().view(1, 1, D)
    w4.kv8_append(cache, zero, zero, table, lens(1))
    assert cache["k_scale"][1, 0] == 0 and torch.all(cache["k"][1, 0, 0] == 128)
    w4.kv8_append(cache, row, row, table, lens(2))
    assert cache["k_scale"][1, 0] > 0 and torch.all(cache["k"][1, 0, 0] == 128)
    bad = row.clone()
    bad[0, 0, 3] = float("nan")
    w4.kv8_append(cache, bad, row, table, lens(3))
    assert torch.isnan(cache["k_scale"][1, 0]) and not torch.isnan(cache["v_scale"][1, 0])
    w4.kv8_append(cache, row, row, table, lens(4))
    assert torch.isnan(cache["k_scale"][1, 0])           # stays while older rows do
    w4.kv8_append(cache, row, row, table, lens(1))
    assert torch.isfinite(cache["k_scale"][1, 0])        # the page begins anew
    bad[0, 0, 3] = float("inf")
    w4.kv8_append(cache, bad, bad, table, lens(17))
    assert torch.isnan(cache["k_scale"][3, 0]) and torch.isfinite(cache["k_scale"][1, 0])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,T", [(64, 16), (128, 32), (64, 64), (128, 128)])
def test_dequant(D, T, dtype):
    c = _case(3, [T * 3], [1], 2, 2, D, T, dtype)
    pages = torch.tensor([3, 0, 3, 1], dtype=torch.int32, device=DEV)
    k, v = w4.kv8_dequant(c["cache"], pages, TDT[dtype])
    n, p = _np(c), pages.cpu().numpy()
    for got, codes, s in ((k, n["k"], n["ks"]), (v, n["v"], n["vs"])):
        want = codes[p].astype(np.float32) * s[p][:, :, None, None]
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(TDT[dtype]))


def _check_attention(c, H, Hkv, D, dtype, causal=True, scale=None, one=False, **more):
    sc = 1 / math.sqrt(D) if scale is None else scale
    tokens = len(c["q"])
    lse = torch.full((tokens, H), 7.0, device=DEV)
    args = dict(cu_seqlens=None if one else c["dev"]["cu"], scale=scale, causal=causal, **more)
    out = w4.kv8_attention(c["q"], c["cache"], c["dev"]["table"], c["dev"]["lens"], lse=lse, **args)
    n = _np(c)
    k = n["k"] * n["ks"].astype(np.float64)[:, :, None, None]
    v = n["v"] * n["vs"].astype(np.float64)[:, :, None, None]
    want, mass, lw, work = kv8.attention(c["q"].float().cpu().numpy(), k, v, c["table"], c["lens"],
                                         c["cu"], c["T"], sc, causal)
    bound, lbound = kv8.attention_bounds(want, mass, work, max(c["lens"] + [1]), D, dtype)
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= bound), (np.max(err / bound), np.argwhere(err > bound)[:4])
    l = lse.double().cpu().numpy()
    empty = np.isinf(lw)
    assert np.array_equal(l[empty], lw[empty])
    assert np.all(np.abs(l[~empty] - lw[~empty]) <= lbound[~empty] + 2.0 ** -22 * np.abs(lw[~empty]))
    again = w4.kv8_attention(c["q"], c["cache"], c["dev"]["table"], c["dev"]["lens"], **args)
    assert torch.equal(out, again)
    return out


ATTENTIONS = [
    # lens, new tokens, H, Hkv, D, T
    ([1], [1], 1, 1, 64, 16),
    ([63, 64, 65], [1, 1, 1], 4, 4, 128, 16),
    ([777], [1], 8, 8, 128, 16),
    ([500, 3, 129, 1000], [1, 1, 1, 1], 10, 2, 128, 64),
    ([5000], [1], 16, 1, 128, 64),
    ([260, 0, 511], [1, 1, 1], 32, 1, 64, 32),
    ([33, 2100], [1, 1], 40, 8, 128, 128),
    ([200, 5, 700], [5, 5, 3], 32, 4, 64, 32),
    ([90, 64, 300], [17, 64, 0], 6, 2, 128, 16),
    ([300], [300], 5, 1, 128, 64),
    ([257, 700, 40], [129, 200, 33], 8, 2, 64, 128),
    ([1200, 333], [260, 333], 7, 1, 128, 32),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,news,H,Hkv,D,T", ATTENTIONS)
def test_attention(lens, news, H, Hkv, D, T, causal, dtype):
    say("attention", lens, news, H, Hkv, D, T, causal, dtype)
    c = _case(len(lens) + T + H, lens, news, H, Hkv, D, T, dtype)
    one = all(n == 1 for n in news)
    _check_attention(c, H, Hkv, D, dtype, causal, one=one, max_new=max(news))


@pytest.mark.parametrize("lens,news", [([3], [7]), ([70, 0, 10], [80, 4, 40]), ([0], [1])])
def test_rows_that_see_nothing(lens, news):
    c = _case(5, lens, news, 4, 2, 64, 16, "bf16")
    out = _check_attention(c, 4, 2, 64, "bf16")
    assert torch.all(out[:news[0] - lens[0]] == 0)


@pytest.mark.parametrize("news", [[1, 1], [3, 2], [70, 40]])
def test_scales_of_very_different_pages(news):
    """Pages whose scales span seven orders of magnitude, inside a unit of 64
    tokens and across units, and scales of zero."""
    lens = [150, 210]
    c = _case(6, lens, news, 8, 2, 64, 16, "bf16")
    r = c["r"]
    P = c["cache"]["num_pages"]
    for n in ("k_scale", "v_scale"):
        s = 10.0 ** r.uniform(-6, 0 if n == "v_scale" else -2, (P, 2))
        s[r.rand(P, 2) < 0.2] = 0
        c["cache"][n].copy_(torch.from_numpy(s.astype(np.float32)))
    # below fp16's normal range a probability of a small-scale page is off by
    # 2^-25 of the unit's largest scale, 128 codes of it, in each of 64 tokens
    out = w4.kv8_attention(c["q"], c["cache"], c["dev"]["table"], c["dev"]["lens"],
                           cu_seqlens=c["dev"]["cu"])
    n = _np(c)
    k = n["k"] * n["ks"].astype(np.float64)[:, :, None, None]
    v = n["v"] * n["vs"].astype(np.float64)[:, :, None, None]
    want, mass, _, work = kv8.attention(c["q"].float().cpu().numpy(), k, v, c["table"], lens,
                                        c["cu"], 16, 1 / 8, True)
    bound, _ = kv8.attention_bounds(want, mass, work, max(lens), 64, "bf16")
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= bound + 64 * 128 * 2.0 ** -25 * n["vs"].max())


@pytest.mark.parametrize("scale_q", [1e-30, 1e-6, 300.0, 1e20])
def test_queries_of_any_magnitude(scale_q):
    c = _case(7, [100, 300], [1, 1], 4, 2, 128, 32, "bf16")
    c["q"] = (c["q"].float() * scale_q).bfloat16()
    _check_attention(c, 4, 2, 128, "bf16", one=True, scale=0.1 / scale_q)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [1.7, -1.7])
@pytest.mark.parametrize("news", [[1, 1], [5, 9], [200, 150]])
@pytest.mark.parametrize("D,T", [(64, 16), (128, 64)])
def test_scores_far_apart(D, T, news, scale, dtype):
    """Scores of hundreds, the largest anywhere in a unit: what fp16 could not
    hold if the running maximum missed a token.  Beside the relative bound a
    probability below fp16's normal range is off by 2^-25 where the largest is
    2^11 and up, 2^-36, in each of the seen tokens of up to 128 codes."""
    lens = [260, 333]
    c = _case(15, lens, news, 8, 2, D, T, dtype)
    out = w4.kv8_attention(c["q"], c["cache"], c["dev"]["table"], c["dev"]["lens"],
                           cu_seqlens=c["dev"]["cu"], scale=scale, max_new=max(news))
    n = _np(c)
    k = n["k"] * n["ks"].astype(np.float64)[:, :, None, None]
    v = n["v"] * n["vs"].astype(np.float64)[:, :, None, None]
    want, mass, _, work = kv8.attention(c["q"].float().cpu().numpy(), k, v, c["table"], lens,
                                        c["cu"], T, scale, True)
    bound, _ = kv8.attention_bounds(want, mass, work, max(lens), D, dtype)
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= bound + max(lens) * 128 * 2.0 ** -36 * n["vs"].max())


@pytest.mark.parametrize("news", [[1, 1], [5, 9], [90, 70]])
def test_masked_places_do_not_matter(news):
    """NaN scales and any codes in pages of no sequence, and rows past a
    sequence's end, leave the results as they are."""
    c = _case(8, [100, 130], news, 8, 2, 128, 16, "f16", spare=4)
    args = dict(cu_seqlens=c["dev"]["cu"])
    base = w4.kv8_attention(c["q"], c["cache"], c["dev"]["table"], c["dev"]["lens"], **args)
    used = set(int(p) for b, L in enumerate(c["lens"]) for p in c["table"][b][:-(-L // 16)])
    for p in range(c["cache"]["num_pages"]):
        if p not in used:
            c["cache"]["k_scale"][p] = float("nan")
            c["cache"]["v_scale"][p] = float("inf")
    last = int(c["table"][0][6])                     # 100 tokens: rows 4 .. 15 are past the end
    c["cache"]["k"][last, :, 4:] = 255
    c["cache"]["v"][last, :, :, :, 4:] = 0
    again = w4.kv8_attention(c["q"], c["cache"], c["dev"]["table"], c["dev"]["lens"], **args)
    assert torch.equal(base, again)


def test_nonfinite_queries_and_pages_reach_their_own_rows_alone():
    c = _case(9, [100, 130], [1, 1], 8, 2, 64, 32, "bf16")
    base = w4.kv8_attention(c["q"], c["cache"], c["dev"]["table"], c["dev"]["lens"])
    c["q"][0, 3, 5] = float("nan")
    c["q"][1, 6, 0] = float("inf")
    out = w4.kv8_attention(c["q"], c["cache"], c["dev"]["table"], c["dev"]["lens"])
    hit = torch.zeros(2, 8, dtype=torch.bool, device=DEV)
    hit[0, 3] = hit[1, 6] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], base[~hit])
    c = _case(9, [100, 130], [1, 1], 8, 2, 64, 32, "bf16")
    c["cache"]["k_scale"][int(c["table"][1][2]), 1] = float("nan")
    out = w4.kv8_attention(c["q"], c["cache"], c["dev"]["table"], c["dev"]["lens"])
    assert torch.isnan(out[1, 4:]).all()
    assert torch.equal(out[0], base[0]) and torch.equal(out[1, :4], base[1, :4])


@pytest.mark.parametrize("news", [6, 70])
def test_pages_ahead_of_a_query_do_not_reach_it(news):
    """The scales of the pages that only later tokens of a call see are NaN:
    the earlier tokens' results stay as they are."""
    T, L = 16, 128 + news
    c = _case(14, [L], [news], 8, 2, 64, T, "f16")
    args = (c["cache"], c["dev"]["table"], c["dev"]["lens"])
    base = w4.kv8_attention(c["q"], *args, cu_seqlens=c["dev"]["cu"])
    last = int(c["table"][0][(L - 1) // T])
    first = ((L - 1) // T) * T - (L - news)              # first new token that sees the last page
    for name in ("k_scale", "v_scale"):
        keep = c["cache"][name][last].clone()
        c["cache"][name][last] = float("nan")
        out = w4.kv8_attention(c["q"], *args, cu_seqlens=c["dev"]["cu"])
        c["cache"][name][last] = keep
        if first > 0:
            assert torch.equal(out[:first], base[:first]), name
        assert torch.isnan(out[max(first, 0):]).all(), name


def test_strides_streams_and_bounds():
    lens, news = [200, 90], [20, 30]
    c = _case(10, lens, news, 8, 2, 64, 64, "f16")
    want = _check_attention(c, 8, 2, 64, "f16", max_new=30, max_len=200)
    wide = torch.zeros(50, 12, 64, dtype=torch.float16, device=DEV)
    wide[:, 2:10] = c["q"]
    out = torch.full((50, 10, 64), 3.0, dtype=torch.float16, device=DEV)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    w4.kv8_attention(wide[:, 2:10], c["cache"], c["dev"]["table"], c["dev"]["lens"],
                     cu_seqlens=c["dev"]["cu"], max_new=30, max_len=200, out=out[:, 1:9], stream=st)
    st.synchronize()
    assert torch.equal(out[:, 1:9], want)
    assert torch.all(out[:, 0] == 3) and torch.all(out[:, 9] == 3)


def test_pages_past_four_gigabytes():
    """A pool of more than 2^32 bytes: the last pages of it."""
    T, D, Hkv = 128, 128, 8
    pages = (1 << 32) // (T * D * Hkv) + 40
    c = _case(11, [200], [1], 16, Hkv, D, T, "bf16", spare=0)
    small = c["cache"]
    big = w4.kv8_cache(1, T, Hkv, D, DEV)
    big["num_pages"] = pages
    for n in ("k", "v", "k_scale", "v_scale"):
        big[n] = torch.empty(pages, *small[n].shape[1:], dtype=small[n].dtype, device=DEV)
        big[n][-2:] = small[n]
    table = c["dev"]["table"].clone()
    table[:, :2] += pages - 2
    lens = c["dev"]["lens"]
    a = w4.kv8_attention(c["q"], small, c["dev"]["table"], lens)
    b = w4.kv8_attention(c["q"], big, table, lens)
    assert torch.equal(a, b)
    w4.kv8_append(small, c["k"] * 3, c["v"] * 3, c["dev"]["table"], lens)
    w4.kv8_append(big, c["k"] * 3, c["v"] * 3, table, lens)
    for n in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(small[n], big[n][-2:])
    at = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    for x, y in zip(w4.kv8_dequant(small, at), w4.kv8_dequant(big, at + (pages - 2))):
        assert torch.equal(x, y)


def test_capture_in_a_graph():
    lens, T, D, H, Hkv = [100, 300], 32, 128, 8, 2
    c = _case(12, lens, [1, 1], H, Hkv, D, T, "bf16")
    cos, sin = _rope(400, D)
    qo, out = torch.empty_like(c["q"]), torch.empty_like(c["q"])
    table, dl = c["dev"]["table"], c["dev"]["lens"]
    space = w4.workspace(w4.kv8_attention_workspace_bytes(2, 2, 1, table.shape[1] * T, H, Hkv, D), DEV)

    def step(cache, qo, out):
        w4.kv8_append(cache, c["k"], c["v"], table, dl, q=c["q"], cos=cos, sin=sin, q_out=qo)
        return w4.kv8_attention(qo, cache, table, dl, out=out, workspace=space)

    eager = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in c["cache"].items()}
    step(eager, torch.empty_like(qo), torch.empty_like(out))
    torch.cuda.synchronize()
    eager = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in c["cache"].items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(c["cache"], qo, out)
    for i in range(4):
        for x in (c["q"], c["k"], c["v"]):
            x.copy_(torch.from_numpy(c["r"].randn(*x.shape)))
        want = step(eager, torch.empty_like(qo), torch.empty_like(out))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(torch.equal(eager[n], c["cache"][n]) for n in ("k", "v", "k_scale", "v_scale"))
        dl += 1


def test_empty_calls():
    cache = w4.kv8_cache(2, 16, 2, 64, DEV)
    table = torch.zeros(3, 1, dtype=torch.int32, device=DEV)
    lens, cu = torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    none = torch.zeros(0, 2, 64, dtype=torch.float16, device=DEV)
    assert w4.kv8_append(cache, none, none, table, lens, cu, q=none).shape == (0, 2, 64)
    assert w4.kv8_attention(none, cache, table, lens, cu).shape == (0, 2, 64)
    k, v = w4.kv8_dequant(cache, torch.zeros(0, dtype=torch.int32, device=DEV))
    assert k.shape == (0, 2, 16, 64) == v.shape


def test_refusals():
    c = _case(13, [20, 30], [1, 1], 4, 2, 64, 16, "f16")
    cache, table, lens = c["cache"], c["dev"]["table"], c["dev"]["lens"]
    cos, sin = _rope(40, 64)
    for bad in (dict(page_size=48), dict(head_dim=96)):
        with pytest.raises(w4.W4A16Error):
            w4.kv8_cache(2, bad.get("page_size", 16), 2, bad.get("head_dim", 64), DEV)
    with pytest.raises(ValueError):
        w4.kv8_append(cache, c["k"][:1], c["v"][:1], table, lens)          # tokens != sequences
    with pytest.raises(ValueError):
        w4.kv8_append(cache, c["k"], c["v"][:1], table, lens)
    with pytest.raises(TypeError):
        w4.kv8_append(cache, c["k"], c["v"].bfloat16(), table, lens)
    with pytest.raises(ValueError):
        w4.kv8_append(cache, c["k"], c["v"], table, lens, cos=cos)
    with pytest.raises(TypeError):
        w4.kv8_append(cache, c["k"], c["v"], table.long(), lens)
    with pytest.raises(w4.W4A16Error, match="status 1"):
        w4.kv8_append(cache, c["k"], c["v"], table, lens, cos=cos[:, :20].contiguous(),
                      sin=sin[:, :20].contiguous())                          # 40 channels turned
    with pytest.raises(ValueError):
        w4.kv8_attention(c["q"][:, :, :32], cache, table, lens)
    with pytest.raises(w4.W4A16Error, match="status 1"):
        w4.kv8_attention(c["q"][:, :3].contiguous(), cache, table, lens)     # 3 heads, 2 kv heads
    with pytest.raises(TypeError):
        w4.kv8_attention(c["q"].float(), cache, table, lens)
    with pytest.raises(ValueError):
        w4.kv8_attention(c["q"].transpose(0, 1), cache, table, lens)
    with pytest.raises(TypeError):
        w4.kv8_attention(c["q"], cache, table, lens, lse=torch.zeros(2, 4, device=DEV).half())
