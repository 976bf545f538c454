"""Attention over the 8-bit cache at the ends of the range that queries, scales
and scores can have, in each kernel, against 64 bits."""

import numpy as np
import pytest
import torch

import bit_weight_only_gemm_amd as w4
from oracle import kv8
from gpu_util import DEV, TDT, say

pytestmark = pytest.mark.gpu

# single tokens, a few (both one kernel) and many rows (another), pages within and
# across a unit of 64 tokens
FORMS = [([1, 1], 64, 16), ([1, 1], 128, 64), ([5, 9], 64, 32), ([80, 70], 64, 16), ([80, 70], 128, 64),
         ([150, 210], 64, 128)]


def _case(seed, news, D, T, dtype, lens=(150, 210), H=8, Hkv=2):
    r = np.random.RandomState(seed)
    width = -(-max(lens) // T)
    cache = w4.kv8_cache(len(lens) * width, T, Hkv, D, DEV)
    for n in ("k", "v"):
        cache[n].copy_(torch.from_numpy(r.randint(1, 256, cache[n].shape).astype(np.uint8)))
        cache[n + "_scale"].copy_(torch.from_numpy((r.rand(*cache[n + "_scale"].shape) * 0.01 + 0.005)
                                                   .astype(np.float32)))
    table = r.permutation(len(lens) * width).reshape(len(lens), width).astype(np.int32)
    q = torch.from_numpy(r.randn(sum(news), H, D)).to(TDT[dtype]).to(DEV)
    return cache, q, table, list(lens), np.concatenate([[0], np.cumsum(news)]).astype(np.int32), r


def _check(cache, q, table, lens, cu, dtype, scale):
    """Output and lse against the oracle, with its bounds and, for the
    probabilities below fp16's normal range, 2^-36 of the largest in each of the
    seen tokens of up to 128 codes."""
    D, T = cache["head_dim"], cache["page_size"]
    dev = lambda x: torch.from_numpy(np.asarray(x, np.int32)).to(DEV)  # noqa: E731
    lse = torch.empty(q.shape[:2], device=DEV)
    out = w4.kv8_attention(q, cache, dev(table), dev(lens), dev(cu), max_new=int(np.diff(cu).max()),
                           scale=scale, lse=lse)
    ks, vs = (cache[n].cpu().numpy().astype(np.float64)[:, :, None, None] for n in ("k_scale", "v_scale"))
    k, v = kv8.rows_k(cache["k"].cpu().numpy()) * ks, kv8.rows_v(cache["v"].cpu().numpy()) * vs
    want, mass, lw, work = kv8.attention(q.double().cpu().numpy(), k, v, table, lens, cu, T, scale, True)
    bound, lbound = kv8.attention_bounds(want, mass, work, max(lens), D, dtype)
    err = np.abs(out.double().cpu().numpy() - want)
    bound = bound + max(lens) * 128 * 2.0 ** -36 * vs.max()
    assert np.all(err <= bound), (np.max(err / bound), np.argwhere(~(err <= bound))[:4])
    l = lse.double().cpu().numpy()
    assert np.all(np.abs(l - lw) <= lbound + 2.0 ** -22 * np.abs(lw))
    return out


@pytest.mark.parametrize("news,D,T", FORMS)
@pytest.mark.parametrize("low,high", [(-44, -43), (-44, -39), (-41, -36), (-39, -30)])
def test_values_of_subnormal_scales(low, high, news, D, T):
    """Values of bf16's least magnitudes: the pages' scales are subnormal in
    fp32, or some are."""
    say("subnormal value scales", low, high, news, D, T)
    cache, q, table, lens, cu, r = _case(1, news, D, T, "bf16")
    s = 10.0 ** r.uniform(low, high, cache["v_scale"].shape)
    s[0, 0] = 0
    cache["v_scale"].copy_(torch.from_numpy(s).float())
    out = _check(cache, q, table, lens, cu, "bf16", D ** -0.5)
    assert torch.isfinite(out).all()


def test_tiny_values_through_the_append():
    r = np.random.RandomState(2)
    cache = w4.kv8_cache(4, 64, 2, 64, DEV)
    mk = lambda h: torch.from_numpy(r.randn(200, h, 64)).to(DEV)  # noqa: E731
    q, k, v = mk(8).bfloat16(), mk(2).bfloat16(), (mk(2) * 1e-37).bfloat16()
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    lens, cu = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([200], [0, 200]))
    w4.kv8_append(cache, k, v, table, lens, cu)
    _check(cache, q, table.cpu().numpy(), [200], [0, 200], "bf16", 0.125)
    _check(cache, q[-1:], table.cpu().numpy(), [200], [0, 1], "bf16", 0.125)


def _onehot_scores(q, cache, r, power):
    """Queries of one channel each and keys whose scores are small integers
    times 2^power: exact in fp32, far apart where they differ, often equal."""
    D = q.shape[2]
    channel = torch.from_numpy(r.randint(0, D, q.shape[:2])).to(DEV)
    q.zero_()
    half = min(power // 2, 14 if q.dtype == torch.float16 else 120)
    q.scatter_(2, channel[..., None], 2.0 ** half)
    codes = r.randint(-5, 6, cache["k"].shape)
    cache["k"].copy_(torch.from_numpy((codes + 128).astype(np.uint8)))
    scales = 2.0 ** r.randint(0, 3, cache["k_scale"].shape)
    cache["k_scale"].copy_(torch.from_numpy(scales.astype(np.float32)))
    return 2.0 ** (power - half)


@pytest.mark.parametrize("news,D,T", FORMS)
@pytest.mark.parametrize("power,dtype", [(18, "f16"), (24, "bf16"), (27, "f16"), (31, "bf16"), (38, "f16"),
                                         (60, "bf16"), (99, "bf16"), (120, "bf16")])
def test_scores_of_any_magnitude(power, dtype, news, D, T):
    """The rows' largest scores take it all, in equal parts, whatever the
    magnitude and sign: probabilities are exact, the output is off by its sums'
    roundings (64 tokens and the joins) and its own."""
    say("scores of 2 **", power, dtype, news, D, T)
    cache, q, table, lens, cu, r = _case(power, news, D, T, dtype)
    scale = _onehot_scores(q, cache, r, power)
    dev = lambda x: torch.from_numpy(np.asarray(x, np.int32)).to(DEV)  # noqa: E731
    lse = torch.empty(q.shape[:2], device=DEV)
    out = w4.kv8_attention(q, cache, dev(table), dev(lens), dev(cu), max_new=max(news), scale=scale, lse=lse)
    ks, vs = (cache[n].cpu().numpy().astype(np.float64)[:, :, None, None] for n in ("k_scale", "v_scale"))
    k, v = kv8.rows_k(cache["k"].cpu().numpy()) * ks, kv8.rows_v(cache["v"].cpu().numpy()) * vs
    want, mass, lw, _ = kv8.attention(q.double().cpu().numpy(), k, v, table, lens, cu, T, scale, True)
    bound, _ = kv8.attention_bounds(want, mass, np.zeros(lw.shape), max(lens), D, dtype)
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= bound), (np.max(err / bound), np.argwhere(~(err <= bound))[:4])
    l = lse.double().cpu().numpy()
    assert np.all(np.abs(l - lw) <= 2.0 ** -18 + 2.0 ** -22 * np.abs(lw))


@pytest.mark.parametrize("news,D,T", FORMS)
@pytest.mark.parametrize("scale", [1e6, 1e7, 1e8, 1e10, 1e30, -1e34])
def test_large_scores_stay_among_the_values(scale, news, D, T):
    say("scale", scale, news, D, T)
    cache, q, table, lens, cu, r = _case(3, news, D, T, "bf16")
    dev = lambda x: torch.from_numpy(np.asarray(x, np.int32)).to(DEV)  # noqa: E731
    out = w4.kv8_attention(q, cache, dev(table), dev(lens), dev(cu), max_new=max(news), scale=scale)
    most = 127 * cache["v_scale"].max() * (1 + 2.0 ** -8)
    assert torch.isfinite(out).all() and torch.all(out.abs() <= most)
    assert torch.all(out.abs().amax(2) > 0)


@pytest.mark.parametrize("news,D,T,lens", [(n, D, T, (150, 210)) for n, D, T in FORMS]
                         + [([1, 1], 64, 16, (3000, 2100)), ([1, 1], 128, 64, (3000, 2100)),
                            ([70, 40], 128, 32, (3000, 2100))])
@pytest.mark.parametrize("low,high", [(24, 27), (30, 32), (33, 34), (-3, 35)])
def test_values_near_the_largest(low, high, news, D, T, lens):
    """Values of up to 1e37, in parts that are joined: over waves, and over
    workgroups where the sequences are long."""
    say("large values", low, high, news, D, T, lens)
    cache, q, table, lens, cu, r = _case(4, news, D, T, "bf16", lens)
    cache["v_scale"].copy_(torch.from_numpy(10.0 ** r.uniform(low, high, cache["v_scale"].shape)).float())
    out = _check(cache, q, table, lens, cu, "bf16", D ** -0.5)
    assert torch.isfinite(out).all()
