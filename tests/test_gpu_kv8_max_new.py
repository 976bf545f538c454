"""A bound max_new below a sequence's new tokens: the rows up to it are
processed as in a call without the others, the rows past it not at all."""

import numpy as np
import pytest
import torch

import bit_weight_only_gemm_amd as w4
from gpu_util import DEV, TDT, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,T,dtype", [(64, 16, "f16"), (128, 64, "bf16")])
@pytest.mark.parametrize("lens,news,max_new", [
    ([5, 40, 90], [3, 1, 6], 1), ([200, 7, 130], [150, 0, 70], 20), ([300, 90], [280, 90], 140), ([4, 9], [7, 3], 2)])
def test_rows_past_the_bound(lens, news, max_new, D, T, dtype):
    say("max_new", lens, news, max_new, D, T, dtype)
    H, Hkv = 4, 2
    r = np.random.RandomState(max_new + D)
    width = -(-max(lens) // T)
    cache = w4.kv8_cache(len(lens) * width, T, Hkv, D, DEV)
    for n in ("k", "v"):
        cache[n].copy_(torch.from_numpy(r.randint(1, 256, cache[n].shape).astype(np.uint8)))
        cache[n + "_scale"].copy_(torch.from_numpy((r.rand(*cache[n + "_scale"].shape) * 0.02).astype(np.float32)))
    table = torch.from_numpy(r.permutation(len(lens) * width).astype(np.int32)).view(len(lens), width).to(DEV)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    mk = lambda h: torch.from_numpy(r.randn(sum(news), h, D)).to(TDT[dtype]).to(DEV)  # noqa: E731
    q, k, v = mk(H), mk(Hkv), mk(Hkv)
    a = torch.from_numpy(r.rand(max(lens), D // 2) * 6).float().to(DEV)
    rope = dict(cos=a.cos(), sin=a.sin())
    cu = np.concatenate([[0], np.cumsum(news)])
    # the same sequences, cut to their first max_new new tokens
    cut = [min(n, max_new) for n in news]
    keep = np.concatenate([np.arange(s, s + n) for s, n in zip(cu, cut)])
    short = [L - n + c for L, n, c in zip(lens, news, cut)]
    rows = torch.from_numpy(keep).to(DEV)
    other = torch.ones(len(q), dtype=torch.bool, device=DEV)
    other[rows] = False

    want = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in cache.items()}
    cut_cu = dev(np.concatenate([[0], np.cumsum(cut)]).tolist())
    if min(short) >= 0:          # (a length below 0 has no cut form; its rows are at negative positions)
        want_q = w4.kv8_append(want, k[rows], v[rows], table, dev(short), cut_cu, q=q[rows], **rope)
    else:
        want_q = None
    q_out = torch.full_like(q, 7.0)
    w4.kv8_append(cache, k, v, table, dev(lens), dev(cu.tolist()), max_new=max_new, q=q, q_out=q_out, **rope)
    assert torch.all(q_out[other] == 7)
    if want_q is not None:
        assert torch.equal(q_out[rows], want_q)
        for n in ("k", "v", "k_scale", "v_scale"):
            assert torch.equal(cache[n], want[n]), n

    # attention sees all of lens; its rows past the bound are left as they are
    full = w4.kv8_attention(q, cache, table, dev(lens), dev(cu.tolist()))
    out = torch.full_like(q, 7.0)
    lse = torch.full((len(q), H), 7.0, device=DEV)
    w4.kv8_attention(q, cache, table, dev(lens), dev(cu.tolist()), max_new=max_new, out=out, lse=lse)
    assert torch.all(out[other] == 7) and torch.all(lse[other] == 7)
    # (another split or kernel than the full call's: two roundings to bf16, 2^-9
    # each, and 2^-11 each of the weighted magnitudes, at most 127 * 0.02)
    d = (out[rows].float() - full[rows].float()).abs()
    assert torch.all(d <= 2.0 ** -6 * full[rows].float().abs() + 2.0 ** -8)
