"""A bound max_len below the sequences' lengths plans the split of the keys and
cuts nothing."""

import math

import numpy as np
import pytest
import torch

import bit_weight_only_gemm_amd as w4
from oracle import kv8
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,T", [(64, 16), (128, 64)])
@pytest.mark.parametrize("news", [[1, 1], [7, 2], [90, 140]])
@pytest.mark.parametrize("max_len", [0, 64, 300, 900])
def test_longer_sequences_are_seen_whole(max_len, news, D, T):
    say("max_len", max_len, news, D, T)
    lens, H, Hkv = [1700, 800], 4, 2
    r = np.random.RandomState(max_len + D)
    width = -(-max(lens) // T)
    cache = w4.kv8_cache(2 * width, T, Hkv, D, DEV)
    for n in ("k", "v"):
        cache[n].copy_(torch.from_numpy(r.randint(1, 256, cache[n].shape).astype(np.uint8)))
        cache[n + "_scale"].copy_(torch.from_numpy((r.rand(*cache[n + "_scale"].shape) * 0.01 + 0.005)
                                                   .astype(np.float32)))
    table = r.permutation(2 * width).reshape(2, width).astype(np.int32)
    q = torch.from_numpy(r.randn(sum(news), H, D)).bfloat16().to(DEV)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    dev = lambda x: torch.from_numpy(np.asarray(x, np.int32)).to(DEV)  # noqa: E731
    out = w4.kv8_attention(q, cache, dev(table), dev(lens), dev(cu), max_new=max(news), max_len=max_len)
    ks, vs = (cache[n].cpu().numpy().astype(np.float64)[:, :, None, None] for n in ("k_scale", "v_scale"))
    k, v = kv8.rows_k(cache["k"].cpu().numpy()) * ks, kv8.rows_v(cache["v"].cpu().numpy()) * vs
    want, mass, _, work = kv8.attention(q.double().cpu().numpy(), k, v, table, lens, cu, T,
                                        1 / math.sqrt(D), True)
    bound, _ = kv8.attention_bounds(want, mass, work, max(lens), D, "bf16")
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= bound), (np.max(err / bound), np.argwhere(err > bound)[:4])
