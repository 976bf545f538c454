"""Attention over the 8-bit cache by the kernel of many rows, where its
workgroups share keys and values: many workgroups at once, each with several
units of 64 tokens whose keys differ by far, so that keys read from the wrong
unit would show."""

import math

import numpy as np
import pytest
import torch

import bit_weight_only_gemm_amd as w4
from oracle import kv8
from gpu_util import DEV, TDT, say

pytestmark = pytest.mark.gpu


def _cache(r, pages, Hkv, D, T):
    """Random codes; scales by page."""
    cache = w4.kv8_cache(pages, T, Hkv, D, DEV)
    cache["k"].copy_(torch.from_numpy(r.randint(1, 256, cache["k"].shape).astype(np.uint8)))
    cache["v"].copy_(torch.from_numpy(r.randint(1, 256, cache["v"].shape).astype(np.uint8)))
    for n in ("k_scale", "v_scale"):
        cache[n].copy_(torch.from_numpy((r.rand(pages, Hkv) * 0.02 + 0.005).astype(np.float32)))
    return cache


def _values(cache):
    return [rows(cache[n].cpu().numpy()) * cache[n + "_scale"].cpu().numpy().astype(np.float64)[:, :, None, None]
            for n, rows in (("k", kv8.rows_k), ("v", kv8.rows_v))]


# the least number of units in which the keys staged first are needed (two), an
# odd number of them, and one whose first workgroups see fewer than the last
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,T", [(64, 32), (64, 128), (128, 16), (128, 64)])
@pytest.mark.parametrize("L,new", [(128, 64), (180, 100), (330, 200)])
def test_the_first_units_keys_are_its_own(L, new, D, T, dtype):
    say("first unit's keys", L, new, D, T, dtype)
    B, Hkv, G = 24, 4, 4
    r = np.random.RandomState(L + D + T)
    width = -(-L // T)
    cache = _cache(r, B * width, Hkv, D, T)
    order = r.permutation(B * width).reshape(B, width).astype(np.int32)
    table = torch.from_numpy(order).to(DEV)
    # unit 2's keys far above unit 0's
    if width > 128 // T:
        cache["k_scale"][table[:, 128 // T:].long()] *= 8
    q = torch.from_numpy(r.randn(B * new, Hkv * G, D)).to(TDT[dtype]).to(DEV)
    lens = torch.full((B,), L, dtype=torch.int32, device=DEV)
    cu = torch.arange(0, (B + 1) * new, new, dtype=torch.int32, device=DEV)
    out = w4.kv8_attention(q, cache, table, lens, cu, max_new=new)
    for _ in range(4):
        assert torch.equal(out, w4.kv8_attention(q, cache, table, lens, cu, max_new=new))
    k, v = _values(cache)
    for b in (0, 11, B - 1):
        rows = slice(b * new, (b + 1) * new)
        want, mass, _, work = kv8.attention(q[rows].float().cpu().numpy(), k, v, order[b:b + 1], [L],
                                            [0, new], T, 1 / math.sqrt(D), True)
        bound, _ = kv8.attention_bounds(want, mass, work, L, D, dtype)
        # (a probability below fp16's normal range: 2^-36 of the largest, in each
        # of the seen tokens of up to 128 codes)
        bound = bound + L * 128 * 2.0 ** -36 * float(cache["v_scale"].max())
        err = np.abs(out[rows].double().cpu().numpy() - want)
        assert np.all(err <= bound), (b, np.max(err / bound))
