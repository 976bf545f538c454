"""Graphs that were captured with a workspace kept for their stream, after calls
on that stream have outgrown it: replays are right and write nothing of others."""

import pytest
import torch

import bit_weight_only_gemm_amd as w4
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def gated(M, K, F=64):
    g = torch.Generator(device=DEV).manual_seed(M + K)
    x = torch.randn(M, K, generator=g, device=DEV).half()
    w = torch.randint(-127, 128, (2 * F, K), generator=g, device=DEV, dtype=torch.int8)
    return x, w, torch.full((2 * F,), 1e-3, device=DEV)


def attention(lens):
    T, H, Hkv, D = 64, 8, 1, 128
    g = torch.Generator(device=DEV).manual_seed(7)
    width = -(-max(lens) // T)
    cache = w4.kv8_cache(len(lens) * width, T, Hkv, D, DEV)
    for n in ("k", "v"):
        cache[n].random_(1, 256, generator=g)
        cache[n + "_scale"].fill_(0.01)
    table = torch.arange(len(lens) * width, dtype=torch.int32, device=DEV).view(len(lens), width)
    q = torch.randn(len(lens), H, D, generator=g, device=DEV).half()
    return q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("op", ["gated", "attention"])
def test_replays_after_the_workspace_has_grown(op):
    say("kept workspace", op)
    st = torch.cuda.Stream()
    if op == "gated":
        small, large = gated(50, 256), gated(300, 1 << 14)
        call = w4.w8a8_gated
    else:
        small, large = attention([3000]), attention([9000] * 40)
        call = w4.kv8_attention_scored
    out = torch.empty_like(call(*small))
    want = call(*small)
    torch.cuda.synchronize()
    call(*small, out=out, stream=st)               # the stream's workspace is there
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call(*small, out=out)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        first = call(*large)                       # outgrows it
        others = [torch.full((1 << 18,), 7, dtype=torch.int32, device=DEV) for _ in range(16)]
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all((t == 7).all() for t in others)
        with torch.cuda.stream(st):
            again = call(*large)
        torch.cuda.synchronize()
        assert torch.equal(again, first)
