"""One attention layer served in 8 bits: prompts of several sequences, then
tokens one at a time, over one paged cache.

    python examples/attention_layer.py [--hidden 4096] [--heads 32] [--kv-heads 8]

Each step is four calls: the fused query/key/value projection
(``w8a8_linear``, int8 weights, rows quantized on the way), ``kv8_append``
(rotation, and the new keys and values into the cache), ``kv8_attention``, and
the output projection on int4 weights (``w4a16_gemm``).  The result of every
step is compared with the same layer in 32-bit floats, on the projection's
weights as given and the values that the int4 weights stand for.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_only_gemm_amd as w4  # noqa: E402


class AttentionLayer:
    """Weights of a layer: qkv [(H + 2 Hkv) D, hidden] in int8, out [hidden, H D] in int4."""

    def __init__(self, qkv, out, heads, kv_heads, positions, dtype=torch.bfloat16):
        self.heads, self.kv_heads, self.dim = heads, kv_heads, out.shape[1] // heads
        self.dtype = dtype
        self.qkv, self.qkv_scale = w4.w8a8_quantize(qkv)
        self.out = w4.w4a16_repack(*w4.w4a16_quantize_rtn(out, 128))
        self.cos, self.sin = angles(positions, self.dim, qkv.device)

    def __call__(self, x, cache, table, lens, cu=None, max_new=None):
        """x [tokens, hidden], the new tokens of all sequences; lens with them."""
        H, Hkv, D = self.heads, self.kv_heads, self.dim
        rows = w4.w8a8_linear(x, self.qkv, self.qkv_scale)
        q, k, v = (t.view(len(x), -1, D) for t in rows.split([H * D, Hkv * D, Hkv * D], dim=1))
        q = w4.kv8_append(cache, k, v, table, lens, cu, max_new, q=q, cos=self.cos, sin=self.sin)
        o = w4.kv8_attention(q, cache, table, lens, cu, max_new)
        return w4.w4a16_gemm(o.view(len(x), H * D), self.out)


def angles(positions, dim, device):
    a = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    return a.cos().float().to(device), a.sin().float().to(device)


def plain(x, qkv, out, heads, kv_heads, cos, sin):
    """The layer on one whole sequence x [n, hidden] in fp32, causal."""
    n, D = len(x), out.shape[1] // heads
    q, k, v = (t.view(n, -1, D) for t in (x.float() @ qkv.T).split(
        [heads * D, kv_heads * D, kv_heads * D], dim=1))

    def turn(t):
        a, b = t[..., :D // 2], t[..., D // 2:]
        c, s = cos[:n, None], sin[:n, None]
        return torch.cat([a * c - b * s, b * c + a * s], dim=-1)

    G = heads // kv_heads
    q, k = turn(q).transpose(0, 1), turn(k).transpose(0, 1).repeat_interleave(G, 0).contiguous()
    v = v.transpose(0, 1).repeat_interleave(G, 0).contiguous()
    s = q @ k.transpose(1, 2).contiguous() * D ** -0.5
    s.masked_fill_(torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1), -torch.inf)
    return (s.softmax(-1) @ v).transpose(0, 1).reshape(n, heads * D) @ out.T


def run(hidden=4096, heads=32, kv_heads=8, prompts=(300, 1, 77, 513), steps=8, page=64,
        dtype=torch.bfloat16, device="cuda"):
    """Relative RMS errors against the fp32 layer: (of the prompts, of the steps)."""
    D = hidden // heads
    g = torch.Generator(device=device).manual_seed(7)

    def mk(*shape):
        return torch.randn(*shape, generator=g, device=device)

    qkv = mk((heads + 2 * kv_heads) * D, hidden) * hidden ** -0.5
    out = mk(hidden, heads * D) * hidden ** -0.5
    longest = max(prompts) + steps
    layer = AttentionLayer(qkv, out, heads, kv_heads, longest, dtype)
    out = w4.w4a16_dequant(layer.out).float()
    xs = [mk(n + steps, hidden).to(dtype) for n in prompts]
    want = [plain(x, qkv, out, heads, kv_heads, layer.cos, layer.sin) for x in xs]

    B, width = len(prompts), -(-longest // page)
    cache = w4.kv8_cache(B * width, page, kv_heads, D, device)
    table = torch.randperm(B * width, generator=g, device=device).int().view(B, width)
    lens = torch.tensor(prompts, dtype=torch.int32, device=device)
    cu = torch.tensor([0, *prompts]).cumsum(0).int().to(device)
    y = layer(torch.cat([x[:n] for x, n in zip(xs, prompts)]), cache, table, lens, cu, max(prompts))
    got = [list(part) for part in y.split(list(prompts))]
    for i in range(steps):
        lens = lens + 1
        y = layer(torch.stack([x[n + i] for x, n in zip(xs, prompts)]), cache, table, lens)
        for b in range(B):
            got[b].append(y[b])

    def error(pick):
        a = torch.cat([torch.stack(rows)[pick(n)].float() for rows, n in zip(got, prompts)])
        b = torch.cat([rows[pick(n)] for rows, n in zip(want, prompts)])
        return ((a - b).norm() / b.norm()).item()

    return error(lambda n: slice(0, n)), error(lambda n: slice(n, None))


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--heads", type=int, default=32)
    p.add_argument("--kv-heads", type=int, default=8)
    a = p.parse_args()
    print("relative RMS error against fp32: prompts %.4f, single tokens %.4f"
          % run(a.hidden, a.heads, a.kv_heads))
