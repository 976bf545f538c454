"""One decoder layer served in 8 bits to beams: attention with capped scores over
a window, a gated feed-forward block, and the cache's pages shared between the
beams of a prompt.

    python examples/decoder_layer.py [--hidden 2048] [--heads 16] [--kv-heads 8]

A prompt is run once (``kv8_reserve``, then the layer) and forked into beams
(``kv8_fork``).  A step gives every beam room for a token and runs the layer on
all of them; now and then beams are dropped (``kv8_free``), others branch in
their place, and the cache is compacted (``kv8_compact``).  The layer is
``w8a8_linear``, ``kv8_append``, ``kv8_attention_scored``, ``w8a8_linear`` and
then ``w8a8_gated`` and ``w8a8_linear``.  What it adds to its input is compared,
for every token of every beam, with the same layer in 32-bit floats over that
beam's whole history.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_only_gemm_amd as w4  # noqa: E402

SOFTCAP = 5.0


def norm(x):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


def angles(positions, dim, device):
    a = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    return a.cos().float().to(device), a.sin().float().to(device)


class DecoderLayer:
    """weights: dict(qkv [(H + 2 Hkv) D, hidden], out [hidden, H D], gate_up [2 F,
    hidden], down [hidden, F]) in fp32, held in int8."""

    def __init__(self, weights, heads, kv_heads, window, positions, dtype=torch.bfloat16):
        self.heads, self.kv_heads, self.window, self.dtype = heads, kv_heads, window, dtype
        self.dim = weights["out"].shape[1] // heads
        self.w = {name: w4.w8a8_quantize(w) for name, w in weights.items()}
        self.cos, self.sin = angles(positions, self.dim, weights["out"].device)

    def __call__(self, x, cache, table, lens, positions, cu=None, max_new=None):
        """What the layer adds to x [tokens, hidden], the new tokens of all rows."""
        H, Hkv, D = self.heads, self.kv_heads, self.dim
        rows = w4.w8a8_linear(norm(x).to(self.dtype), *self.w["qkv"])
        q, k, v = (t.view(len(x), -1, D) for t in rows.split([H * D, Hkv * D, Hkv * D], dim=1))
        q = w4.kv8_append(cache, k, v, table, lens, cu, max_new, q=q, cos=self.cos, sin=self.sin)
        first = (positions - (self.window - 1)).int()
        o = w4.kv8_attention_scored(q, cache, table, lens, cu, max_new, softcap=SOFTCAP, first=first)
        a = w4.w8a8_linear(o.view(len(x), H * D), *self.w["out"])
        y = w4.w8a8_gated(norm(x + a.float()).to(self.dtype), *self.w["gate_up"], act="silu")
        return a.float() + w4.w8a8_linear(y, *self.w["down"]).float()


def plain(x, w, heads, kv_heads, window, cos, sin):
    """The same on one whole history x [n, hidden] in fp32."""
    n, D, G = len(x), w["out"].shape[1] // heads, heads // kv_heads
    q, k, v = (t.view(n, -1, D) for t in (norm(x) @ w["qkv"].T).split(
        [heads * D, kv_heads * D, kv_heads * D], dim=1))

    def turn(t):
        a, b = t[..., :D // 2], t[..., D // 2:]
        c, s = cos[:n, None], sin[:n, None]
        return torch.cat([a * c - b * s, b * c + a * s], dim=-1).transpose(0, 1)

    q, k = turn(q), turn(k).repeat_interleave(G, 0)
    v = v.transpose(0, 1).repeat_interleave(G, 0).contiguous()
    s = SOFTCAP * torch.tanh(q @ k.transpose(1, 2).contiguous() * (D ** -0.5 / SOFTCAP))
    far = torch.arange(n, device=x.device)[:, None] - torch.arange(n, device=x.device)
    s.masked_fill_((far < 0) | (far >= window), -torch.inf)
    a = (s.softmax(-1) @ v).transpose(0, 1).reshape(n, heads * D) @ w["out"].T
    g, u = (norm(x + a) @ w["gate_up"].T).chunk(2, 1)
    return a + (torch.nn.functional.silu(g) * u) @ w["down"].T


def run(hidden=2048, heads=16, kv_heads=8, prompts=(300, 17, 140), beams=3, steps=10, window=128, page=32,
        dtype=torch.bfloat16, device="cuda"):
    """Relative RMS error of what the layer adds, over all tokens of all beams,
    and the pages in use at the end."""
    D, F = hidden // heads, 2 * hidden
    gen = torch.Generator(device=device).manual_seed(11)

    def mk(*shape):
        return torch.randn(*shape, generator=gen, device=device)

    w = {"qkv": mk((heads + 2 * kv_heads) * D, hidden), "out": mk(hidden, heads * D), "gate_up": mk(2 * F, hidden),
         "down": mk(hidden, F)}
    w = {name: t * t.shape[1] ** -0.5 for name, t in w.items()}
    S, longest = len(prompts), max(prompts) + steps
    rows, width = S * 2 * beams + S, -(-longest // page)
    layer = DecoderLayer(w, heads, kv_heads, window, longest, dtype)
    # pages for every prompt, and for each beam two pages of its own and the next
    num = sum(-(-n // page) for n in prompts) + S * 2 * beams * (2 + steps // page)
    cache = w4.kv8_cache(num, page, kv_heads, D, device)
    refs = w4.kv8_refs(num, device)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=device)
    lens = torch.zeros(rows, dtype=torch.int32, device=device)
    status = []

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=device)

    def grow(add):
        status.append(w4.kv8_reserve(refs, table, lens, ints(add), page))

    # ---- the prompts, in rows 0 .. S - 1
    past = {s: mk(n, hidden) for s, n in enumerate(prompts)}
    grow([*prompts, *[0] * (rows - S)])
    cu = torch.tensor([0, *prompts]).cumsum(0).int().to(device)
    at = torch.cat([torch.arange(n, device=device) for n in prompts])
    y = layer(torch.cat(list(past.values())), cache, table[:S], lens[:S], at, cu, max(prompts))
    done = dict(enumerate(y.split(list(prompts))))

    # ---- beams: children of prompt s in rows S + beams s .., and as many to branch into
    def branch(pairs):
        src, dst = zip(*pairs)
        status.append(w4.kv8_fork(cache, refs, table, lens, ints(src), ints(dst)))
        for a, b in pairs:
            past[b], done[b] = past[a], done[a]

    def drop(gone):
        w4.kv8_free(refs, table, lens, ints(gone), page)

    alive = list(range(S, S + S * beams))
    branch([(s, S + s * beams + i) for s in range(S) for i in range(beams)])
    drop(list(range(S)))
    errors, sizes = 0.0, 0.0

    def close(gone):
        nonlocal errors, sizes
        for b in gone:
            want = plain(past[b], w, heads, kv_heads, window, layer.cos, layer.sin)
            errors += (done[b] - want).square().sum().item()
            sizes += want.square().sum().item()

    for step in range(steps):
        grow([1 if b in alive else 0 for b in range(rows)])
        x = mk(len(alive), hidden)
        pick = torch.tensor(alive, device=device)
        y = layer(x, cache, table[pick], lens[pick], lens[pick].long() - 1)
        for i, b in enumerate(alive):
            past[b] = torch.cat([past[b], x[i:i + 1]])
            done[b] = torch.cat([done[b], y[i:i + 1]])
        if step % 4 == 2:
            # every prompt goes on with copies of its first beam but one, and that
            spare = [b for b in range(S, rows) if b not in alive]
            kept, pairs, gone = [], [], []
            for s in range(S):
                mine = alive[s * beams:(s + 1) * beams]
                new = spare[s * beams:s * beams + beams - 1]
                pairs += [(mine[0], b) for b in new]
                gone += mine[1:]
                kept += [mine[0], *new]
            branch(pairs)
            close(gone)
            drop(gone)
            alive = kept
            table, refs, used = w4.kv8_compact(cache, refs, table, lens)
    close(alive)
    assert all(s.item() == 0 for s in status), [s.item() for s in status]
    table, refs, used = w4.kv8_compact(cache, refs, table, lens)
    return (errors / sizes) ** 0.5, used.item()


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--heads", type=int, default=16)
    p.add_argument("--kv-heads", type=int, default=8)
    a = p.parse_args()
    print("relative RMS error of what the layer adds, against fp32: %.4f; %d pages in use" % run(
        a.hidden, a.heads, a.kv_heads))
