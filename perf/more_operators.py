"""The cases by which four operators of an 8-bit serving path are measured:
attention over the paged 8-bit cache with capped scores, distance bias,
document and prefix masks (``scored``), the gated feed-forward product
(``gated``), the step of a beam over the cache's pages (``beam``: children
freed, forked anew and given room for a token) and the compaction of a cache
(``compact``).

A case's ``op`` says which.  ``run`` makes one pass: with ``own`` false in
elementary torch operations in 32 bits, with ``own`` true through the library's
entry points.  ``exact`` is the same result from the definition in 64 bits.

Cache layout: a page holds T tokens of every kv head; codes are uint8 c,
standing for (c - 128) * scale with one fp32 scale per (page, head): k [pages,
Hkv, T, D], v [pages, Hkv, T / 16, D, 16], k_scale and v_scale [pages, Hkv].
refs [pages] counts the table rows that hold a page, 0 where it is free.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
INV127 = 1.0 / 127.0


def listed():
    return [
        # ---- attention over the cache; cap: of the scores (0: none), slopes: distance bias,
        # doc: mean length of the documents in a sequence (0: one), prefix: share of the new
        # tokens that see each other both ways
        # one token of two sequences under capped scores: latency
        {"name": "scored_token", "op": "scored", "B": 2, "new": 1, "ctx": 1213, "H": 32, "Hkv": 8, "D": 128, "T": 16,
         "cap": 50.0, "slopes": False, "doc": 0, "prefix": 0.0, "dtype": "f16"},
        # a decode batch of ragged contexts with distance bias: the cache's bytes
        {"name": "scored_batch", "op": "scored", "B": 64, "new": 1, "ctx": 8192, "H": 40, "Hkv": 8, "D": 128, "T": 64,
         "cap": 0.0, "slopes": True, "doc": 0, "prefix": 0.0, "dtype": "bf16"},
        # prompts' chunks over their own earlier context, capped: vector work beside the matrix rate
        {"name": "scored_prompt", "op": "scored", "B": 4, "new": 2048, "ctx": 8192, "H": 40, "Hkv": 8, "D": 128, "T": 64,
         "cap": 50.0, "slopes": False, "doc": 0, "prefix": 0.0, "dtype": "bf16"},
        # long prompts packed from documents, the first half seen both ways, small heads
        {"name": "scored_documents", "op": "scored", "B": 3, "new": 4001, "ctx": 6001, "H": 32, "Hkv": 4, "D": 64, "T": 32,
         "cap": 30.0, "slopes": True, "doc": 1500, "prefix": 0.5, "dtype": "f16"},
        # ---- gated feed-forward product, 16-bit activations quantized per token in the call
        # one token: the weight stream of both projections
        {"name": "gated_token", "op": "gated", "M": 1, "K": 4096, "F": 11008, "act": "silu", "bias": False, "dtype": "f16"},
        # a small decode batch
        {"name": "gated_batch", "op": "gated", "M": 16, "K": 4096, "F": 11008, "act": "gelu", "bias": False, "dtype": "bf16"},
        # a mixed batch of odd length, with a bias
        {"name": "gated_mixed", "op": "gated", "M": 333, "K": 5120, "F": 13824, "act": "gelu_tanh", "bias": True, "dtype": "bf16"},
        # a long prompt: the matrix rate
        {"name": "gated_prompt", "op": "gated", "M": 8192, "K": 5120, "F": 27648, "act": "silu", "bias": False, "dtype": "bf16"},
        # ---- a beam's step over the pages: `seqs` sequences, `beams` children each, `layers` caches
        # one prompt and four beams, one cache: latency
        {"name": "beam_one", "op": "beam", "seqs": 1, "beams": 4, "ctx": 777, "layers": 1, "Hkv": 32, "D": 128, "T": 16, "spare": 400},
        # a batch of sequences, the caches of a whole model
        {"name": "beam_batch", "op": "beam", "seqs": 24, "beams": 5, "ctx": 4000, "layers": 16, "Hkv": 8, "D": 128, "T": 64, "spare": 700},
        # ---- compaction; used: share of the pool in use
        # a small cache, nearly full
        {"name": "compact_one", "op": "compact", "B": 9, "ctx": 500, "layers": 1, "Hkv": 8, "D": 64, "T": 16, "used": 0.8},
        # a pool after half of its sequences have ended, several caches
        {"name": "compact_batch", "op": "compact", "B": 48, "ctx": 6000, "layers": 4, "Hkv": 8, "D": 128, "T": 64, "used": 0.5},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scored", "scored", "gated", "gated", "beam", "compact"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "gated":
        K = 16 * _log_int(rng, 32, 1728)
        F = 8 * _log_int(rng, 16, 3456)
        M = _log_int(rng, 1, min(8192, 1_150_000_000_000 // (F * K)))
        return {"op": op, "M": M, "K": K, "F": F, "act": rng.choice(["silu", "gelu", "gelu_tanh"]),
                "bias": rng.random() < 0.5, "dtype": dtype}
    Hkv = rng.choice([1, 2, 4, 8, 16, 32])
    D = rng.choice([64, 128])
    T = rng.choice([16, 32, 64, 128])
    if op == "beam":
        seqs, beams = _log_int(rng, 1, 40), rng.randint(1, 8)
        layers = _log_int(rng, 1, max(1, min(32, 4_000_000_000 // (seqs * (beams + 2) * 128 * 2 * Hkv * D))))
        tokens = 12_000_000_000 // (2 * Hkv * D * layers) - seqs * (beams + 2) * T
        return {"op": op, "seqs": seqs, "beams": beams, "ctx": _log_int(rng, 1, max(2, min(8000, tokens // seqs))),
                "layers": layers, "Hkv": Hkv, "D": D, "T": T, "spare": seqs * beams * 2 + _log_int(rng, 1, 200)}
    if op == "compact":
        B, used = _log_int(rng, 1, 64), rng.uniform(0.2, 0.95)
        layers = rng.randint(1, 8)
        ctx = _log_int(rng, 10, max(11, min(8000, int(used * 8_000_000_000 / (B * 2 * Hkv * D * layers)) - T)))
        return {"op": op, "B": B, "ctx": ctx, "layers": layers, "Hkv": Hkv, "D": D, "T": T, "used": used}
    H = Hkv * rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16, 32) if g * Hkv <= 64])
    form = rng.choice(["token", "few", "chunk"])
    if form == "chunk":
        B = rng.randint(1, 4)
        new = _log_int(rng, 17, 2048)
        ctx = new + _log_int(rng, 1, 6144)
        H, Hkv = min(H, 40), min(Hkv, 40)
        H -= H % Hkv
    else:
        B = _log_int(rng, 1, 64)
        new = 1 if form == "token" else rng.randint(2, 16)
        ctx = new + _log_int(rng, 1, max(2, min(131000, 500_000_000 // (B * H * D * new))))
        ctx = min(ctx, max(new, 400_000_000 // (B * Hkv * D)))
    return {"op": op, "B": B, "new": new, "ctx": ctx, "H": H, "Hkv": Hkv, "D": D, "T": T,
            "cap": rng.choice([0.0, 20.0, 30.0, 50.0]), "slopes": rng.random() < 0.5,
            "doc": 0 if rng.random() < 0.5 else _log_int(rng, 16, max(17, ctx)),
            "prefix": 0.0 if rng.random() < 0.6 else rng.uniform(0.1, 1.0), "dtype": dtype}


# --------------------------------------------------- what a case stands for ---

def _sequences(case):
    """Of each sequence: its length with the new tokens, their count, the
    position at which each new token's document begins, and the prefix."""
    r = random.Random(1000 * case["B"] + case["ctx"] + case["new"])
    got = []
    for b in range(case["B"]):
        n = case["new"] if b == 0 or case["new"] == 1 else max(1, int(case["new"] * r.uniform(0.4, 1.0)))
        n0 = case["ctx"] - case["new"]
        old = n0 if b == 0 else int(n0 * r.uniform(0.3, 1.0))
        starts = [0]
        while case["doc"]:
            at = starts[-1] + max(1, int(case["doc"] * r.uniform(0.3, 1.7)))
            if at >= old + n:
                break
            starts.append(at)
        first, i = [], 0
        for p in range(old, old + n):
            while i + 1 < len(starts) and starts[i + 1] <= p:
                i += 1
            first.append(starts[i])
        got.append((old + n, n, first, old + int(case["prefix"] * n) if case["prefix"] else 0))
    return got


def _beam_lens(case):
    r = random.Random(7 * case["seqs"] + case["ctx"])
    return [case["ctx"] if s == 0 else max(1, int(case["ctx"] * r.uniform(0.3, 1.0))) for s in range(case["seqs"])]


def _compact_rows(case):
    """(length, row whose whole pages it shares or -1) of each table row."""
    r = random.Random(13 * case["B"] + case["ctx"])
    rows = []
    for b in range(case["B"]):
        if b % 6 == 5:      # a forked row
            rows.append((max(1, int(rows[-1][0] * r.uniform(0.9, 1.0))), b - 1))
        else:
            rows.append((case["ctx"] if b == 0 else max(1, int(case["ctx"] * r.uniform(0.2, 1.0))), -1))
    return rows


def _compact_pool(case):
    """Pages in use and in the pool (a multiple of 4: the arrays of every
    cache begin at 16 bytes)."""
    T = case["T"]
    used = 0
    for L, share in _compact_rows(case):
        used += -(-L // T) - (L // T if share >= 0 else 0)
    return used, -(-max(used + 1, int(used / case["used"])) // 4) * 4


def work(case):
    if case["op"] == "gated":
        M, F, K = case["M"], case["F"], case["K"]
        return {"bytes": 2 * M * K + 2 * F * K + 8 * F + 2 * M * F + (4 * F if case["bias"] else 0),
                "flops": 4 * M * F * K}
    T, Hkv, D = case["T"], case["Hkv"], case["D"]
    page = 2 * Hkv * D * T + 8 * Hkv
    if case["op"] == "beam":
        # partly filled pages read once for each sequence and written for each child; the rows of
        # the table read for each sequence and written for each child; the counters
        lens, n = _beam_lens(case), case["beams"]
        half = sum(1 for L in lens if L % T)
        entries = sum(-(-L // T) for L in lens)
        return {"bytes": case["layers"] * page * half * (n + 1) + 4 * entries * (n + 1) + 8 * entries, "flops": 0}
    if case["op"] == "compact":
        used, pool = _compact_pool(case)
        # with pages in use anywhere in the pool, those above `used` move
        moved = used * (pool - used) // pool
        entries = sum(-(-L // T) for L, _ in _compact_rows(case))
        return {"bytes": case["layers"] * page * moved * 2 + 8 * entries + 8 * pool, "flops": 0}
    keys = tokens = pairs = 0
    for L, n, first, prefix in _sequences(case):
        ends = [max(p + 1, min(prefix, L)) for p in range(L - n, L)]
        keys += max(ends) - min(first)
        tokens += n
        pairs += sum(e - f for e, f in zip(ends, first))
    return {"bytes": 2 * keys * Hkv * D + 4 * tokens * case["H"] * D, "flops": 4 * D * case["H"] * pairs}


# ------------------------------------------------------------------- inputs ---

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _codes(x, dims):
    """Codes (uint8, + 128) and scales of x with one scale over ``dims``."""
    s = x.abs().amax(dims, keepdim=True) * INV127
    return (torch.round(x / s).clamp(-127, 127) + 128).to(torch.uint8), s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"gated": _prepare_gated, "scored": _prepare_scored, "beam": _prepare_beam,
            "compact": _prepare_compact}[case["op"]](case, gen)


def _prepare_gated(case, gen):
    M, F, K, dt = case["M"], case["F"], case["K"], DT[case["dtype"]]
    # activations with a few strong channels, weights of a layer, quantized per channel
    x = _randn(gen, M, K)
    x *= torch.where(torch.rand(K, generator=gen, device=DEV) < 0.01, 12.0, 1.0)
    w = _randn(gen, 2 * F, K) * 0.02
    ws = w.abs().amax(1) * INV127
    wq = torch.round(w / ws[:, None]).clamp(-127, 127).to(torch.int8)
    bias = (_randn(gen, 2 * F) * 0.5).to(dt) if case["bias"] else None
    return {"case": case, "x": x.to(dt), "wq": wq, "ws": ws, "bias": bias}


def _prepare_scored(case, gen):
    B, H, Hkv, D, T = case["B"], case["H"], case["Hkv"], case["D"], case["T"]
    seqs = _sequences(case)
    counts = [-(-s[0] // T) for s in seqs]
    pages, width = sum(counts) + 3, max(counts)
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    news = [s[1] for s in seqs]
    # keys with a few strong channels, values without
    strong = torch.where(torch.rand(Hkv, 1, D, generator=gen, device=DEV) < 0.03, 4.0, 1.0)
    kc = torch.empty(pages, Hkv, T, D, dtype=torch.uint8, device=DEV)
    vc = torch.empty(pages, Hkv, T // 16, D, 16, dtype=torch.uint8, device=DEV)
    ks, vs = torch.empty(pages, Hkv, device=DEV), torch.empty(pages, Hkv, device=DEV)
    step = max(1, (1 << 27) // (Hkv * T * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        c, s = _codes(_randn(gen, n, Hkv, T, D) * strong, (2, 3))
        kc[p:p + n], ks[p:p + n] = c, s.view(n, Hkv)
        c, s = _codes(_randn(gen, n, Hkv, T // 16, D, 16), (2, 3, 4))
        vc[p:p + n], vs[p:p + n] = c, s.view(n, Hkv)
    cache = {"page_size": T, "kv_heads": Hkv, "head_dim": D, "num_pages": pages,
             "k": kc, "v": vc, "k_scale": ks, "v_scale": vs}
    # scores large enough for the cap to bend them; slopes as they are spread over heads, 2^-8 to 1/2
    q = (_randn(gen, sum(news), H, D) * (4.0 if case["cap"] else 1.2)).to(DT[case["dtype"]])
    slopes = 2.0 ** (-8.0 * torch.arange(1, H + 1, device=DEV, dtype=torch.float32) / H) if case["slopes"] else None
    return {"case": case, "cache": cache, "table": table, "lens": _ints([s[0] for s in seqs]),
            "cu": torch.tensor([0] + news).cumsum(0).to(torch.int32).to(DEV), "q": q, "max_new": max(news),
            "max_len": max(s[0] for s in seqs), "slopes": slopes,
            "first": _ints([f for s in seqs for f in s[2]]) if case["doc"] else None,
            "prefix": _ints([s[3] for s in seqs]) if case["prefix"] else None}


def _caches(case, pages, gen):
    """The caches of all layers, side by side in memory."""
    L, Hkv, D, T = case["layers"], case["Hkv"], case["D"], case["T"]
    k = torch.randint(0, 256, (L, pages, Hkv, T, D), generator=gen, device=DEV, dtype=torch.uint8)
    v = torch.randint(0, 256, (L, pages, Hkv, T // 16, D, 16), generator=gen, device=DEV, dtype=torch.uint8)
    ks = torch.rand(L, pages, Hkv, generator=gen, device=DEV)
    vs = torch.rand(L, pages, Hkv, generator=gen, device=DEV)
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs,
            "list": [{"k": k[i], "v": v[i], "k_scale": ks[i], "v_scale": vs[i], "page_size": T, "kv_heads": Hkv,
                      "head_dim": D, "num_pages": pages} for i in range(L)]}


def _prepare_beam(case, gen):
    T, S, n = case["T"], case["seqs"], case["beams"]
    lens = _beam_lens(case)
    counts = [-(-L // T) for L in lens]
    pages = -(-(sum(counts) + case["spare"]) // 4) * 4
    width = max(counts) + 2
    # the sequences first, then their children, empty so far
    table = torch.full((S + S * n, width), -1, dtype=torch.int32, device=DEV)
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    at = 0
    for s, c in enumerate(counts):
        table[s, :c] = order[at:at + c]
        at += c
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[order[:at].long()] = 1
    src = [s for s in range(S) for _ in range(n)]
    return {"case": case, "caches": _caches(case, pages, gen), "refs": refs, "table": table,
            "lens": _ints(lens + [0] * (S * n)), "src": _ints(src), "dst": _ints(range(S, S + S * n)),
            "added": _ints([0] * S + [1] * (S * n))}


def _prepare_compact(case, gen):
    T = case["T"]
    rows = _compact_rows(case)
    used, pool = _compact_pool(case)
    order = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    refs = torch.zeros(pool, dtype=torch.int32, device=DEV)
    table = torch.full((len(rows), max(-(-L // T) for L, _ in rows)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, (L, share) in enumerate(rows):
        whole = L // T if share >= 0 else 0
        table[b, :whole] = table[share, :whole]
        c = -(-L // T) - whole
        table[b, whole:whole + c] = order[at:at + c]
        refs[table[b, :whole + c].long()] += 1
        at += c
    return {"case": case, "caches": _caches(case, pool, gen), "refs": refs, "table": table,
            "lens": _ints([L for L, _ in rows])}


def run(state):
    case = state["case"]
    if own:
        import bit_weight_only_gemm_amd as w4
        if case["op"] == "gated":
            return w4.w8a8_gated(state["x"], state["wq"], state["ws"], bias=state["bias"], act=case["act"])
        if case["op"] == "scored":
            cu = None if case["new"] == 1 else state["cu"]
            return w4.kv8_attention_scored(state["q"], state["cache"], state["table"], state["lens"], cu_seqlens=cu,
                                           max_new=state["max_new"], max_len=state["max_len"], softcap=case["cap"],
                                           slopes=state["slopes"], first=state["first"], prefix=state["prefix"])
        caches, refs, table, lens = (state[n] for n in ("caches", "refs", "table", "lens"))
        if case["op"] == "beam":
            w4.kv8_free(refs, table, lens, state["dst"], case["T"])
            short = w4.kv8_fork(caches["list"], refs, table, lens, state["src"], state["dst"])
            short2 = w4.kv8_reserve(refs, table, lens, state["added"], case["T"])
            return _pages_out(state, table, refs, {"lens": lens, "short": [short, short2]})
        table, refs, used = w4.kv8_compact(caches["list"], refs, table, lens)
        return _pages_out(state, table, refs, {"used": used})
    return {"gated": _plain_gated, "scored": _plain_scored, "beam": _plain_beam,
            "compact": _plain_compact}[case["op"]](state)


def _pages_out(st, table, refs, more):
    """What a pass over the pages leaves.  Pages move as they are: their codes
    are compared as whole numbers."""
    c = st["caches"]
    return {"table": table, "refs": refs, "k": c["k"], "v": c["v"], "k_scale": c["k_scale"], "v_scale": c["v_scale"],
            **more}


# -------------------------------------------------------------- plain forms ---

def _plain_gated(st):
    x = st["x"].float()
    xs = x.abs().amax(1, keepdim=True) * INV127
    xs = torch.where(xs == 0, 1.0, xs)
    y = (torch.round(x / xs).clamp(-127, 127) @ st["wq"].float().t()) * xs * st["ws"]
    if st["bias"] is not None:
        y = y + st["bias"].float()
    g, u = y.chunk(2, 1)
    act = st["case"]["act"]
    if act == "silu":
        a = g / (1.0 + torch.exp(-g))
    elif act == "gelu":
        a = 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    else:
        a = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))
    return (a * u).to(st["x"].dtype)


def _plain_scored(st):
    case, cache = st["case"], st["cache"]
    B, H, Hkv, D, T = case["B"], case["H"], case["Hkv"], case["D"], case["T"]
    table = st["table"].clamp(min=0).long()
    L, G, n = table.shape[1] * T, H // Hkv, st["max_new"]
    k = cache["k"][table].float().sub_(128).mul_(cache["k_scale"][table][..., None, None])
    k = k.permute(0, 2, 4, 1, 3).reshape(B, Hkv, D, L)
    v = cache["v"][table].float().sub_(128).mul_(cache["v_scale"][table][..., None, None, None])
    v = v.permute(0, 2, 1, 3, 5, 4).reshape(B, Hkv, L, D)
    count = st["cu"][1:] - st["cu"][:-1]
    j = torch.arange(n, device=DEV)
    src = (st["cu"][:-1, None] + j).clamp(max=st["q"].shape[0] - 1).long()
    q = st["q"][src].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    s = torch.matmul(q, k).mul_(1.0 / math.sqrt(D)).view(B, Hkv, G, n, L)
    if case["cap"]:
        s.div_(case["cap"]).tanh_().mul_(case["cap"])
    pos = (st["lens"] - count)[:, None] + j
    at = torch.arange(L, device=DEV)
    if case["slopes"]:
        far = (pos[:, :, None] - at).abs().float()
        s.addcmul_(st["slopes"].view(Hkv, G, 1, 1), far[:, None, None], value=-1.0)
    end = pos + 1
    if st["prefix"] is not None:
        end = torch.maximum(end, torch.minimum(st["prefix"], st["lens"])[:, None])
    seen = at < end[:, :, None]
    if st["first"] is not None:
        seen &= at >= st["first"][src][:, :, None]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = s.sub_(m).exp_()
    o = torch.matmul(p.view(B, Hkv, G * n, L), v).view(B, Hkv, G, n, D)
    z = p.sum(-1, keepdim=True)
    o = torch.where(z > 0, o / z, 0.0).permute(0, 3, 1, 2, 4).reshape(B, n, H, D)
    tok = torch.arange(st["q"].shape[0], device=DEV)
    seq = torch.searchsorted(st["cu"][1:].contiguous(), tok.int(), right=True)
    return o[seq, tok - st["cu"][seq].long()].to(DT[case["dtype"]])


def _copy_pages(st, src, dst):
    for name in ("k", "v", "k_scale", "v_scale"):
        a = st["caches"][name]
        a[:, dst] = a[:, src]


def _plain_beam(st):
    refs, table, lens, T = st["refs"], st["table"], st["lens"], st["case"]["T"]
    src, dst = st["src"].long(), st["dst"].long()
    at = torch.arange(table.shape[1], device=DEV)
    # the children's pages go back
    held = at < ((lens[dst] + T - 1) // T)[:, None]
    old = table[dst]
    refs.index_add_(0, torch.where(held, old, 0).flatten().long(), -held.flatten().int())
    table[dst] = torch.where(held, -1, old)
    lens[dst] = 0
    # whole pages shared, the last one copied where it is partly filled
    free = (refs == 0).nonzero().flatten()
    whole, half = lens[src] // T, lens[src] % T != 0
    rank = half.cumsum(0) - 1
    short = (half.sum() - free.numel()).clamp(min=0).int().view(1)
    fresh = free[rank.clamp(min=0)]
    shared = at < whole[:, None]
    rows = table[src]
    refs.index_add_(0, torch.where(shared, rows, 0).flatten().long(), shared.flatten().int())
    last = (at == whole[:, None]) & half[:, None]
    table[dst] = torch.where(last, fresh[:, None].int(), torch.where(shared, rows, table[dst]))
    lens[dst] = lens[src]
    taken, kids = fresh[half], src[half]
    refs[taken] = 1
    _copy_pages(st, table[kids, whole[half].long()].long(), taken)
    # room for the next token
    free = (refs == 0).nonzero().flatten()
    have, want = (lens + T - 1) // T, (lens + st["added"] + T - 1) // T
    need = want - have
    end = need.cumsum(0)
    short2 = (end[-1] - free.numel()).clamp(min=0).int().view(1)
    get = (at >= have[:, None]) & (at < want[:, None])
    pick = free[(end - need)[:, None].add(at - have[:, None]).clamp(0, free.numel() - 1)]
    table.copy_(torch.where(get, pick.int(), table))
    refs[pick[get]] = 1
    lens += st["added"]
    return _pages_out(st, table, refs, {"lens": lens, "short": [short, short2]})


def _plain_compact(st):
    refs, table, lens, T = st["refs"], st["table"], st["lens"], st["case"]["T"]
    used = refs > 0
    count = used.sum()
    ids = torch.arange(refs.numel(), device=DEV)
    high, low = ids >= count, ids < count
    movers, holes = (used & high).nonzero().flatten(), (~used & low).nonzero().flatten()
    to = ids.clone()
    to[movers] = holes
    held = torch.arange(table.shape[1], device=DEV) < ((lens + T - 1) // T)[:, None]
    table = torch.where(held, to[table.clamp(min=0).long()].int(), table)
    refs = refs.clone()
    refs[holes] = refs[movers]
    refs[movers] = 0
    _copy_pages(st, movers, holes)
    return _pages_out(st, table, refs, {"used": count.int().view(1)})


# ------------------------------------------------ the definition, in 64 bits ---

def exact(case, seed):
    st = prepare(case, seed)
    return {"gated": _exact_gated, "scored": _exact_scored, "beam": _exact_beam, "compact": _exact_compact}[case["op"]](case, st)


def _exact_pages(st, table, refs, moved, more):
    """The arrays after pages moved, (from, to) pairs of them; the scales in 64 bits."""
    c = dict(st["caches"])
    for name in ("k", "v", "k_scale", "v_scale"):
        a = c[name].double() if name.endswith("scale") else c[name].clone()
        if moved:
            src, dst = (torch.tensor(t, device=DEV) for t in zip(*moved))
            a[:, dst] = a[:, src]
        c[name] = a
    return _pages_out({"caches": c}, _ints(table), _ints(refs), more)


def _exact_beam(case, st):
    T, table, refs, lens = case["T"], st["table"].tolist(), st["refs"].tolist(), st["lens"].tolist()

    def take():
        page = refs.index(0)
        refs[page] = 1
        return page

    moved = []
    for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
        for i in range(lens[s] // T):
            table[d][i] = table[s][i]
            refs[table[s][i]] += 1
        if lens[s] % T:
            table[d][lens[s] // T] = take()
            moved.append((table[s][lens[s] // T], table[d][lens[s] // T]))
        lens[d] = lens[s]
    for b, n in enumerate(st["added"].tolist()):
        for i in range(-(-lens[b] // T), -(-(lens[b] + n) // T)):
            table[b][i] = take()
        lens[b] += n
    return _exact_pages(st, table, refs, moved, {"lens": _ints(lens), "short": [_ints([0]), _ints([0])]})


def _exact_compact(case, st):
    T, table, refs = case["T"], st["table"].tolist(), st["refs"].tolist()
    used = sum(n > 0 for n in refs)
    holes = [p for p in range(used) if refs[p] == 0]
    to = dict(zip((p for p in range(used, len(refs)) if refs[p]), holes))
    for b, L in enumerate(st["lens"].tolist()):
        for i in range(-(-L // T)):
            table[b][i] = to.get(table[b][i], table[b][i])
    for p, q in to.items():
        refs[p], refs[q] = 0, refs[p]
    return _exact_pages(st, table, refs, list(to.items()), {"used": _ints([used])})


def _exact_gated(case, st):
    x, F = st["x"].double(), case["F"]
    step = x.abs().max(dim=1).values / 127
    step[step == 0] = 1
    codes = (x / step[:, None]).round()
    out = torch.empty(case["M"], F, dtype=torch.float64, device=DEV)
    for f in range(0, F, 8192):
        e = min(f + 8192, F)
        part = []
        for rows in (slice(f, e), slice(F + f, F + e)):
            w = st["wq"][rows].double() * st["ws"][rows].double()[:, None]
            y = torch.mm(codes, w.t().contiguous()).mul_(step[:, None])
            part.append(y if st["bias"] is None else y.add_(st["bias"][rows].double()))
        g, u = part
        if case["act"] == "silu":
            g = g * torch.sigmoid(g)
        elif case["act"] == "gelu":
            g = g * torch.special.ndtr(g)
        else:
            g = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
        out[:, f:e] = g * u
    return out


def _exact_scored(case, st):
    H, Hkv, D, T = case["H"], case["Hkv"], case["D"], case["T"]
    G, cache = H // Hkv, st["cache"]
    seqs, table = _sequences(case), st["table"].tolist()
    if 4 * D * H * sum(L * n for L, n, _, _ in seqs) > 40e12:
        return None
    out = torch.empty(st["q"].shape[0], H, D, dtype=torch.float64, device=DEV)
    at = 0
    for b, (L, n, first, prefix) in enumerate(seqs):
        ids = torch.tensor(table[b][:-(-L // T)], device=DEV)
        k = (cache["k"][ids].double() - 128) * cache["k_scale"][ids].double()[:, :, None, None]
        v = (cache["v"][ids].double() - 128) * cache["v_scale"][ids].double()[:, :, None, None, None]
        k = k.transpose(0, 1).reshape(Hkv, -1, D)[:, :L]
        v = v.permute(1, 0, 2, 4, 3).reshape(Hkv, -1, D)[:, :L]
        p, l = torch.arange(L - n, L, device=DEV)[:, None], torch.arange(L, device=DEV)[None, :]
        hide = (l > p) & (l >= prefix)
        if case["doc"]:
            hide |= l < torch.tensor(first, device=DEV)[:, None]
        far = (p - l).abs().double()
        for h in range(H):
            s = torch.mm(st["q"][at:at + n, h].double(), k[h // G].t().contiguous()) / D ** 0.5
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            if case["slopes"]:
                s = s - 2.0 ** (-8.0 * (h + 1) / H) * far
            s[hide] = -math.inf
            out[at:at + n, h] = torch.mm(torch.softmax(s, 1), v[h // G].contiguous())
        at += n
    return out
