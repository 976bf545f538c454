"""A paged key/value cache in 8 bits, one scale per (page, kv head): the append
that fills it and the attention that reads it (the ``kv8_*`` entry points of
``include/w4a16.h``).

    cache = kv8_cache(num_pages, 64, kv_heads, head_dim)
    q = kv8_append(cache, k, v, page_table, seq_lens, q=q, cos=cos, sin=sin)
    o = kv8_attention(q, cache, page_table, seq_lens)

(kv8_attention_scored: with capped scores, a bias by distance, document and
prefix masks.)  page_table int32 [B, max_pages], seq_lens int32 [B] (the new tokens included)
and cu_seqlens int32 [B + 1] stay on the device; without cu_seqlens each
sequence has one new token.  Rows of q, k and v are [tokens, heads, D] and may
be slices of a fused projection.

(A decode step's calls are short: the checks below look at each tensor once.)
"""

import math

import torch

from . import _DT, _here, _lib, _need, _stream
from .w8a8 import _empty, _space


# Workspaces of kv8_attention by (device, stream): it keeps counters in them,
# zero between calls, so no other operator writes there.
_COUNTED = {}


def kv8_cache(num_pages, page_size, kv_heads, head_dim, device="cuda"):
    """An empty cache: dict(k, v, k_scale, v_scale, page_size, kv_heads,
    head_dim, num_pages); k uint8 [pages, Hkv, T, D], v uint8 [pages, Hkv,
    T / 16, D, 16], a code c standing for (c - 128) * scale [pages, Hkv]."""
    T, D = page_size, head_dim
    if T not in (16, 32, 64, 128) or D not in (64, 128):
        raise _lib.W4A16Error("kv8_cache: unsupported page_size %d or head_dim %d" % (T, D))
    n = (num_pages, kv_heads)
    return {"k": torch.full((*n, T, D), 128, dtype=torch.uint8, device=device),
            "v": torch.full((*n, T // 16, D, 16), 128, dtype=torch.uint8, device=device),
            "k_scale": torch.zeros(n, device=device), "v_scale": torch.zeros(n, device=device),
            "page_size": T, "kv_heads": kv_heads, "head_dim": D, "num_pages": num_pages}


def _cache(c):
    """The cache's sizes and the addresses of its arrays."""
    pages, Hkv, T, D = c["num_pages"], c["kv_heads"], c["page_size"], c["head_dim"]
    k, v, ks, vs = c["k"], c["v"], c["k_scale"], c["v_scale"]
    _need(k, torch.uint8, "cache k", pages * Hkv * T * D)
    _need(v, torch.uint8, "cache v", pages * Hkv * T * D)
    _need(ks, torch.float32, "cache k_scale", pages * Hkv)
    _need(vs, torch.float32, "cache v_scale", pages * Hkv)
    return pages, Hkv, T, D, (k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr())


def _heads(t, dtype, name, tokens=None, heads=None, D=None):
    """Checks rows [tokens, heads, D], contiguous within a token; (tokens,
    heads, row stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    if t.dtype not in _DT or (dtype is not None and t.dtype != dtype):
        raise TypeError("%s must be %s, got %s" % (name, dtype or "float16 or bfloat16", t.dtype))
    if t.dim() != 3:
        raise ValueError("%s must be [tokens, heads, D]" % name)
    n, h, d = t.shape
    if d != D or (tokens is not None and n != tokens) or (heads is not None and h != heads):
        raise ValueError("%s has shape %s, expected [%s, %s, %d]"
                         % (name, tuple(t.shape), tokens or "tokens", heads or "heads", D))
    if t.is_contiguous():
        return n, h, h * D
    step, head, one = t.stride()
    if n and (one != 1 or (h > 1 and head != D)):
        raise ValueError("%s must be contiguous within a token" % name)
    return n, h, step if n > 1 else h * D


def _sequences(page_table, seq_lens, cu_seqlens, max_new, tokens):
    _need(page_table, torch.int32, "page_table")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, width = page_table.shape
    _need(seq_lens, torch.int32, "seq_lens", B)
    if cu_seqlens is None:
        if tokens != B:
            raise ValueError("%d tokens for %d sequences: pass cu_seqlens" % (tokens, B))
        return B, width, 1 if B else 0, None
    _need(cu_seqlens, torch.int32, "cu_seqlens", B + 1)
    return B, width, tokens if max_new is None else min(int(max_new), tokens), cu_seqlens.data_ptr()


def kv8_append(cache, k, v, page_table, seq_lens, cu_seqlens=None, max_new=None, q=None,
               cos=None, sin=None, interleaved=False, q_out=None, stream=None):
    """Appends k, v [tokens, Hkv, D] to the cache, the keys rotated by their
    positions (cos, sin fp32 [positions, rope_dim / 2]), and returns the
    rotated queries q [tokens, H, D] (None without q).  max_new: an upper bound
    of the new tokens of one sequence (all of them when not given; the kernel
    for single tokens runs where it is 1); rows past it are not processed."""
    pages, Hkv, T, D, arrays = _cache(cache)
    tokens, _, k_stride = _heads(k, None, "k", None, Hkv, D)
    dtype = k.dtype
    _, _, v_stride = _heads(v, dtype, "v", tokens, Hkv, D)
    B, width, max_new, cu = _sequences(page_table, seq_lens, cu_seqlens, max_new, tokens)
    H, q_at, q_stride, o_at, o_stride = Hkv, None, 0, None, 0
    if q is not None:
        _, H, q_stride = _heads(q, dtype, "q", tokens, None, D)
        if q_out is None:
            q_out = _empty((tokens, H, D), dtype, q.device, stream)
            o_stride = H * D
        else:
            _, _, o_stride = _heads(q_out, dtype, "q_out", tokens, H, D)
        q_at, o_at = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rows = dim = 0
    cos_at = sin_at = None
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        _need(cos, torch.float32, "cos")
        _need(sin, torch.float32, "sin", cos.numel())
        if cos.dim() != 2:
            raise ValueError("cos must be [positions, rope_dim / 2]")
        rows, dim = cos.shape
        dim *= 2
        cos_at, sin_at = cos.data_ptr(), sin.data_ptr()
    status = _lib.lib().kv8_append(
        q_at, q_stride, o_at, o_stride, k.data_ptr(), k_stride, v.data_ptr(), v_stride, *arrays,
        pages, T, page_table.data_ptr(), width, seq_lens.data_ptr(), cu, cos_at, sin_at, rows, dim,
        1 if interleaved else 0, tokens, B, max_new, H, Hkv, D, _DT[dtype], _stream(stream))
    if status:
        _lib.check(status, "kv8_append")
    return q_out


def kv8_dequant(cache, pages, dtype=torch.bfloat16, stream=None):
    """The values of pages (int32 [n]) of the cache: k, v [n, Hkv, T, D]."""
    num, Hkv, T, D, arrays = _cache(cache)
    if dtype not in _DT:
        raise TypeError("dtype must be float16 or bfloat16")
    _need(pages, torch.int32, "pages")
    n = pages.numel()
    shape, device = (n, Hkv, T, D), pages.device
    k, v = _empty(shape, dtype, device, stream), _empty(shape, dtype, device, stream)
    status = _lib.lib().kv8_dequant(*arrays, num, T, Hkv, D, pages.data_ptr(), n, _DT[dtype],
                                    k.data_ptr(), v.data_ptr(), _stream(stream))
    if status:
        _lib.check(status, "kv8_dequant")
    return k, v


def kv8_attention_workspace_bytes(tokens, B, max_new, max_len, heads, kv_heads, head_dim):
    n = int(_lib.lib().kv8_attention_workspace_bytes(tokens, B, max_new, max_len, heads, kv_heads,
                                                     head_dim))
    if n < 0:
        raise _lib.W4A16Error("kv8_attention_workspace_bytes: invalid sizes")
    return n


def kv8_attention(q, cache, page_table, seq_lens, cu_seqlens=None, max_new=None, max_len=None,
                  scale=None, causal=True, out=None, lse=None, workspace=None, stream=None):
    """Attention of q [tokens, H, D] over the cached tokens of their sequences:
    [tokens, H, D] in q's dtype.  scale: 1 / sqrt(D) when not given; max_new,
    max_len: upper bounds of the new tokens and of the length of one sequence
    (all tokens, the table's width), by which the kernel and the split of the
    keys are chosen: pass them where cu_seqlens is.  Rows past max_new are not
    processed.  lse: fp32 [tokens, H], written if given.  workspace: one of
    kv8_attention_workspace_bytes, kept for these calls alone and zero before
    the first (one per stream is kept when not given; a call that is captured
    finds it there from a call before, or is given one): it holds counters, and
    one that another operator has written in leaves results unwritten."""
    return _attention("kv8_attention", None, q, cache, page_table, seq_lens, cu_seqlens, max_new,
                      max_len, scale, causal, out, lse, workspace, stream)


def kv8_attention_scored(q, cache, page_table, seq_lens, cu_seqlens=None, max_new=None,
                         max_len=None, scale=None, causal=True, softcap=0.0, slopes=None,
                         first=None, prefix=None, out=None, lse=None, workspace=None, stream=None,
                         end=None):
    """kv8_attention of scores s = scale q . k that become softcap tanh(s /
    softcap) (0 or None: as they are), less slopes[h] |distance| (fp32 [H]).
    first (int32 [tokens]): the first position that each query sees, the start of
    its document or of a window.  prefix (int32 [B]): with causal, positions below
    it are seen by every query of the sequence.  end (int32 [tokens]): no query
    sees this position or those after it; documents that share a sequence need it
    beside first where they are seen both ways (causal=False, or a prefix, which
    reaches into the documents after a query's own).  A query that sees nothing
    gives 0.  The other arguments as for kv8_attention, its workspace among them."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [tokens, heads, D]")
    _need(seq_lens, torch.int32, "seq_lens")
    extra = [0.0 if softcap is None else float(softcap), None, None, None, None]
    for i, (t, dtype, name, n) in enumerate(((slopes, torch.float32, "slopes", q.shape[1]),
                                             (first, torch.int32, "first", q.shape[0]),
                                             (end, torch.int32, "end", q.shape[0]),
                                             (prefix, torch.int32, "prefix", seq_lens.numel()))):
        if t is not None:
            _need(t, dtype, name, n)
            extra[1 + i] = t.data_ptr()
    _here(stream, q, cache["k"], page_table, seq_lens, cu_seqlens, slopes, first, end, prefix, out,
          lse, workspace)
    name = "kv8_attention_scored"
    if end is None:
        del extra[3]
    else:
        name += "_ends"
    return _attention(name, extra, q, cache, page_table, seq_lens, cu_seqlens, max_new, max_len,
                      scale, causal, out, lse, workspace, stream)


def _attention(name, extra, q, cache, page_table, seq_lens, cu_seqlens, max_new, max_len, scale,
               causal, out, lse, workspace, stream):
    pages, Hkv, T, D, arrays = _cache(cache)
    tokens, H, q_stride = _heads(q, None, "q", None, None, D)
    dtype = q.dtype
    B, width, max_new, cu = _sequences(page_table, seq_lens, cu_seqlens, max_new, tokens)
    max_len = width * T if max_len is None else min(int(max_len), width * T)
    if out is None:
        out = _empty((tokens, H, D), dtype, q.device, stream)
        o_stride = H * D
    else:
        _, _, o_stride = _heads(out, dtype, "out", tokens, H, D)
    if lse is not None:
        _need(lse, torch.float32, "lse", tokens * H)
    L = _lib.lib()
    need = L.kv8_attention_workspace_bytes(tokens, B, max_new, max_len, H, Hkv, D)
    workspace, nbytes = _space(workspace, need, q.device, stream, _COUNTED)
    status = getattr(L, name)(
        q.data_ptr(), q_stride, *arrays, pages, T, page_table.data_ptr(), width,
        seq_lens.data_ptr(), cu, 1.0 / math.sqrt(D) if scale is None else float(scale),
        1 if causal else 0, *(extra or ()), out.data_ptr(), o_stride,
        None if lse is None else lse.data_ptr(), tokens, B, max_new, max_len, H, Hkv, D, _DT[dtype],
        None if workspace is None else workspace.data_ptr(), nbytes, _stream(stream))
    if status:
        _lib.check(status, name)
    return out
