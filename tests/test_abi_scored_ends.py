"""Host-only checks of kv8_attention_scored_ends (an end of what each query sees),
and its oracle against the definition of a document mask."""

import ctypes
import os

import numpy as np
import pytest

from bit_weight_only_gemm_amd import _lib
from oracle import kv8

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libw4a16.so not built", allow_module_level=True)

L = _lib.load()
NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(0x10000)        # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x10008)         # misaligned
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 5


def call(q=FAKE, q_stride=256, pages=8, T=16, table=FAKE, width=4, cap=0.0, slopes=NULL, first=NULL, end=FAKE,
         prefix=NULL, out=FAKE, tokens=2, B=2, max_new=1, max_len=64, D=64, dtype=0, space=NULL, nbytes=0):
    return L.kv8_attention_scored_ends(q, q_stride, FAKE, FAKE, FAKE, FAKE, pages, T, table, width, FAKE, NULL, 0.125,
                                       1, cap, slopes, first, end, prefix, out, 256, NULL, tokens, B, max_new, max_len,
                                       4, 2, D, dtype, space, nbytes, NULL)


def test_refusals_and_workspace():
    for bad in (dict(cap=-1.0), dict(cap=float("nan")), dict(tokens=3), dict(max_len=65), dict(q=NULL), dict(out=NULL),
                dict(q_stride=248), dict(dtype=2)):
        assert call(**bad) == INVALID, bad
    assert call(T=20) == UNSUPPORTED and call(D=80) == UNSUPPORTED
    for bad in (dict(end=ODD), dict(first=ODD), dict(prefix=ODD), dict(slopes=ODD), dict(space=ODD)):
        assert call(**bad) == MISALIGNED, bad
    assert call(tokens=0, B=0, max_new=0) == OK
    need = L.kv8_attention_workspace_bytes(2, 2, 1, 8192, 4, 2, 64)
    assert call(width=512, max_len=8192, space=FAKE, nbytes=need - 1) == WORKSPACE


@pytest.mark.parametrize("prefix", [None, 0, 7, 20])
@pytest.mark.parametrize("causal", [True, False])
def test_first_and_end_are_a_document_mask(causal, prefix):
    """Same document, and (causal) not after the query or below the prefix."""
    r = np.random.RandomState(1)
    n, cuts = 24, [0, 5, 6, 17, 24]
    q, k, v = r.randn(n, 1, 64), r.randn(2, 1, 16, 64), r.randn(2, 1, 16, 64)
    doc = np.searchsorted(cuts, np.arange(n), side="right") - 1
    o, _, _, _ = kv8.attention_scored(q, k, v, [[1, 0]], [n], [0, n], 16, 0.125, causal,
                                      first=[cuts[d] for d in doc], end=[cuts[d + 1] for d in doc],
                                      prefix=None if prefix is None else [prefix])
    keys, vals = (t[[1, 0]].reshape(32, 64)[:n] for t in (k, v))
    at = np.arange(n)
    seen = doc[:, None] == doc[None, :]
    if causal:
        seen &= (at[None, :] <= at[:, None]) | (at[None, :] < (prefix or 0))
    s = np.where(seen, q[:, 0] @ keys.T * 0.125, -np.inf)
    p = np.exp(s - s.max(1, keepdims=True))
    assert np.allclose(o[:, 0], p / p.sum(1, keepdims=True) @ vals)
