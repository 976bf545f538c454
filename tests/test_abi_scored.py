"""Host-only checks of kv8_attention_scored, and pins of its oracle."""

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


def call(q=FAKE, q_stride=256, kc=FAKE, pages=8, T=16, table=FAKE, width=4, lens=FAKE, cu=NULL, cap=0.0, slopes=NULL,
         first=NULL, prefix=NULL, out=FAKE, out_stride=256, lse=NULL, tokens=2, B=2, max_new=1, max_len=64, H=4, Hkv=2,
         D=64, dtype=0, space=NULL, nbytes=0):
    return L.kv8_attention_scored(q, q_stride, kc, FAKE, FAKE, FAKE, pages, T, table, width, lens, cu, 0.125, 1, cap,
                                  slopes, first, prefix, out, out_stride, lse, tokens, B, max_new, max_len, H, Hkv, D,
                                  dtype, space, nbytes, NULL)


def test_refusals_and_workspace():
    for bad in (dict(cap=-1.0), dict(cap=1e-4), dict(cap=2e30), dict(cap=float("nan")), dict(pages=0), dict(H=5),
                dict(tokens=3), dict(max_len=65), dict(dtype=2), dict(q=NULL), dict(out=NULL), dict(q_stride=248),
                dict(out_stride=64)):
        assert call(**bad) == INVALID, bad
    assert call(T=20) == UNSUPPORTED and call(D=80) == UNSUPPORTED
    for bad in (dict(slopes=ODD), dict(first=ODD), dict(prefix=ODD), dict(lse=ODD), dict(cu=ODD), dict(out=ODD)):
        assert call(**bad) == MISALIGNED, bad
    assert call(tokens=0, B=0, max_new=0, cap=30.0) == OK
    need = L.kv8_attention_workspace_bytes(2, 2, 1, 8192, 4, 2, 64)
    assert call(width=512, max_len=8192, cap=30.0, space=FAKE, nbytes=need - 1) == WORKSPACE


def test_oracle():
    """Of two keys by hand, and plain attention where nothing is set."""
    r = np.random.RandomState(0)
    q, k, v = r.randn(3, 2, 64), r.randn(2, 1, 16, 64), r.randn(2, 1, 16, 64)
    table, lens, cu = [[1, 0]], [20], [0, 3]
    a = kv8.attention(q, k, v, table, lens, cu, 16, 0.125, True)
    b = kv8.attention_scored(q, k, v, table, lens, cu, 16, 0.125, True)
    assert np.allclose(a[0], b[0], rtol=1e-12) and np.allclose(a[2], b[1], rtol=1e-12)
    # token 1 (position 18) sees 17 and 18; token 2 nothing; token 0 (17) by its prefix 16 to 18
    o, lse, _, _ = kv8.attention_scored(q, k, v, table, lens, cu, 16, 0.125, True, 2.0, [0.5, 0.25], [16, 17, 20], [19])
    assert not o[2].any() and np.isneginf(lse[2]).all()
    s = 2.0 * np.tanh(np.array([k[0, 0, 1] @ q[1, 1], k[0, 0, 2] @ q[1, 1]]) * 0.125 / 2.0) - 0.25 * np.array([1, 0])
    w = np.exp(s)
    assert np.allclose(o[1, 1], (w[0] * v[0, 0, 1] + w[1] * v[0, 0, 2]) / w.sum())
    s = 2.0 * np.tanh(k[0, 0, :3] @ q[0, 0] * 0.125 / 2.0) - 0.5 * np.array([1, 0, 1])
    assert np.allclose(lse[0, 0], np.log(np.exp(s).sum()))
