"""Host-only checks of the 8-bit entry points (w8a8_*, kv8_*): what they refuse
before touching the GPU, calls with nothing to do, and workspace sizes."""

import ctypes
import os

import pytest

from bit_weight_only_gemm_amd import _lib

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libw4a16.so not built", allow_module_level=True)

L = _lib.load()
NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(0x10000)        # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x10008)         # misaligned
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 5


def test_quantize_refusals():
    def call(x=FAKE, M=4, K=64, stride=64, dtype=0, codes=FAKE, scales=FAKE):
        return L.w8a8_quantize(x, M, K, stride, dtype, codes, scales, NULL)
    for bad in (dict(M=0), dict(K=0), dict(K=72), dict(stride=56), dict(stride=68), dict(dtype=3),
                dict(dtype=-1), dict(x=NULL), dict(codes=NULL), dict(scales=NULL)):
        assert call(**bad) == INVALID, bad
    assert call(x=ODD) == MISALIGNED and call(codes=ODD) == MISALIGNED
    assert call(K=(1 << 17) + 16, stride=(1 << 17) + 16) == UNSUPPORTED
    assert call(M=(1 << 21) + 1) == UNSUPPORTED


def test_product_refusals():
    def call(xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, bias=NULL, out=FAKE, M=4, N=64, K=64, dtype=0,
             space=NULL, nbytes=0):
        return L.w8a8_gemm(xq, xs, wq, ws, bias, out, M, N, K, dtype, space, nbytes, NULL)
    for bad in (dict(M=0), dict(N=0), dict(N=60), dict(K=40), dict(dtype=2), dict(xq=NULL),
                dict(xs=NULL), dict(wq=NULL), dict(ws=NULL), dict(out=NULL)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(xs=ODD), dict(bias=ODD), dict(out=ODD), dict(space=ODD, nbytes=1 << 20)):
        assert call(**bad) == MISALIGNED, bad
    assert call(M=1 << 20, N=1 << 17) == UNSUPPORTED                    # 2^37 results


def test_linear_refusals_and_workspace():
    def call(x=FAKE, stride=64, wq=FAKE, ws=FAKE, bias=NULL, out=FAKE, M=64, N=64, K=64, dtype=1,
             space=FAKE, nbytes=1 << 20):
        return L.w8a8_linear(x, stride, wq, ws, bias, out, M, N, K, dtype, space, nbytes, NULL)
    for bad in (dict(stride=60), dict(stride=48), dict(dtype=2), dict(x=NULL), dict(wq=NULL)):
        assert call(**bad) == INVALID, bad
    assert call(x=ODD) == MISALIGNED and call(space=ODD) == MISALIGNED
    need = L.w8a8_workspace_bytes(64, 64, 64, 1)
    assert need == 64 * 64 + 256                                        # codes and scales
    assert call(nbytes=need - 1) == WORKSPACE and call(space=NULL, nbytes=0) == WORKSPACE
    # rows that the product quantizes for itself, and codes, need none
    assert L.w8a8_workspace_bytes(4, 4096, 4096, 1) == 0
    assert L.w8a8_workspace_bytes(4, 4096, 4112, 1) > 0
    assert L.w8a8_workspace_bytes(64, 64, 64, 0) == 0
    assert L.w8a8_workspace_bytes(0, 64, 64, 1) == -1
    assert L.w8a8_workspace_bytes(1, 64, 40, 1) == -1


def append(q=NULL, q_stride=256, q_out=NULL, q_out_stride=256, k=FAKE, k_stride=128, v=FAKE,
           v_stride=128, kc=FAKE, pages=8, T=16, table=FAKE, width=4, lens=FAKE, cu=NULL, cos=NULL,
           sin=NULL, rows=64, rope=64, tokens=2, B=2, max_new=1, H=4, Hkv=2, D=64, dtype=0):
    return L.kv8_append(q, q_stride, q_out, q_out_stride, k, k_stride, v, v_stride, kc, FAKE, FAKE,
                        FAKE, pages, T, table, width, lens, cu, cos, sin, rows, rope, 0, tokens, B,
                        max_new, H, Hkv, D, dtype, NULL)


def test_append_refusals():
    for bad in (dict(pages=0), dict(width=0), dict(tokens=-1), dict(B=-1), dict(H=3), dict(Hkv=0),
                dict(tokens=3), dict(max_new=2), dict(dtype=2), dict(k=NULL), dict(kc=NULL),
                dict(table=NULL), dict(lens=NULL), dict(k_stride=120), dict(k_stride=132),
                dict(v_stride=64), dict(q=FAKE, q_out=FAKE, q_stride=248),
                dict(q=FAKE, q_out=FAKE, q_out_stride=252), dict(cos=FAKE),
                dict(cos=FAKE, sin=FAKE, rope=24), dict(cos=FAKE, sin=FAKE, rope=80)):
        assert append(**bad) == INVALID, bad
    for bad in (dict(T=48), dict(T=8), dict(D=96), dict(D=256, k_stride=512, v_stride=512),
                dict(pages=(1 << 30) + 1), dict(width=1 << 27)):
        assert append(**bad) == UNSUPPORTED, bad
    assert append(k=ODD) == MISALIGNED and append(table=ODD) == MISALIGNED
    assert append(tokens=0, B=0, max_new=0) == OK


def test_dequant_refusals():
    def call(kc=FAKE, num=8, T=16, Hkv=2, D=64, pages=FAKE, n=1, dtype=0, ko=FAKE, vo=FAKE):
        return L.kv8_dequant(kc, FAKE, FAKE, FAKE, num, T, Hkv, D, pages, n, dtype, ko, vo, NULL)
    for bad in (dict(num=0), dict(Hkv=0), dict(n=-1), dict(dtype=2), dict(kc=NULL), dict(pages=NULL),
                dict(ko=NULL), dict(vo=NULL)):
        assert call(**bad) == INVALID, bad
    assert call(T=24) == UNSUPPORTED and call(D=32) == UNSUPPORTED
    assert call(ko=ODD) == MISALIGNED
    assert call(n=0) == OK


def attention(q=FAKE, q_stride=256, kc=FAKE, pages=8, T=16, table=FAKE, width=4, lens=FAKE, cu=NULL,
              out=FAKE, out_stride=256, lse=NULL, tokens=2, B=2, max_new=1, max_len=64, H=4, Hkv=2,
              D=64, dtype=0, space=NULL, nbytes=0):
    return L.kv8_attention(q, q_stride, kc, FAKE, FAKE, FAKE, pages, T, table, width, lens, cu, 0.125,
                           1, out, out_stride, lse, tokens, B, max_new, max_len, H, Hkv, D, dtype,
                           space, nbytes, NULL)


def test_attention_refusals_and_workspace():
    for bad in (dict(pages=0), dict(H=5), dict(tokens=3), dict(max_new=2), dict(max_len=65),
                dict(max_len=-1), dict(dtype=2), dict(q=NULL), dict(kc=NULL), dict(table=NULL),
                dict(out=NULL), dict(q_stride=248), dict(q_stride=260), dict(out_stride=64)):
        assert attention(**bad) == INVALID, bad
    assert attention(T=20) == UNSUPPORTED and attention(D=80) == UNSUPPORTED
    for bad in (dict(q=ODD), dict(out=ODD), dict(lse=ODD), dict(cu=ODD), dict(space=ODD, nbytes=16)):
        assert attention(**bad) == MISALIGNED, bad
    assert attention(tokens=0, B=0, max_new=0) == OK
    # keys split over workgroups leave partial results
    long = dict(width=512, max_len=8192, T=16)
    need = L.kv8_attention_workspace_bytes(2, 2, 1, 8192, 4, 2, 64)
    assert need > 2 * 4 * 64 * 4
    assert attention(**long) == WORKSPACE
    assert attention(**long, space=FAKE, nbytes=need - 1) == WORKSPACE
    assert L.kv8_attention_workspace_bytes(2, 2, 1, 64, 4, 2, 64) == 0
    assert L.kv8_attention_workspace_bytes(0, 0, 0, 64, 4, 2, 64) == 0
    assert L.kv8_attention_workspace_bytes(2, 2, 1, 64, 4, 3, 64) == -1
    assert L.kv8_attention_workspace_bytes(2, 2, 1, -1, 4, 2, 64) == -1
