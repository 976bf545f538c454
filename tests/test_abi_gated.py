"""Host-only checks of w8a8_gated: refusals, workspace sizes, and pins of its
oracle."""

import ctypes
import math
import os

import numpy as np
import pytest

from bit_weight_only_gemm_amd import _lib
from oracle import w8a8

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libw4a16.so not built", allow_module_level=True)

L = _lib.load()
NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(0x10000)        # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x10008)         # misaligned
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 5


def call(x=FAKE, stride=64, wq=FAKE, ws=FAKE, bias=NULL, act=0, out=FAKE, M=64, F=64, K=64, dtype=1, space=FAKE,
         nbytes=1 << 20):
    return L.w8a8_gated(x, stride, wq, ws, bias, act, out, M, F, K, dtype, space, nbytes, NULL)


def test_refusals():
    for bad in (dict(M=0), dict(F=0), dict(F=-8), dict(F=60), dict(K=40), dict(stride=60), dict(stride=48),
                dict(dtype=2), dict(act=-1), dict(act=3), dict(x=NULL), dict(wq=NULL), dict(ws=NULL), dict(out=NULL)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(x=ODD), dict(ws=ODD), dict(bias=ODD), dict(out=ODD), dict(space=ODD)):
        assert call(**bad) == MISALIGNED, bad
    for bad in (dict(F=(1 << 23) + 8), dict(F=1 << 62), dict(M=(1 << 21) + 1), dict(M=1 << 20, F=1 << 16),
                dict(K=(1 << 17) + 16, stride=(1 << 17) + 16)):
        assert call(**bad) == UNSUPPORTED, bad


def test_out_over_x():
    at = 0x100000
    end = 2 * (63 * 80 + 64)       # bytes of x
    for out in (at, at + 16, at + end - 16, at - 2 * 64 * 64 + 16):
        assert call(x=ctypes.c_void_p(at), stride=80, out=ctypes.c_void_p(out)) == INVALID, out - at


def test_workspace():
    need = L.w8a8_gated_workspace_bytes(64, 64, 64)
    assert need == 64 * 64 + 256 == L.w8a8_workspace_bytes(64, 128, 64, 1)       # codes and scales
    assert call(nbytes=need - 1) == WORKSPACE and call(space=NULL, nbytes=0) == WORKSPACE
    # quantized inside: up to 16 rows of 16384 values in all, w below 2 GB
    for M, F, K in ((4, 2048, 4096), (16, 4096, 1024), (1, 65528, 16384)):
        assert L.w8a8_gated_workspace_bytes(M, F, K) == 0, (M, F, K)
    for M, F, K in ((17, 2048, 64), (16, 4096, 1040), (1, 8, 16400), (1, 65536, 16384)):
        assert L.w8a8_gated_workspace_bytes(M, F, K) >= M * K + 4 * M, (M, F, K)
    for bad in ((0, 64, 64), (1, 60, 64), (1, 64, 40), (1, 0, 64), (1, 1 << 62, 64)):
        assert L.w8a8_gated_workspace_bytes(*bad) == -1, bad


def test_oracle():
    xq, wq = np.array([[1, 2]]), np.array([[3, 0], [1, -1], [2, 2], [0, 1]])
    for act, f in (("silu", lambda g: g / (1 + math.exp(-g))),
                   ("gelu", lambda g: g / 2 * (1 + math.erf(g / math.sqrt(2)))),
                   ("gelu_tanh", lambda g: g / 2 * (1 + math.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))))):
        y = w8a8.gated(xq, [0.5], wq, [1.0, 1.0, 1.0, 2.0], [0.5, 0.0, 0.0, -1.0], act)[0]
        assert np.allclose(y, [[f(2.0) * 3.0, f(-0.5) * 1.0]], rtol=1e-14)
