"""Host-only checks of the largest grids of the 8-bit cache's calls: what would
pass 2^32 work-items is refused before a launch."""

import ctypes
import os

import pytest
import torch

from bit_weight_only_gemm_amd import _lib

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libw4a16.so not built", allow_module_level=True)
if torch.cuda.is_available():
    pytest.skip("the addresses are not real", allow_module_level=True)

L = _lib.load()
NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(0x10000)        # 16-byte aligned, never dereferenced
UNSUPPORTED = 2


def append(tokens, B, Hkv, T=16, D=64, q=NULL, max_new=None):
    return L.kv8_append(q, Hkv * D, q, Hkv * D, FAKE, Hkv * D, FAKE, Hkv * D, FAKE, FAKE, FAKE, FAKE, 8,
                        T, FAKE, 1 << 20, FAKE, FAKE, NULL, NULL, 0, 0, 0, tokens, B,
                        tokens if max_new is None else max_new, Hkv, Hkv, D, 0, NULL)


def test_append():
    assert append(1 << 24, 1, 8) == UNSUPPORTED                   # (2^20 + 2) pages of 8 heads, 2 each
    assert append(1 << 20, 1 << 20, 16, max_new=8) == UNSUPPORTED  # 2 pages a sequence
    assert append(1 << 24, 1, 1, T=128, q=FAKE) == UNSUPPORTED    # 2^24 rows of queries
    # within the limits: nothing but the missing GPU fails
    assert append((1 << 24) - 2000000, 1, 1, T=128, q=FAKE) not in (0, 1, UNSUPPORTED)
    # 65536 new tokens in 256 sequences, no bound of one sequence's given
    assert append(65536, 256, 8) not in (0, 1, UNSUPPORTED)


def test_dequant():
    def call(n):
        return L.kv8_dequant(FAKE, FAKE, FAKE, FAKE, 8, 128, 8, 128, FAKE, n, 0, FAKE, FAKE, NULL)
    assert call(1 << 20) == UNSUPPORTED
    assert call(1 << 17) not in (0, 1, UNSUPPORTED)


def test_attention():
    def call(tokens, H, D):
        return L.kv8_attention(FAKE, H * D, FAKE, FAKE, FAKE, FAKE, 8, 64, FAKE, 1 << 20, FAKE, FAKE, 0.1,
                               1, FAKE, H * D, NULL, tokens, 1, tokens, 1 << 20, H, H, D, 0, FAKE,
                               1 << 60, NULL)
    assert call(1 << 24, 128, 128) == UNSUPPORTED
    assert call(1 << 24, 128, 64) == UNSUPPORTED
    assert call(1 << 23, 128, 128) not in (0, 1, UNSUPPORTED)
