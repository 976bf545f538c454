"""w8a8_gated_workspace_bytes: what is enough for a batch is enough for every
smaller one (host-only)."""

import os

import pytest

from bit_weight_only_gemm_amd import _lib

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libw4a16.so not built", allow_module_level=True)

L = _lib.load()
# F, K: with and without splits of K, of one tile's width and of many, kept in registers and in LDS
SHAPES = [(520, 12304), (72, 13328), (904, 10592), (1376, 4096), (8192, 1040), (8200, 1040), (24, 4112), (8, 16),
          (8, 131072), (4096, 912), (11008, 4096), (136, 8240), (64, 1024), (8192, 7680), (272, 19680)]


@pytest.mark.parametrize("F,K", SHAPES)
def test_it_never_falls_as_the_batch_grows(F, K):
    last = 0
    for M in [*range(1, 1200), *range(1200, 9000, 61), 65536, 1 << 20]:
        need = L.w8a8_gated_workspace_bytes(M, F, K)
        assert need >= last, (M, F, K, need, last)
        last = need


@pytest.mark.parametrize("F,K", SHAPES)
def test_it_stays_next_to_the_codes(F, K):
    """Codes and scales, and at most 16 MB of sums and their counters."""
    for M in (1, 2, 16, 17, 64, 100, 512, 700, 4096, 1 << 18):
        need = L.w8a8_gated_workspace_bytes(M, F, K)
        assert need == 0 or 0 <= need - L.w8a8_workspace_bytes(max(M, 64), 2 * F, K, 1) <= (16 << 20) + 1024 or M < 64
        assert need <= M * K + 4 * M + 512 + (16 << 20) + 1024
