"""w8a8_gated_plan (host-only): what it refuses, and the kernel that each shape of
the GPU tests goes through, so that a change of the rule shows here."""

import ctypes
import os

import pytest

import bit_weight_only_gemm_amd as w4
from bit_weight_only_gemm_amd import _lib

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libw4a16.so not built", allow_module_level=True)

L = _lib.load()
NULL = ctypes.c_void_p(0)


def test_refusals_and_lengths():
    buf, n = ctypes.create_string_buffer(96), ctypes.c_int64(0)
    for bad in ((0, 64, 64), (1, 60, 64), (1, 64, 40), (1, 0, 64), (1, -8, 64)):
        assert L.w8a8_gated_plan(*bad, buf, 96, NULL) == 1, bad
    for bad in ((1, 1 << 62, 64), ((1 << 21) + 1, 64, 64), (1 << 20, 1 << 16, 64)):
        assert L.w8a8_gated_plan(*bad, buf, 96, NULL) == 2, bad
    assert L.w8a8_gated_plan(1, 64, 64, NULL, 8, NULL) == 1 and L.w8a8_gated_plan(1, 64, 64, buf, -1, NULL) == 1
    assert L.w8a8_gated_plan(1, 64, 64, NULL, 0, ctypes.byref(n)) == 0
    assert n.value == len("w8a8_gated_stream_kernel")
    assert L.w8a8_gated_plan(1, 64, 64, buf, 8, ctypes.byref(n)) == 0
    assert buf.value == b"w8a8_ga" and n.value == len("w8a8_gated_stream_kernel")


@pytest.mark.parametrize("M,F,K,quantized,kernel", [
    (1, 2048, 4096, False, "w8a8_gated_stream_kernel"), (4, 2048, 4096, False, "w8a8_gated_stream_kernel"),
    (5, 2048, 4096, True, "w8a8_gated_stream_kernel"), (16, 24, 7680, True, "w8a8_gated_stream_kernel"),
    (1, 65544, 16384, True, "w8a8_tile_kernel 64x64/1"),        # w of more than 2 GB
    (17, 72, 13328, True, "w8a8_tile_kernel 64x64/5"), (64, 1376, 4096, True, "w8a8_tile_kernel 64x64/3"),
    (571, 904, 10592, True, "w8a8_tile_kernel 128x128/3"),
    (2304, 2304, 512, True, "w8a8_wide_kernel 192x256"), (333, 13832, 272, True, "w8a8_wide_kernel 192x256"),
    (8192, 2304, 144, True, "w8a8_wide_kernel 256x256"), (8192, 27648, 5120, True, "w8a8_wide_kernel 256x256"),
])
def test_kernels(M, F, K, quantized, kernel):
    assert w4.w8a8_gated_plan(M, F, K) == (["w8a8_quantize_kernel"] if quantized else []) + [kernel]


@pytest.mark.parametrize("M,F,K", [(1, 2048, 4096), (16, 1000, 2064), (17, 72, 13328), (571, 904, 10592), (333, 13832, 272)])
def test_workspace_follows_the_plan(M, F, K):
    plan, need = w4.w8a8_gated_plan(M, F, K), w4.w8a8_gated_workspace_bytes(M, F, K)
    codes = -(-M * K // 256) * 256 + -(-M * 4 // 256) * 256
    if len(plan) == 1:
        assert need == 0
    elif "/" in plan[1] and not plan[1].endswith("/1"):
        rows, splits = int(plan[1].split("x")[1].split("/")[0]), int(plan[1].split("/")[1])
        tiles = -(-M // rows) * -(-2 * F // rows)
        assert need >= codes + 4 * tiles + splits * tiles * rows * rows * 4
    else:
        assert need >= codes
