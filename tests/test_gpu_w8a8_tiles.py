"""Large 8-bit products, in which a workgroup takes several tiles of 256 x 256
one after another: each against the same rows and channels in small calls (other
kernels), bit for bit, with scales and a bias of its own in every row and
channel, so that one tile's in another's results would show."""

import numpy as np
import pytest
import torch

import bit_weight_only_gemm_amd as w4
from gpu_util import DEV, TDT, say

pytestmark = pytest.mark.gpu


def _operands(M, N, K, dtype):
    r = np.random.RandomState(M + N + K)
    code = lambda *s: torch.from_numpy(r.randint(-127, 128, s).astype(np.int8)).to(DEV)  # noqa: E731
    scale = lambda n: torch.from_numpy(r.uniform(1e-4, 1e-2, n).astype(np.float32)).to(DEV)  # noqa: E731
    bias = torch.from_numpy(r.randn(N)).to(TDT[dtype]).to(DEV)
    return code(M, K), scale(M), code(N, K), scale(N), bias


# more than 256 and more than 512 tiles of 256 x 256 (two and three a workgroup),
# last row blocks of 44 to 256 rows and last channel blocks of 32 to 256;
# sums of one step of 128 codes (16 .. 128 of them), with a tail, and longer
WIDE = [(384, 55296, 256), (384, 55296, 128), (300, 55368, 16), (700, 60000, 128), (700, 60000, 144),
        (700, 60000, 16), (1280, 20000, 400)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", WIDE)
def test_many_tiles_of_a_workgroup(M, N, K, dtype):
    say("w8a8 many tiles", M, N, K, dtype)
    xq, xs, wq, ws, bias = _operands(M, N, K, dtype)
    y = w4.w8a8_gemm(xq, xs, wq, ws, bias, dtype=TDT[dtype])
    again = w4.w8a8_gemm(xq, xs, wq, ws, bias, dtype=TDT[dtype])
    assert torch.equal(y, again)
    rows, cols = 352, 2048
    for m in range(0, M, rows):
        for n in range(0, N, cols):
            a, b = slice(m, m + rows), slice(n, n + cols)
            part = w4.w8a8_gemm(xq[a].clone(), xs[a].clone(), wq[b].clone(), ws[b].clone(),
                                bias[b].clone(), dtype=TDT[dtype])
            assert torch.equal(y[a, b], part), (m, n)


@pytest.mark.parametrize("M,N,K", [(320, 8200, 144), (700, 4872, 400)])
def test_tiles_of_128_in_fp16(M, N, K):
    say("w8a8 tiles of 128", M, N, K)
    xq, xs, wq, ws, bias = _operands(M, N, K, "f16")
    y = w4.w8a8_gemm(xq, xs, wq, ws, bias, dtype=torch.float16)
    for m in range(0, M, 64):
        part = w4.w8a8_gemm(xq[m:m + 64].clone(), xs[m:m + 64].clone(), wq, ws, bias, dtype=torch.float16)
        assert torch.equal(y[m:m + 64], part), m


def test_linear_of_many_tiles():
    M, N, K = 384, 55296, 144
    _, _, wq, ws, bias = _operands(M, N, K, "bf16")
    x = torch.from_numpy(np.random.RandomState(1).randn(M, K)).bfloat16().to(DEV)
    y = w4.w8a8_linear(x, wq, ws, bias)
    assert torch.equal(y, w4.w8a8_gemm(*w4.w8a8_quantize(x), wq, ws, bias))
    for n in range(0, N, 2048):
        b = slice(n, n + 2048)
        assert torch.equal(y[:, b], w4.w8a8_linear(x, wq[b].clone(), ws[b].clone(), bias[b].clone())), n


def test_expanded_and_overlapping_rows_are_refused():
    wq, ws = w4.w8a8_quantize(torch.ones(16, 64, device=DEV))
    row = torch.ones(1, 64, dtype=torch.float16, device=DEV)
    over = torch.ones(160, dtype=torch.float16, device=DEV).as_strided((5, 64), (16, 1))
    for x in (row.expand(5, 64), row[0].expand(2, 3, 64), over):
        with pytest.raises(ValueError, match="elements apart"):
            w4.w8a8_quantize(x)
        with pytest.raises(ValueError, match="elements apart"):
            w4.w8a8_linear(x, wq, ws)
    assert torch.equal(w4.w8a8_linear(row.expand(1, 64), wq, ws), w4.w8a8_linear(row, wq, ws))
