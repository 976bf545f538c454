"""8-bit integer products on the GPU against exact integer sums and 64-bit
scales: odd rows, tails of K and N, biases, strided and scaled inputs, and
rows that quantization cannot hold."""

import numpy as np
import pytest
import torch

import bit_weight_only_gemm_amd as w4
from oracle import w8a8
from gpu_util import DEV, TDT, say

pytestmark = pytest.mark.gpu


def _normal(seed, *shape):
    return torch.from_numpy(np.random.RandomState(seed).randn(*shape)).float()


def _codes(seed, *shape):
    return torch.from_numpy(np.random.RandomState(seed).randint(-127, 128, shape).astype(np.int8))


def _check_product(y, xq, xs, wq, ws, bias, dtype):
    ref, mag = w8a8.product(xq.cpu().numpy(), xs.cpu().numpy(), wq.cpu().numpy(), ws.cpu().numpy(),
                            None if bias is None else bias.float().cpu().numpy())
    err = np.abs(y.double().cpu().numpy() - ref)
    bound = w8a8.product_bound(ref, mag, dtype)
    assert np.all(err <= bound), (np.max(err / bound), np.argwhere(err > bound)[:4])


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (17, 2048), (5, 5120), (2, 16400), (1, 33040)])
def test_quantize_is_the_fp32_formula(M, K, dtype):
    x = _normal(M + K, M, K) * torch.logspace(-4, 3, M)[:, None]
    if M > 2:
        x[1] = 0.0
    x = x.to(TDT.get(dtype, torch.float32)).to(DEV)
    say("quantize", M, K, dtype)
    c, s = w4.w8a8_quantize(x)
    xf = x.float().cpu().numpy()
    want = np.abs(xf).max(1) * np.float32(1 / 127)
    want[want == 0] = 1
    assert np.array_equal(s.cpu().numpy(), want)
    codes = np.clip(np.rint(xf / want[:, None]), -127, 127)
    assert np.array_equal(c.cpu().numpy(), codes.astype(np.int8))
    # and the 64-bit definition: at most half a step off, and 2^-16 for fp32
    c64, s64 = w8a8.quantize(xf)
    assert np.all(np.abs(xf / s64[:, None] - c.cpu().numpy()) <= 0.5 + 2.0 ** -15)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantize_strided_tiny_and_nonfinite_rows(dtype):
    x = _normal(1, 6, 96).to(TDT[dtype]).to(DEV)
    x[1] *= 1e-6 if dtype == "f16" else 1e-38
    x[3, 7] = float("inf")
    x[4, 95] = float("nan")
    part = x[:, 16:80]
    c, s = w4.w8a8_quantize(part)
    cc, ss = w4.w8a8_quantize(part.contiguous())
    assert torch.equal(c, cc) and torch.equal(s, ss)
    assert not torch.isnan(s).any()                                      # columns 7 and 95 lie outside
    c, s = w4.w8a8_quantize(x)
    assert torch.isnan(s).cpu().tolist() == [False, False, False, True, True, False]
    f = x[1].float().cpu().numpy()
    step = np.abs(f).max() * np.float32(1 / 127)
    step = step if step else np.float32(1)
    assert np.array_equal(c[1].cpu().numpy(), np.clip(np.rint(f / step), -127, 127).astype(np.int8))


SHAPES = [(1, 8, 16), (1, 4096, 4096), (2, 24, 48), (4, 4096, 1040), (7, 264, 4112), (16, 1000, 2064),
          (17, 72, 64), (31, 4096, 512), (33, 136, 80), (64, 512, 4096), (100, 640, 1104),
          (128, 4104, 256), (129, 264, 5120), (255, 1032, 1008), (256, 256, 16), (257, 520, 8192),
          (333, 1792, 1280), (512, 2560, 512), (1000, 1016, 688), (2049, 776, 320)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, dtype):
    say("w8a8_gemm", M, N, K, dtype)
    xq, wq = _codes(M, M, K).to(DEV), _codes(N + 1, N, K).to(DEV)
    xs, ws = (_normal(2, M).abs() * 1e-3 + 1e-4).to(DEV), (_normal(3, N).abs() * 1e-2).to(DEV)
    bias = _normal(4, N).to(TDT[dtype]).to(DEV) if (M + N) % 16 else None
    y = w4.w8a8_gemm(xq, xs, wq, ws, bias, dtype=TDT[dtype])
    _check_product(y, xq, xs, wq, ws, bias, dtype)
    again = w4.w8a8_gemm(xq, xs, wq, ws, bias, dtype=TDT[dtype])
    assert torch.equal(y, again)
    plain = w4.w8a8_gemm(xq, xs, wq, ws, bias, dtype=TDT[dtype], use_workspace=False)
    assert torch.equal(y, plain)


@pytest.mark.parametrize("M,N,K", [(16, 12296, 160), (48, 4104, 272), (320, 8200, 144), (700, 4872, 400),
                                   (1100, 16392, 112), (2100, 5128, 208)])
def test_a_result_does_not_depend_on_the_kernel(M, N, K):
    """Each call against the same rows and channels in small calls, bit for bit (copies: scales are read 16 bytes at a time)."""
    say("w8a8 whole and parts", M, N, K)
    xq, wq = _codes(M, M, K).to(DEV), _codes(N + 1, N, K).to(DEV)
    xs, ws = (_normal(2, M).abs() * 1e-3 + 1e-4).to(DEV), (_normal(3, N).abs() * 1e-2).to(DEV)
    bias = _normal(4, N).bfloat16().to(DEV)
    y = w4.w8a8_gemm(xq, xs, wq, ws, bias)
    for rows in (slice(0, 9), slice(M // 2, M // 2 + 40), slice(M - 8, M)):
        for cols in (slice(0, 64), slice(N - 2056, N)):
            part = w4.w8a8_gemm(xq[rows].clone(), xs[rows].clone(), wq[cols].clone(),
                                ws[cols].clone(), bias[cols].clone())
            assert torch.equal(y[rows, cols], part), (rows, cols)


def test_quantize_many_rows_as_each_alone():
    for M, K in ((512, 2064), (513, 2064), (1200, 16400)):
        say("quantize many rows", M, K)
        x = (_normal(M, M, K) * torch.logspace(-3, 3, M)[:, None]).bfloat16().to(DEV)
        c, s = w4.w8a8_quantize(x)
        for m in (0, 1, M // 2, M - 1):
            cm, sm = w4.w8a8_quantize(x[m:m + 1])
            assert torch.equal(c[m:m + 1], cm) and torch.equal(s[m:m + 1], sm)


@pytest.mark.parametrize("M,N,K", [(1, 40, 131072), (70, 48, 131072), (300, 264, 131072)])
def test_the_longest_sum_is_exact(M, N, K):
    say("w8a8 longest", M, N, K)
    xq = torch.full((M, K), 127, dtype=torch.int8, device=DEV)
    wq = torch.full((N, K), 127, dtype=torch.int8, device=DEV)
    wq[1] = -127
    one = torch.ones(max(M, N), device=DEV) * 2.0 ** -20
    y = w4.w8a8_gemm(xq, one[:M].contiguous(), wq, one[:N].contiguous() * 2.0 ** 4)
    want = torch.tensor(127 * 127 * 131072 * 2.0 ** -36).bfloat16().item()
    assert torch.all(y[:, 0] == want) and torch.all(y[:, 1] == -want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_is_quantize_and_product(M, N, K, dtype):
    say("w8a8_linear", M, N, K, dtype)
    x = _normal(M + K, M, K).to(TDT[dtype]).to(DEV)
    x[:, K // 3] *= 20
    wq, ws = w4.w8a8_quantize(_normal(N, N, K).to(DEV) * 0.02)
    bias = _normal(4, N).to(TDT[dtype]).to(DEV) if N % 16 else None
    y = w4.w8a8_linear(x, wq, ws, bias)
    xq, xs = w4.w8a8_quantize(x)
    assert torch.equal(y, w4.w8a8_gemm(xq, xs, wq, ws, bias, dtype=TDT[dtype]))
    _check_product(y, xq, xs, wq, ws, bias, dtype)


@pytest.mark.parametrize("M", [1, 3, 40])
def test_linear_rows_of_a_wider_buffer_and_bad_rows(M):
    K, N = 512, 96
    buf = _normal(9, M, 1024).bfloat16().to(DEV)
    wq, ws = w4.w8a8_quantize(_normal(8, N, K).to(DEV))
    y = w4.w8a8_linear(buf[:, 512:], wq, ws)
    assert torch.equal(y, w4.w8a8_linear(buf[:, 512:].contiguous(), wq, ws))
    x = buf[:, :512].contiguous()
    good = w4.w8a8_linear(x, wq, ws)
    x[M - 1, 5] = float("inf")
    y = w4.w8a8_linear(x, wq, ws)
    assert torch.isnan(y[M - 1]).all() and torch.equal(y[:M - 1], good[:M - 1])


def test_leading_dimensions_and_streams():
    x = _normal(5, 2, 3, 256).half().to(DEV)
    wq, ws = w4.w8a8_quantize(_normal(6, 64, 256).half().to(DEV))
    y = w4.w8a8_linear(x, wq, ws)
    assert y.shape == (2, 3, 64)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    z = w4.w8a8_linear(x, wq, ws, stream=st)
    st.synchronize()
    assert torch.equal(y, z)


def test_capture_in_a_graph():
    x = _normal(5, 24, 512).half().to(DEV)
    wq, ws = w4.w8a8_quantize(_normal(6, 4096, 512).half().to(DEV))
    out = torch.empty(24, 4096, dtype=torch.float16, device=DEV)
    ws_buf = w4.workspace(w4.w8a8_workspace_bytes(24, 4096, 512), DEV)
    w4.w8a8_linear(x, wq, ws, out=out, workspace=ws_buf)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.w8a8_linear(x, wq, ws, out=out, workspace=ws_buf)
    for i in range(4):
        x.copy_(_normal(50 + i, 24, 512).half())
        want = w4.w8a8_linear(x, wq, ws)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals():
    x = torch.zeros(4, 64, dtype=torch.float16, device=DEV)
    wq, ws = w4.w8a8_quantize(torch.ones(16, 64, device=DEV))
    with pytest.raises(TypeError):
        w4.w8a8_linear(x.float(), wq, ws)
    with pytest.raises(TypeError):
        w4.w8a8_linear(x, wq, ws.half())
    with pytest.raises(TypeError):
        w4.w8a8_linear(x, wq, ws, bias=torch.zeros(16, device=DEV))
    with pytest.raises(TypeError):
        w4.w8a8_quantize(x.cpu())
    with pytest.raises(ValueError):
        w4.w8a8_linear(x[:, :48], wq, ws)
    with pytest.raises(ValueError):
        w4.w8a8_quantize(x.t())
    with pytest.raises(ValueError):
        w4.w8a8_gemm(wq, ws[:8], wq, ws)
    with pytest.raises(w4.W4A16Error, match="status 1"):
        w4.w8a8_quantize(torch.zeros(4, 24, device=DEV))
    with pytest.raises(w4.W4A16Error, match="status 3"):
        w4.w8a8_quantize(torch.zeros(4 * 64 + 4, dtype=torch.float16, device=DEV)[4:].view(4, 64))
    big = torch.zeros(64, 512, dtype=torch.float16, device=DEV)
    w2, s2 = w4.w8a8_quantize(torch.ones(16, 512, device=DEV))
    with pytest.raises(w4.W4A16Error, match="status 5"):
        w4.w8a8_linear(big, w2, s2, workspace=torch.zeros(16, dtype=torch.int32, device=DEV))
