"""The gated feed-forward product on the GPU against 64 bits: every kernel it
may go through, tails, biases, strided rows, gates far out, and rows that
quantization cannot hold."""

import numpy as np
import pytest
import torch

import bit_weight_only_gemm_amd as w4
from gpu_util import DEV, TDT, say
from oracle import w8a8

pytestmark = pytest.mark.gpu
ACTS = ("silu", "gelu", "gelu_tanh")


def inputs(seed, M, F, K, dtype, bias=True, scale=1.0):
    r = np.random.RandomState(seed)
    x = torch.from_numpy(r.randn(M, K).astype(np.float32)).to(TDT[dtype]).to(DEV)
    wq = torch.from_numpy(r.randint(-127, 128, (2 * F, K)).astype(np.int8)).to(DEV)
    # results of unit size, some channels larger
    ws = torch.from_numpy((scale * (0.5 + 2 * r.rand(2 * F)) / 73 / np.sqrt(K)).astype(np.float32)).to(DEV)
    b = torch.from_numpy(r.randn(2 * F).astype(np.float32)).to(TDT[dtype]).to(DEV) if bias else None
    return x, wq, ws, b


def check(y, x, wq, ws, b, act, dtype):
    xq, xs = (t.cpu().numpy() for t in w4.w8a8_quantize(x))
    parts = w8a8.gated(xq, xs, wq.cpu().numpy(), ws.cpu().numpy(), None if b is None else b.float().cpu().numpy(), act)
    err = np.abs(y.double().cpu().numpy() - parts[0])
    bound = w8a8.gated_bound(*parts, act, dtype)
    assert np.all(err <= bound), (np.max(err / bound), np.argwhere(err > bound)[:4])


SHAPES = [  # M, F, K
    (1, 8, 16), (1, 2048, 4096), (2, 24, 48), (4, 1000, 1040), (1, 8200, 512), (2, 16392, 256),  # w streamed
    (3, 40, 4112), (7, 264, 4112), (16, 1000, 2064), (5, 5504, 5136), (16, 8192, 640), (13, 520, 16),
    (1, 264, 122880), (16, 24, 7680),                                                            # all of LDS
    (17, 72, 5136), (31, 2048, 512), (33, 136, 80), (64, 512, 4096), (16, 264, 7696), (1, 40, 122896),
    (100, 640, 1104), (129, 264, 5120), (255, 520, 1008),                                        # 64 x 64 tiles
    (128, 2752, 272), (250, 11008, 80),
    (333, 1792, 1280), (1000, 1016, 688), (512, 2568, 512),                                      # 128 x 128
    (2049, 2312, 320), (2304, 2304, 16), (8192, 2304, 144),                                      # 256 x 256
    (333, 13832, 272), (1150, 4616, 144), (380, 27648, 64),                                      # 192 x 256
    (17, 72, 13328), (14, 272, 19680), (65, 24, 4112), (200, 136, 8240), (300, 520, 12304),      # K split
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_every_shape(i, dtype):
    M, F, K = SHAPES[i]
    act = ACTS[(i + (dtype == "bf16")) % 3]
    say("gated", M, F, K, act, dtype)
    x, wq, ws, b = inputs(i, M, F, K, dtype, bias=i % 2 == 0)
    check(w4.w8a8_gated(x, wq, ws, b, act), x, wq, ws, b, act, dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("scale", [1e-6, 12.0, 1e3])
def test_small_and_far_gates(act, scale):
    """Gates from next to 0 to where the exponential leaves fp32."""
    for M, dtype in ((3, "f16"), (40, "bf16"), (200, "bf16")):
        x, wq, ws, b = inputs(50 + M, M, 512, 256, dtype, bias=False, scale=scale)
        if dtype == "f16" and scale > 100:
            ws[512:] *= 1e-3                    # fp16 ends at 65504
        check(w4.w8a8_gated(x, wq, ws, act=act), x, wq, ws, None, act, dtype)


@pytest.mark.parametrize("act", ACTS)
def test_a_row_does_not_depend_on_the_others(act):
    """The kernels form a result by the same operations: the same bits."""
    M, F, K = 2304, 2304, 512
    x, wq, ws, b = inputs(60, M, F, K, "bf16")
    y = w4.w8a8_gated(x, wq, ws, b, act)
    assert torch.equal(y, w4.w8a8_gated(x, wq, ws, b, act))
    for rows in (slice(0, 1), slice(5, 9), slice(20, 36), slice(100, 160), slice(300, 812)):
        assert torch.equal(y[rows], w4.w8a8_gated(x[rows].contiguous(), wq, ws, b, act)), rows


def test_agrees_with_the_linear_product():
    """Its two halves are w8a8_linear's results before their rounding."""
    x, wq, ws, b = inputs(61, 48, 256, 320, "f16")
    v = w4.w8a8_linear(x, wq, ws, b).double()
    g, u = v[:, :256], v[:, 256:]
    y = w4.w8a8_gated(x, wq, ws, b, "silu").double()
    want = g * torch.sigmoid(g) * u
    # three roundings of 2^-11: of g (slope at most 1.13), u and y
    assert torch.all((y - want).abs() <= 2.0 ** -11 * 1.01 * (1.13 * (g * u).abs() + 2 * want.abs()) + 2.0 ** -23)


@pytest.mark.parametrize("M", [1, 4, 5, 70])
def test_strided_rows_and_given_outputs(M):
    x, wq, ws, b = inputs(62, M, 128, 192, "bf16")
    wide = torch.zeros(M, 264, dtype=torch.bfloat16, device=DEV)
    wide[:, 40:232] = x
    out = torch.empty(M, 128, dtype=torch.bfloat16, device=DEV)
    space = torch.full((max(w4.w8a8_gated_workspace_bytes(M, 128, 192), 16),), 255, dtype=torch.uint8, device=DEV)
    y = w4.w8a8_gated(wide[:, 40:232], wq, ws, b, out=out, workspace=space)
    assert y is out and torch.equal(y, w4.w8a8_gated(x, wq, ws, b))
    assert torch.equal(w4.w8a8_gated(x.view(1, M, 192), wq, ws, b), y.view(1, M, 128))


@pytest.mark.parametrize("act", ACTS)
def test_rows_of_zeros_infinities_and_nan(act):
    for M in (4, 40):
        x, wq, ws, b = inputs(63, M, 64, 128, "f16")
        x[0] = 0
        x[1, 5] = float("inf")
        x[2, 6] = float("nan")
        y = w4.w8a8_gated(x, wq, ws, b, act)
        assert torch.isnan(y[1:3]).all() and not torch.isnan(y[[0, *range(3, M)]]).any()
        check(y[[0, *range(3, M)]], x[[0, *range(3, M)]], wq, ws, b, act, "f16")


def test_no_bytes_beyond_the_results():
    for M, F, K in ((1, 24, 48), (5, 24, 48), (70, 40, 80), (333, 1032, 272), (2049, 2312, 64)):
        x, wq, ws, b = inputs(64, M, F, K, "bf16")
        room = torch.full((M * F + 4096,), 7.0, dtype=torch.bfloat16, device=DEV)
        w4.w8a8_gated(x, wq, ws, b, out=room[2048:2048 + M * F].view(M, F))
        assert (room[:2048] == 7).all() and (room[2048 + M * F:] == 7).all(), (M, F, K)


@pytest.mark.parametrize("M", [2, 50])
def test_captured_in_a_graph(M):
    x, wq, ws, b = inputs(65, M, 256, 512, "f16")
    out = torch.empty(M, 256, dtype=torch.float16, device=DEV)
    space = w4.workspace(w4.w8a8_gated_workspace_bytes(M, 256, 512), DEV)
    w4.w8a8_gated(x, wq, ws, b, out=out, workspace=space)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.w8a8_gated(x, wq, ws, b, out=out, workspace=space)
    for i in range(4):
        x.copy_(torch.randn(M, 512, generator=torch.Generator().manual_seed(i)))
        want = w4.w8a8_gated(x, wq, ws, b)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_on_another_stream():
    x, wq, ws, b = inputs(66, 50, 256, 512, "f16")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y = w4.w8a8_gated(x, wq, ws, b, stream=st)
    st.synchronize()
    assert torch.equal(y, w4.w8a8_gated(x, wq, ws, b))


def test_refusals():
    x, wq, ws, b = inputs(67, 5, 24, 64, "f16")
    with pytest.raises(ValueError, match="act"):
        w4.w8a8_gated(x, wq, ws, act="relu")
    with pytest.raises(ValueError, match="2 F"):
        w4.w8a8_gated(x, wq[:47], ws[:47])
    with pytest.raises(w4.W4A16Error, match="status 1"):
        w4.w8a8_gated(x, wq[:40], ws[:40])                     # F = 20
    with pytest.raises(TypeError):
        w4.w8a8_gated(x.float(), wq, ws)
    with pytest.raises(TypeError):
        w4.w8a8_gated(x, wq, ws, b.bfloat16())
    with pytest.raises(ValueError):
        w4.w8a8_gated(x, wq, ws[:40])
    with pytest.raises(ValueError):
        w4.w8a8_gated(x[:, :48], wq, ws)
    with pytest.raises(ValueError):
        w4.w8a8_gated(x, wq, ws, out=torch.empty(5, 48, dtype=torch.float16, device=DEV))
    with pytest.raises(TypeError):
        w4.w8a8_gated(x.cpu(), wq, ws)
    with pytest.raises(w4.W4A16Error, match="status 5"):
        w4.w8a8_gated(x.repeat(4, 1), wq, ws, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_weights_at_two_gigabytes():
    """The last rows of w below and beyond what one buffer holds, bit for bit as alone."""
    K = 16384
    w = torch.empty(2 * 65536, K, dtype=torch.int8, device=DEV)
    for i in range(0, len(w), 8192):
        w[i:i + 8192] = torch.randint(-127, 128, (8192, K), device=DEV, dtype=torch.int8)
    ws = torch.rand(2 * 65536, device=DEV) * 1e-4
    x = inputs(68, 1, 8, K, "bf16")[0]
    for F in (65528, 65536):
        say("gated, rows of w", 2 * F)
        y = w4.w8a8_gated(x, w[:2 * F], ws[:2 * F])
        for at in (0, F // 2 + 4, F - 8):
            rows = [*range(at, at + 8), *range(F + at, F + at + 8)]
            alone = w4.w8a8_gated(x, w[rows].contiguous(), ws[rows].contiguous())
            assert torch.equal(y[:, at:at + 8], alone), (F, at)


def test_two_streams_at_once():
    """Each stream has a workspace of its own."""
    cases = [inputs(70 + i, 100, 512, 1024, "f16") for i in range(2)]
    want = [w4.w8a8_gated(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            got[i].append(w4.w8a8_gated(*cases[i], stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])


@pytest.mark.parametrize("M,F,K", [(17, 72, 13328), (571, 904, 10592), (64, 1376, 4096)])
def test_splits_of_k(M, F, K):
    """Sums over split K are whole whatever the workspace held, on every call and
    every replay, and the same bits as without a split (rows alone go through the
    kernel for few tokens where they fit there)."""
    x, wq, ws, b = inputs(80, M, F, K, "bf16")
    need = w4.w8a8_gated_workspace_bytes(M, F, K)
    assert need > w4.w8a8_workspace_bytes(M, 2 * F, K)
    space = torch.full((need + 4096,), 255, dtype=torch.uint8, device=DEV)
    y = w4.w8a8_gated(x, wq, ws, b, workspace=space[:need])
    assert (space[need:] == 255).all()
    for rows in (slice(0, 4), slice(M - 7, M)):
        assert torch.equal(y[rows], w4.w8a8_gated(x[rows].contiguous(), wq, ws, b))
    for _ in range(10):
        space.random_(0, 256)
        assert torch.equal(y, w4.w8a8_gated(x, wq, ws, b, workspace=space[:need]))
    g, out = torch.cuda.CUDAGraph(), torch.empty_like(y)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        w4.w8a8_gated(x, wq, ws, b, out=out, workspace=space[:need])
    for i in range(4):
        x.copy_(torch.randn(M, K, generator=torch.Generator().manual_seed(i)))
        want = w4.w8a8_gated(x, wq, ws, b)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
