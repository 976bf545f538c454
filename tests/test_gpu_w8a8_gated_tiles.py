"""Every kernel of the gated product, by the plan and not by a guess: odd numbers of
tokens, channels that end inside a tile, several steps of K of which the last is
partial, each activation and type; and the same bits from each."""

import numpy as np
import pytest
import torch

import bit_weight_only_gemm_amd as w4
from gpu_util import DEV, TDT, say
from oracle import w8a8

pytestmark = pytest.mark.gpu
ACTS = ("silu", "gelu", "gelu_tanh")
FORMS = {  # kernel: M, F, K
    "w8a8_tile_kernel 64x64/1": (131, 2056, 656),
    "w8a8_tile_kernel 64x64/3": (77, 264, 5136),
    "w8a8_tile_kernel 128x128/1": (999, 2056, 656),
    "w8a8_tile_kernel 128x128/3": (571, 904, 10592),
    "w8a8_wide_kernel 192x256": (333, 13832, 656),
    "w8a8_wide_kernel 256x256": (4001, 2040, 656),
    "several tiles a workgroup: w8a8_wide_kernel 256x256": (7001, 2056, 656),
}


def inputs(seed, M, F, K, dtype, bias=True):
    r = np.random.RandomState(seed)
    x = torch.from_numpy(r.randn(M, K).astype(np.float32)).to(TDT[dtype]).to(DEV)
    wq = torch.from_numpy(r.randint(-127, 128, (2 * F, K)).astype(np.int8)).to(DEV)
    ws = torch.from_numpy(((0.5 + 2 * r.rand(2 * F)) / 73 / np.sqrt(K)).astype(np.float32)).to(DEV)
    b = torch.from_numpy(r.randn(2 * F).astype(np.float32)).to(TDT[dtype]).to(DEV) if bias else None
    return x, wq, ws, b


def check(y, x, wq, ws, b, act, dtype):
    xq, xs = (t.cpu().numpy() for t in w4.w8a8_quantize(x))
    parts = w8a8.gated(xq, xs, wq.cpu().numpy(), ws.cpu().numpy(), None if b is None else b.float().cpu().numpy(), act)
    err = np.abs(y.double().cpu().numpy() - parts[0])
    bound = w8a8.gated_bound(*parts, act, dtype)
    assert np.all(err <= bound), (np.max(err / bound), np.argwhere(err > bound)[:4])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("form", FORMS)
def test_every_kernel(form, act, dtype):
    M, F, K = FORMS[form]
    assert w4.w8a8_gated_plan(M, F, K)[-1] == form.split(": ")[-1]
    assert M % 2 and K // 128 >= 5 and K % 128
    say("gated", form, M, F, K, act, dtype)
    x, wq, ws, b = inputs(M + len(act), M, F, K, dtype, bias=(dtype == "f16") != (act == "gelu"))
    y = w4.w8a8_gated(x, wq, ws, b, act)
    check(y, x, wq, ws, b, act, dtype)
    assert torch.equal(y, w4.w8a8_gated(x, wq, ws, b, act))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,F", [(4001, 2040), (7001, 2056)])
def test_rows_of_the_largest_tiles_alone(M, F, act, dtype):
    """Rows that went through 256 x 256 tiles have the bits that smaller tiles and the
    stream give them."""
    K = 656
    x, wq, ws, b = inputs(60 + M, M, F, K, dtype)
    assert w4.w8a8_gated_plan(M, F, K)[-1] == "w8a8_wide_kernel 256x256"
    y = w4.w8a8_gated(x, wq, ws, b, act)
    seen = set()
    for n, at in ((1, 0), (5, M - 5), (40, 1234), (700, M - 700), (2304, 100)):
        say("rows", n, at, w4.w8a8_gated_plan(n, F, K))
        seen.add(w4.w8a8_gated_plan(n, F, K)[-1].split("/")[0])
        assert torch.equal(y[at:at + n], w4.w8a8_gated(x[at:at + n].contiguous(), wq, ws, b, act)), (n, at)
    assert seen == {"w8a8_gated_stream_kernel", "w8a8_tile_kernel 64x64", "w8a8_tile_kernel 128x128", "w8a8_wide_kernel 192x256"}
