"""The 8-bit product's check of rows: what the kernels are told of a matrix has
to lie inside its storage (host-only: the tensors here only claim to be on the
GPU, and no call is made)."""

import pytest
import torch

from bit_weight_only_gemm_amd import w8a8


class OnGpu(torch.Tensor):
    is_cuda = True


def rows(t, *args):
    return w8a8._rows(t.as_subclass(OnGpu), (torch.float16,), "x", *args)


def test_rows_inside_their_storage():
    x = torch.zeros(6, 64, dtype=torch.float16)
    assert rows(x) == (6, 64, 64)
    assert rows(x[:, 16:48], 32) == (6, 32, 64)
    assert rows(x[::2]) == (3, 64, 128)
    assert rows(x.view(2, 3, 64)) == (6, 64, 64)
    assert rows(x[0]) == (1, 64, 64)
    assert rows(x[:1].expand(1, 64)) == (1, 64, 64)


@pytest.mark.parametrize("x", [
    torch.zeros(1, 64, dtype=torch.float16).expand(5, 64),
    torch.zeros(64, dtype=torch.float16).expand(2, 3, 64),
    torch.zeros(160, dtype=torch.float16).as_strided((5, 64), (16, 1)),
    torch.zeros(64, dtype=torch.float16).unfold(0, 32, 8),
])
def test_expanded_and_overlapping_rows_are_refused(x):
    with pytest.raises(ValueError, match="elements apart"):
        rows(x)
