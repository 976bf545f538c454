"""Captured calls without a workspace of their own: refused where none is kept for
the stream, and the capture goes on; right on every replay where one is."""

import pytest
import torch

import bit_weight_only_gemm_amd as w4
from gpu_util import DEV

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def test_refused_without_ending_the_capture():
    refs, table, lens = w4.kv8_refs(8, DEV), torch.full((2, 3), -1, dtype=torch.int32, device=DEV), ints([0, 0])
    added, status, space = ints([5, 1]), ints([9]), w4.workspace(w4.kv8_pages_workspace_bytes(8, 2), DEV)
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    w4._WS.pop((refs.device, st.cuda_stream), None)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        with pytest.raises(w4.W4A16Error, match="before it is captured"):
            w4.kv8_reserve(refs, table, lens, added, 16, status=status)
        w4.kv8_reserve(refs, table, lens, added, 16, status=status, workspace=space)
    assert lens.tolist() == [0, 0]
    for i in range(1, 4):
        g.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [5 * i, i] and status.tolist() == [0] and table[:, 0].tolist() == [0, 1]


def test_one_kept_for_the_stream_is_used():
    refs, table, lens = w4.kv8_refs(8, DEV), torch.full((2, 3), -1, dtype=torch.int32, device=DEV), ints([0, 0])
    added, none = ints([5, 1]), ints([0, 0])
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    w4.kv8_reserve(refs, table, lens, none, 16, stream=st)
    st.synchronize()
    with torch.cuda.graph(g, stream=st):
        status = w4.kv8_reserve(refs, table, lens, added, 16)
    for i in range(1, 4):
        g.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [5 * i, i] and status.tolist() == [0]
