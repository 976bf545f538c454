"""The workspaces kept for calls that pass none (host-only: no stream is used)."""

import contextlib
import gc
import weakref

import pytest
import torch

import bit_weight_only_gemm_amd as w4


class Stream:
    cuda_stream = 5
    device_index = 0

    def synchronize(self):
        pass


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda st: contextlib.nullcontext())


def test_one_that_grows_leaves_the_old_memory_where_it_is():
    """A graph captured on the stream goes on writing there."""
    kept, device = {}, torch.device("cpu")
    first = w4._ws_cache(device, 1 << 20, Stream(), kept)
    at, ref = first.data_ptr(), weakref.ref(first)
    assert w4._ws_cache(device, 4096, Stream(), kept) is first
    del first
    second = w4._ws_cache(device, 3 << 20, Stream(), kept)
    gc.collect()
    assert second.numel() * 4 >= 3 << 20
    assert ref() is not None and ref().data_ptr() == at


def test_growing_in_small_steps_keeps_little():
    """All that is kept is less than twice what is in use."""
    kept, device, sizes = {}, torch.device("cpu"), []
    for mb in range(1, 40):
        w = w4._ws_cache(device, mb << 20, Stream(), kept)
        assert w.numel() * 4 >= mb << 20
        if not sizes or sizes[-1] != w.numel():
            sizes.append(w.numel())
    assert sum(sizes) <= 2 * sizes[-1] and sizes[-1] * 4 <= 2 * (39 << 20)


def test_what_does_not_fit_twice_is_made_as_large_as_needed(monkeypatch):
    made = []

    def limited(nbytes, device):
        if nbytes > 5 << 20:
            raise torch.OutOfMemoryError
        made.append(nbytes)
        return torch.zeros(nbytes // 4, dtype=torch.int32)

    monkeypatch.setattr(w4, "workspace", limited)
    kept, device = {}, torch.device("cpu")
    for need in (3 << 20, 4 << 20):
        assert w4._ws_cache(device, need, Stream(), kept).numel() * 4 >= need
    assert made == [3 << 20, 4 << 20]
    with pytest.raises(torch.OutOfMemoryError):
        w4._ws_cache(device, 6 << 20, Stream(), kept)
    assert w4._ws_cache(device, 4 << 20, Stream(), kept).numel() * 4 == 4 << 20
