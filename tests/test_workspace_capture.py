"""A call that is captured and finds no workspace kept for its stream is refused
before anything that would end the capture (host-only: no stream is used)."""

import contextlib

import pytest
import torch

import bit_weight_only_gemm_amd as w4


class Stream:
    cuda_stream = 7
    device_index = 0

    def synchronize(self):
        raise RuntimeError("operation not permitted when stream is capturing")


def test_refused_and_nothing_kept(monkeypatch):
    on = []

    @contextlib.contextmanager
    def stream(st):
        on.append(st)
        yield
        on.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: bool(on))
    kept, st = {}, Stream()
    with pytest.raises(w4.W4A16Error, match="before it is captured"):
        w4._ws_cache(torch.device("cpu"), 4096, st, kept)
    assert not kept
    there = kept[torch.device("cpu"), 7] = torch.zeros(1 << 18, dtype=torch.int32)
    assert w4._ws_cache(torch.device("cpu"), 4096, st, kept) is there
