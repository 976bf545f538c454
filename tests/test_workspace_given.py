"""Workspaces that a caller passes: memory that the kernels cannot write over is
refused before the library is called (host-only: the tensors here only claim to be
on the GPU, and the library's entry points are replaced)."""

import os

import pytest
import torch

import bit_weight_only_gemm_amd as w4
from bit_weight_only_gemm_amd import _lib

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libw4a16.so not built", allow_module_level=True)


class OnGpu(torch.Tensor):
    is_cuda = True


class Sizes:
    """The library's sizes, and nothing that launches."""

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(_lib.load(), name)

        def entry(*args):
            raise AssertionError("%s was called" % name)
        return entry


def z(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def cache():
    c = {"k": z(8, 2, 16, 64, dtype=torch.uint8), "v": z(8, 2, 1, 64, 16, dtype=torch.uint8),
         "k_scale": z(8, 2, dtype=torch.float32), "v_scale": z(8, 2, dtype=torch.float32)}
    return {**c, "page_size": 16, "kv_heads": 2, "head_dim": 64, "num_pages": 8}


def linear(fn, M, K, **kw):
    x = z(M, K, dtype=torch.float16)
    return fn(x, z(256, K, dtype=torch.int8), z(256, dtype=torch.float32), **kw)


def int4(**kw):
    packed = {"codes": z(64), "scales": z(64), "zeros": z(64), "perm": None, "K": 128, "N": 64, "group_size": 128}
    return w4.w4a16_gemm(z(1, 128, dtype=torch.float16), packed, **kw)


def nf4(**kw):
    q = {"qweight": z(64), "absmax_q": z(64), "absmax_scale": z(64), "K": 128, "N": 64, "blocksize": 64}
    return w4.nf4_gemm(z(1, 128, dtype=torch.float16), q, **kw)


def attention(fn, **kw):
    return fn(z(2, 4, 64, dtype=torch.float16), cache(), z(2, 4), z(2), **kw)


CALLS = {
    "kv8_reserve": lambda **kw: w4.kv8_reserve(z(8), z(3, 4), z(3), z(3), 16, status=z(1), **kw),
    "kv8_fork": lambda **kw: w4.kv8_fork(cache(), z(8), z(3, 4), z(3), z(1), z(1), status=z(1), **kw),
    "kv8_compact": lambda **kw: w4.kv8_compact(cache(), z(8), z(3, 4), z(3), z(3, 4), z(8), **kw),
    "w8a8_linear": lambda **kw: linear(w4.w8a8_linear, 70, 128, **kw),
    "w8a8_gated": lambda **kw: linear(w4.w8a8_gated, 70, 128, **kw),
    "kv8_attention": lambda **kw: attention(w4.kv8_attention, **kw),
    "kv8_attention_scored": lambda **kw: attention(w4.kv8_attention_scored, **kw),
    "w4a16_gemm": int4,
    "nf4_gemm": nf4,
}


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    monkeypatch.setattr(_lib, "lib", Sizes)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)


@pytest.mark.parametrize("name", CALLS)
def test_a_good_one_reaches_the_library(name):
    with pytest.raises(AssertionError, match=name + " was called"):
        CALLS[name](workspace=z(1 << 20))


@pytest.mark.parametrize("name", CALLS)
def test_host_memory_is_refused(name):
    with pytest.raises((TypeError, ValueError)):
        CALLS[name](workspace=torch.zeros(1 << 20, dtype=torch.int32))


@pytest.mark.parametrize("name", CALLS)
def test_less_memory_than_elements_is_refused(name):
    with pytest.raises(ValueError, match="contiguous"):
        CALLS[name](workspace=z(1).expand(1 << 20))


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_another_device_is_refused(name):
    with pytest.raises(ValueError):
        CALLS[name](workspace=torch.zeros(1 << 20, dtype=torch.int32, device="meta").as_subclass(OnGpu))
