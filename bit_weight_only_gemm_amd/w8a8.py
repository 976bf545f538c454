"""Products of 8-bit integers with a scale per token and per output channel
(the ``w8a8_*`` entry points of ``include/w4a16.h``).

    wq, ws = w8a8_quantize(W)                  # once per layer, W [N, K]
    y = w8a8_linear(x, wq, ws)                 # x [M, K] fp16/bf16, quantized per token

    y = w8a8_gated(x, wq, ws, act="silu")      # W [2 F, K], gate and up: [M, F]

or, for rows quantized once and used by several layers:

    xq, xs = w8a8_quantize(x)
    y = w8a8_gemm(xq, xs, wq, ws, dtype=torch.bfloat16)
"""

import torch

from . import _DT, _here, _lib, _names, _need, _space_bytes, _stream, _ws_cache

_QDT = dict(_DT)
_QDT[torch.float32] = 2
_ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


def _empty(shape, dtype, device, stream=None):
    """An output tensor of the stream that the kernel runs on (the caching
    allocator reuses a block in the order of its own stream)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(t, dtypes, name, K=None):
    """Checks a matrix of rows [..., K] whose last dimension is contiguous and
    whose rows are evenly spaced and do not overlap; (rows, K, row stride in
    elements)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(map(str, dtypes)), t.dtype))
    shape = t.shape
    if len(shape) < 1 or shape[-1] == 0:
        raise ValueError("%s has no columns" % name)
    if K is not None and shape[-1] != K:
        raise ValueError("%s last dim %d != K %d" % (name, shape[-1], K))
    if len(shape) != 2:
        try:
            t = t.view(-1, shape[-1])
        except RuntimeError:
            raise ValueError("%s must have evenly spaced rows" % name) from None
    step, one = t.stride()
    if one != 1 and shape[-1] > 1:
        raise ValueError("%s must be contiguous within a row" % name)
    M = t.shape[0]
    if M > 1 and step < shape[-1]:      # expanded or overlapping rows
        raise ValueError("%s must have rows at least %d elements apart, got %d"
                         % (name, shape[-1], step))
    return M, shape[-1], step if M > 1 else shape[-1]


def _at(t):
    return None if t is None else t.data_ptr()


def w8a8_workspace_bytes(M, N, K, linear=True):
    """Bytes that w8a8_linear (or, linear=False, w8a8_gemm: 0) needs at this shape."""
    n = int(_lib.lib().w8a8_workspace_bytes(M, N, K, int(linear)))
    if n < 0:
        raise _lib.W4A16Error("w8a8_workspace_bytes: invalid shape M=%d N=%d K=%d" % (M, N, K))
    return n


def w8a8_quantize(x, stream=None):
    """Rows of x [..., K] (fp16, bf16 or fp32) -> (codes int8 [..., K], scales
    fp32 [...]): scale = max|row| / 127 (1 for a row of zeros)."""
    M, K, stride = _rows(x, tuple(_QDT), "x")
    codes = _empty(x.shape, torch.int8, x.device, stream)
    scales = _empty(x.shape[:-1], torch.float32, x.device, stream)
    _lib.check(_lib.lib().w8a8_quantize(_at(x), M, K, stride, _QDT[x.dtype], _at(codes),
                                        _at(scales), _stream(stream)), "w8a8_quantize")
    return codes, scales


def _weights(wq, w_scale, bias, dtype):
    _need(wq, torch.int8, "wq")
    if wq.dim() != 2:
        raise ValueError("wq must be [N, K]")
    N, K = wq.shape
    _need(w_scale, torch.float32, "w_scale", N)
    if bias is not None:
        _need(bias, dtype, "bias", N)
    return N, K


def _output(out, shape, dtype, device, stream):
    if out is None:
        return _empty(shape, dtype, device, stream)
    n = 1
    for d in shape:
        n *= d
    _need(out, dtype, "out", n)
    return out


def _space(workspace, need, device, stream, kept=None):
    if workspace is None and need > 0:
        workspace = _ws_cache(device, need, stream, kept)
    return workspace, _space_bytes(workspace, device)


def w8a8_gemm(xq, x_scale, wq, w_scale, bias=None, dtype=torch.bfloat16, out=None,
              workspace=None, use_workspace=True, stream=None):
    """y = (xq @ wq^T) * x_scale * w_scale + bias in ``dtype`` (fp16 or bf16)
    for codes xq [..., K], wq [N, K] from w8a8_quantize.  workspace and
    use_workspace are taken as by the other products; no shape needs one."""
    if dtype not in _DT:
        raise TypeError("dtype must be float16 or bfloat16")
    N, K = _weights(wq, w_scale, bias, dtype)
    _need(xq, torch.int8, "xq")
    if xq.shape[-1] != K:
        raise ValueError("xq last dim %d != K %d" % (xq.shape[-1], K))
    M = xq.numel() // K
    _need(x_scale, torch.float32, "x_scale", M)
    out = _output(out, (*xq.shape[:-1], N), dtype, xq.device, stream)
    workspace, nbytes = _space(workspace if use_workspace else None, 0, xq.device, stream)
    _lib.check(_lib.lib().w8a8_gemm(_at(xq), _at(x_scale), _at(wq), _at(w_scale), _at(bias),
                                    _at(out), M, N, K, _DT[dtype], _at(workspace), nbytes,
                                    _stream(stream)), "w8a8_gemm")
    return out


def w8a8_linear(x, wq, w_scale, bias=None, out=None, workspace=None, stream=None):
    """y = x @ (wq * w_scale)^T + bias for x [..., K] fp16/bf16, quantized per
    row on the way (w8a8_quantize and w8a8_gemm in one call).  workspace: one of
    w8a8_workspace_bytes (kept per stream when not given); it is written over,
    so never kv8_attention's."""
    N, K = _weights(wq, w_scale, bias, x.dtype)
    M, _, stride = _rows(x, _DT, "x", K)
    dtype = x.dtype
    out = _output(out, (*x.shape[:-1], N), dtype, x.device, stream)
    L = _lib.lib()
    workspace, nbytes = _space(workspace, L.w8a8_workspace_bytes(M, N, K, 1), x.device, stream)
    status = L.w8a8_linear(x.data_ptr(), stride, wq.data_ptr(), w_scale.data_ptr(), _at(bias),
                           out.data_ptr(), M, N, K, _DT[dtype], _at(workspace), nbytes,
                           _stream(stream))
    if status:
        _lib.check(status, "w8a8_linear")
    return out


def w8a8_gated_workspace_bytes(M, F, K):
    """Bytes that w8a8_gated needs at this shape."""
    n = int(_lib.lib().w8a8_gated_workspace_bytes(M, F, K))
    if n < 0:
        raise _lib.W4A16Error("w8a8_gated_workspace_bytes: invalid shape M=%d F=%d K=%d" % (M, F, K))
    return n


def w8a8_gated_plan(M, F, K):
    """Kernels a w8a8_gated call of this shape launches (host-only query), with the
    tiles' rows x columns and the workgroups that share a tile's K."""
    return _names(_lib.lib().w8a8_gated_plan, M, F, K).split(" + ")


def w8a8_gated(x, wq, w_scale, bias=None, act="silu", out=None, workspace=None, stream=None):
    """y = act(x @ Wg^T + bg) * (x @ Wu^T + bu) in one kernel, for x [..., K]
    fp16/bf16 quantized per row on the way: [..., F].  wq int8 [2 F, K], w_scale
    and bias [2 F] hold the gate's rows and then the up projection's.  act:
    "silu", "gelu" (with the error function) or "gelu_tanh".  workspace: one of
    w8a8_gated_workspace_bytes (kept per stream when not given); it is written
    over, so never kv8_attention's, and calls that overlap in time (graphs
    replayed side by side) must not share one; a call that is captured finds the
    kept one there from a call before, or is given one.  out must not overlap x."""
    if act not in _ACT:
        raise ValueError("act must be one of %s, got %r" % (", ".join(_ACT), act))
    N, K = _weights(wq, w_scale, bias, x.dtype)
    if N % 2:
        raise ValueError("wq must be [2 F, K], got %d rows" % N)
    M, _, stride = _rows(x, _DT, "x", K)
    _here(stream, x, wq, w_scale, bias, out, workspace)
    F, dtype = N // 2, x.dtype
    out = _output(out, (*x.shape[:-1], F), dtype, x.device, stream)
    L = _lib.lib()
    workspace, nbytes = _space(workspace, L.w8a8_gated_workspace_bytes(M, F, K), x.device, stream)
    status = L.w8a8_gated(x.data_ptr(), stride, wq.data_ptr(), w_scale.data_ptr(), _at(bias),
                          _ACT[act], out.data_ptr(), M, F, K, _DT[dtype], _at(workspace), nbytes,
                          _stream(stream))
    if status:
        _lib.check(status, "w8a8_gated")
    return out
