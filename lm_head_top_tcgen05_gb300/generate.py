"""Generation operators: the 8-bit LM head and the sampler (C ABI in include/fkl_generate.h).

On-policy distillation trains on text that the student draws.  One step of drawing it is

    q, scale = quantize_int8(W)                       # once: a head's rows in 8 bits
    logits = int8_linear(h, q, scale, out_dtype=torch.float32)
    token, logprob = sample(logits, u, temperature=0.8, top_p=0.95)

with ``h`` the hidden states [M, K] of the rows' last tokens and ``u`` one uniform random
number per row.  ``int8_matmul`` is the product of operands that are already in 8 bits.
``draw_token`` is the step as one call.  None of these has a gradient.  Inputs are on the
current device, and calls run on its current stream.  A product without a ``workspace`` uses a buffer that the calling thread keeps for
that stream, so calls of several threads and on several streams never share one; a call that is captured in
a CUDA graph has a buffer of the graph's own memory.  A ``Workspace`` that is given belongs to one thread
and one stream at a time, and one given to a captured call to that graph.
"""
from __future__ import annotations

import ctypes
import functools
import threading
from typing import Optional, Tuple, Union

import torch

from ._lib import DTYPES, FklError, FklSampleParams, check, lib

__all__ = ["quantize_int8", "int8_matmul", "int8_linear", "sample", "draw_token"]

_Setting = Union[float, int, torch.Tensor]
_local = threading.local()  # .buffers: the calling thread's default workspaces, by (device, stream)

# A generation step is a handful of microseconds on the device, so the calls below keep the
# host's part short: the raw stream without a Stream object, workspace sizes looked up by shape.
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None
_capturing = torch.cuda.is_current_stream_capturing


def _stream(device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(fn: str, M: int, N: int, K: int, device_index: int) -> int:
    n = getattr(lib(), fn)(M, N, K)
    if n == 0:
        raise FklError(1, fn, f"unsupported shape M={M} N={N} K={K}")
    return n


def _workspace(nbytes: int, device, stream: int, given) -> torch.Tensor:
    """`given` (a Workspace), or the calling thread's buffer of the stream.  A product is two
    launches that hand the tokens over in it, and the interpreter's lock is not held meanwhile: two
    threads that share a stream may queue their launches in any order, so they never share a buffer."""
    if given is not None:
        return given.get(nbytes, device)
    if _capturing():
        # a graph keeps the address: the buffer must be the graph's, not one that a later call may drop
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    try:
        buffers = _local.buffers
    except AttributeError:
        buffers = _local.buffers = {}
    key = (device.index, stream)
    buf = buffers.get(key)
    if buf is None or buf.numel() < nbytes:
        buffers[key] = buf = None
        buffers[key] = buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    return buf


def default_workspace(device: torch.device) -> Optional[torch.Tensor]:
    """The calling thread's default workspace of the device's current stream, or None.  Its first word
    is the status of the last product that used it (``read_status``)."""
    return getattr(_local, "buffers", {}).get((device.index, _stream(device)))


def _dtype(dtype: torch.dtype, name: str) -> int:
    kind = DTYPES.get(dtype)
    if kind is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16")
    return kind


def _rows(t: torch.Tensor, name: str):
    """Checks a CUDA matrix whose rows are contiguous: (rows, cols, row stride)."""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1:
        ld = max(cols, 1)
    elif ld < cols:
        raise ValueError(f"the rows of {name} must not overlap")
    return rows, cols, ld


def _vector(t: torch.Tensor, name: str, dtype: torch.dtype, n: int, device) -> int:
    if t.dtype != dtype or t.shape != (n,) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape [{n}] on {device}")
    return t.data_ptr()


def quantize_int8(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """(q int8 [M, K], scale float32 [M]): each row of x in 8-bit integers, x ~ q * scale.

    scale = largest magnitude * fl(1/127), q = x / scale rounded to nearest even.  A row with a NaN or an infinity
    has scale NaN."""
    M, K, ld = _rows(x, "x")
    kind = _dtype(x.dtype, "x")
    q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    scale = torch.empty(M, dtype=torch.float32, device=x.device)
    st = lib().fkl_quantize_int8(x.data_ptr(), kind, M, K, ld, q.data_ptr(), scale.data_ptr(), _stream(x.device))
    check(st, "fkl_quantize_int8")
    return q, scale


def _weight(wq: torch.Tensor, K: int, device) -> int:
    if wq.dtype != torch.int8 or wq.dim() != 2 or wq.shape[1] != K or wq.device != device or not wq.is_contiguous():
        raise ValueError(f"wq must be a contiguous int8 tensor [N, {K}] on {device}")
    return wq.shape[0]


def _output(out: Optional[torch.Tensor], M: int, N: int, dtype: torch.dtype, device):
    """The output and its row stride."""
    if out is None:
        return torch.empty((M, N), dtype=dtype, device=device), N
    if out.dtype != dtype or out.shape != (M, N) or out.device != device:
        raise ValueError(f"out must be {dtype} [{M}, {N}] on {device}")
    return out, _rows(out, "out")[2]


def int8_matmul(xq: torch.Tensor, x_scale: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor,
                out_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                workspace=None) -> torch.Tensor:
    """out [M, N] = (xq wq^T) * x_scale[:, None] * w_scale[None, :] for int8 xq [M, K], wq [N, K].

    K is a multiple of 16.  ``out`` may be given, with rows any stride apart.  Should a wait inside the
    kernel run out (5 s), what is not finished is NaN and ``read_status`` gives FKL_ERR_TIMEOUT."""
    if xq.dtype != torch.int8 or xq.dim() != 2 or not xq.is_cuda or not xq.is_contiguous():
        raise ValueError("xq must be a contiguous int8 CUDA tensor [M, K]")
    M, K = xq.shape
    device = xq.device
    kind = _dtype(out_dtype, "out_dtype")
    N = _weight(wq, K, device)
    xs, ws = _vector(x_scale, "x_scale", torch.float32, M, device), _vector(w_scale, "w_scale", torch.float32, N, device)
    out, ldo = _output(out, M, N, out_dtype, device)
    stream = _stream(device)
    work = _workspace(_workspace_bytes("fkl_int8_matmul_workspace_size", M, N, K, device.index), device, stream, workspace)
    st = lib().fkl_int8_matmul(xq.data_ptr(), xs, wq.data_ptr(), ws, M, N, K, kind, out.data_ptr(), ldo,
                               work.data_ptr(), work.numel(), stream)
    check(st, "fkl_int8_matmul")
    return out


def int8_linear(x: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor, out_dtype: Optional[torch.dtype] = None,
                out: Optional[torch.Tensor] = None, workspace=None) -> torch.Tensor:
    """out [M, N] = x W^T for a weight in 8 bits (``quantize_int8``): x [M, K] is brought to 8 bits
    with a scale per row, and the product is ``int8_matmul``'s.

    x is float32, bfloat16 or float16 with contiguous rows any stride apart; out_dtype defaults
    to x's.  K is a multiple of 16."""
    M, K, ldx = _rows(x, "x")
    device = x.device
    x_kind = _dtype(x.dtype, "x")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    out_kind = _dtype(out_dtype, "out_dtype")
    N = _weight(wq, K, device)
    ws = _vector(w_scale, "w_scale", torch.float32, N, device)
    out, ldo = _output(out, M, N, out_dtype, device)
    stream = _stream(device)
    work = _workspace(_workspace_bytes("fkl_int8_linear_workspace_size", M, N, K, device.index), device, stream, workspace)
    st = lib().fkl_int8_linear(x.data_ptr(), x_kind, ldx, wq.data_ptr(), ws, M, N, K, out_kind, out.data_ptr(), ldo,
                               work.data_ptr(), work.numel(), stream)
    check(st, "fkl_int8_linear")
    return out


def sample(logits: torch.Tensor, u: torch.Tensor, temperature: _Setting = 1.0, top_k: _Setting = 0,
           top_p: _Setting = 1.0, min_p: _Setting = 0.0) -> Tuple[torch.Tensor, torch.Tensor]:
    """One token per row of logits [B, V] (float32, bfloat16 or float16; rows any stride apart):
    (token int32 [B], logprob float32 [B], its log-probability among the ids kept).

    ``u`` (float32 [B], in [0, 1)) are the random numbers: the token is the first id at which the
    cumulative probability of the kept ids, in the order of ids, exceeds u.  Each setting is one
    number, or a tensor [B] (float32; int32 for top_k) with one per row: temperature (0 takes the
    largest logit), top_k (0 keeps all), top_p (1 keeps all) and min_p (0 keeps all), applied in
    this order; ties keep the lower id.  The same inputs always give the same tokens.  A row
    whose logits are all -inf (or NaN, which counts as -inf) gives token -1 and logprob NaN."""
    B, V, ld = _rows(logits, "logits")
    kind = _dtype(logits.dtype, "logits")
    device = logits.device
    up = _vector(u, "u", torch.float32, B, device)
    rows = [None, None, None, None]
    if isinstance(temperature, torch.Tensor):
        rows[0], temperature = _vector(temperature, "temperature", torch.float32, B, device), 1.0
    if isinstance(top_k, torch.Tensor):
        rows[1], top_k = _vector(top_k, "top_k", torch.int32, B, device), 0
    if isinstance(top_p, torch.Tensor):
        rows[2], top_p = _vector(top_p, "top_p", torch.float32, B, device), 1.0
    if isinstance(min_p, torch.Tensor):
        rows[3], min_p = _vector(min_p, "min_p", torch.float32, B, device), 0.0
    p = FklSampleParams(temperature, max(0, min(int(top_k), 2**31 - 1)), top_p, min_p, *rows)
    token = torch.empty(B, dtype=torch.int32, device=device)
    logprob = torch.empty(B, dtype=torch.float32, device=device)
    st = lib().fkl_sample(logits.data_ptr(), kind, B, V, ld, up, ctypes.byref(p), token.data_ptr(), logprob.data_ptr(),
                          _stream(device))
    check(st, "fkl_sample")
    return token, logprob


def draw_token(h: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor, u: torch.Tensor, temperature: _Setting = 1.0,
               top_k: _Setting = 0, top_p: _Setting = 1.0, min_p: _Setting = 0.0,
               logits: Optional[torch.Tensor] = None, workspace=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One generation step: the 8-bit head's float32 logits of h [M, K] (``int8_linear``; written
    to ``logits`` if given) and a token per row drawn from them (``sample``)."""
    logits = int8_linear(h, wq, w_scale, out_dtype=torch.float32, out=logits, workspace=workspace)
    return sample(logits, u, temperature, top_k, top_p, min_p)
