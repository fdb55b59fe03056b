"""Scoring: log-probabilities of given tokens, entropies and alternatives (C ABI in include/fkl_score.h).

Text that was drawn (``sample``, ``draw_token``) is scored from logits in memory,

    r = token_logprobs(logits, tokens, temperature=0.8, top_n=20)
    r.logprob, r.entropy, r.top_ids, r.top_logprobs

or straight from hidden states and the LM head, whose logits are never written,

    logprob, entropy = fused_logprobs(H, W, tokens, mask)

Both are differentiable (``logprob`` and ``entropy``; in the logits, or in H and W), for a policy
gradient, a cross-entropy or an entropy bonus on the drawn text:

    loss = -(advantage * logprob).sum() / n - 0.01 * entropy.sum() / n
    loss.backward()

``logprob_forward`` and ``logprob_backward`` are the explicit calls of the fused form.  Inputs are on the
current device, and calls run on its current stream.  A call without a ``workspace`` takes its scratch from
PyTorch's allocator for as long as it runs, so calls of several threads, streams and captured graphs share none.
A step that is captured in a CUDA graph takes its gradients with ``torch.autograd.grad`` or the explicit calls;
``backward()`` would add into leaves on the stream of an eager graph that they still belong to.
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional, Tuple, Union

import torch
from torch.autograd.function import once_differentiable

from ._lib import FKL_ACCUMULATE_DH, FKL_ACCUMULATE_DW, FklError, check, lib
from .generate import _dtype, _rows, _stream, _vector

__all__ = ["TokenLogprobs", "token_logprobs", "fused_logprobs", "logprob_forward", "logprob_backward"]

_TOKEN_BYTES = {torch.int32: 4, torch.int64: 8}


class TokenLogprobs(NamedTuple):
    """What ``token_logprobs`` returns; the last two are None without alternatives (top_n = 0)."""

    logprob: torch.Tensor
    entropy: torch.Tensor
    top_ids: Optional[torch.Tensor]
    top_logprobs: Optional[torch.Tensor]


def _tokens(tokens: torch.Tensor, n: int, device) -> int:
    """Bytes of a token id, of checked tokens."""
    size = _TOKEN_BYTES.get(tokens.dtype)
    if size is None or tokens.shape != (n,) or tokens.device != device or not tokens.is_contiguous():
        raise ValueError(f"tokens must be a contiguous int32 or int64 tensor of shape [{n}] on {device}")
    return size


def _mask(mask: Optional[torch.Tensor], n: int, device) -> Optional[torch.Tensor]:
    if mask is None:
        return None
    if mask.dtype not in (torch.uint8, torch.bool) or mask.shape != (n,) or mask.device != device:
        raise ValueError(f"mask must be a uint8 or bool tensor of shape [{n}] on {device}")
    return mask.contiguous()


def _address(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _temperature(temperature, n: int, device):
    """(number, address of the rows' values or None)."""
    if isinstance(temperature, torch.Tensor):
        return 1.0, _vector(temperature, "temperature", torch.float32, n, device)
    return float(temperature), None


# ---------------------------------------------------------------- logits in memory
def _score(logits, tokens, temperature, top_n, mask, want_stats):
    B, V, ld = _rows(logits, "logits")
    kind = _dtype(logits.dtype, "logits")
    device = logits.device
    size = _tokens(tokens, B, device)
    mask = _mask(mask, B, device)
    number, per_row = _temperature(temperature, B, device)
    logprob = torch.empty(B, dtype=torch.float32, device=device)
    entropy = torch.empty(B, dtype=torch.float32, device=device)
    stats = torch.empty((B, 2), dtype=torch.float32, device=device) if want_stats else None
    ids = logs = None
    if top_n > 0:
        ids = torch.empty((B, top_n), dtype=torch.int32, device=device)
        logs = torch.empty((B, top_n), dtype=torch.float32, device=device)
    st = lib().fkl_token_logprobs(logits.data_ptr(), kind, B, V, ld, tokens.data_ptr(), size, _address(mask), number,
                                  per_row, top_n, logprob.data_ptr(), entropy.data_ptr(), _address(stats),
                                  _address(ids), _address(logs), _stream(device))
    check(st, "fkl_token_logprobs")
    return logprob, entropy, ids, logs, stats


def _grad_like(logits: torch.Tensor) -> torch.Tensor:
    """A tensor for the logits' gradient whose rows lie in 16-byte vectors as the logits' do, where they can."""
    B, V = logits.shape
    unit = 16 // logits.element_size()
    if V % unit and B > 1 and logits.stride(0) % unit == 0:
        wide = torch.empty((B, (V + unit - 1) // unit * unit), dtype=logits.dtype, device=logits.device)
        return wide[:, :V]
    return torch.empty((B, V), dtype=logits.dtype, device=logits.device)


def _score_backward(ctx, grad_logprob, grad_entropy, _ids, _logs):
    logits, tokens, entropy, stats, mask, rows = ctx.saved_tensors
    if grad_logprob is None and grad_entropy is None:
        return None, None, None, None, None
    B, V, ld = _rows(logits, "logits")
    out = _grad_like(logits)
    if grad_logprob is not None:
        grad_logprob = grad_logprob.contiguous()
    if grad_entropy is not None:
        grad_entropy = grad_entropy.contiguous()
    st = lib().fkl_token_logprobs_backward(
        logits.data_ptr(), _dtype(logits.dtype, "logits"), B, V, ld, tokens.data_ptr(), _TOKEN_BYTES[tokens.dtype],
        _address(mask), ctx.number, _address(rows), stats.data_ptr(), entropy.data_ptr(), _address(grad_logprob),
        _address(grad_entropy), out.data_ptr(), out.stride(0) if B > 1 else V, _stream(logits.device))
    check(st, "fkl_token_logprobs_backward")
    return out, None, None, None, None


# The engine's thread calls a backward, and a short one is mostly Python: the wrapper that makes a second
# derivative an error (about 10 us) is only taken where one can be asked for (create_graph=True).
_score_backward_once = once_differentiable(_score_backward)


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature, top_n, mask):
        mask = _mask(mask, logits.shape[0], logits.device)
        logprob, entropy, ids, logs, stats = _score(logits, tokens, temperature, top_n, mask, True)
        rows = temperature if isinstance(temperature, torch.Tensor) else None
        ctx.save_for_backward(logits, tokens, entropy, stats, mask, rows)
        ctx.number = 1.0 if rows is not None else float(temperature)
        ctx.set_materialize_grads(False)
        if ids is not None:
            ctx.mark_non_differentiable(ids, logs)
        return logprob, entropy, ids, logs

    @staticmethod
    def backward(ctx, *grads):
        return _score_backward_once(ctx, *grads) if torch.is_grad_enabled() else _score_backward(ctx, *grads)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, temperature: Union[float, torch.Tensor] = 1.0,
                   top_n: int = 0, mask: Optional[torch.Tensor] = None) -> TokenLogprobs:
    """Scores ``tokens`` [B] (int32 or int64) under softmax(logits / temperature), logits [B, V] (float32,
    bfloat16 or float16; rows any stride apart): the tokens' log-probability and the distribution's entropy
    (float32 [B], differentiable in the logits) and the ``top_n`` (at most 128, and V) likeliest ids, int32 and
    float32 [B, top_n], likeliest first, ties by the lower id.

    ``temperature`` is one number or a float32 tensor [B], a constant: one that wants a gradient is refused.  ``mask``
    (uint8 or bool [B]) leaves rows out: log-probability, entropy and gradient 0, ids -1.  -inf bans an id, NaN counts as
    -inf (in ``fused_logprobs`` it makes its row NaN), +inf ids share all the probability.  A token outside [0, V) in
    another row gives NaN, in its log-probability and its row of the gradient; so does a row without any logit, and
    a temperature in a tensor that is not finite and above 4.25e-39."""
    if not 0 <= top_n <= 128:
        raise ValueError("top_n must be between 0 and 128")
    if isinstance(temperature, torch.Tensor) and temperature.requires_grad and torch.is_grad_enabled():
        raise ValueError("temperature gets no gradient from the scores: pass temperature.detach()")
    if logits.requires_grad and torch.is_grad_enabled():
        return TokenLogprobs(*_TokenLogprobs.apply(logits, tokens, temperature, top_n, mask))
    return TokenLogprobs(*_score(logits, tokens, temperature, top_n, mask, False)[:4])


# ---------------------------------------------------------------- hidden states and head
def _operands(H, W, tokens, mask):
    if not (H.is_cuda and W.is_cuda) or H.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise TypeError("H and W must be bfloat16 CUDA tensors")
    if H.dim() != 2 or W.dim() != 2 or H.shape[1] != W.shape[1] or not (H.is_contiguous() and W.is_contiguous()):
        raise ValueError("H must be [T, d] and W [V, d], contiguous")
    if W.device != H.device:
        raise ValueError("H and W must be on one device")
    T = H.shape[0]
    return _tokens(tokens, T, H.device), _mask(mask, T, H.device)


def _scratch(workspace, nbytes: int, device) -> torch.Tensor:
    return workspace.get(nbytes, device) if workspace is not None else torch.empty(nbytes, dtype=torch.uint8, device=device)


def _floats(t: Optional[torch.Tensor], name: str, T: int, device) -> Optional[torch.Tensor]:
    if t is None:
        return None
    if t.dtype != torch.float32 or t.shape != (T,) or t.device != device:
        raise ValueError(f"{name} must be a float32 tensor of shape [{T}] on {device}")
    return t.detach().contiguous()


@functools.lru_cache(maxsize=1024)
def _forward_bytes(T: int, d: int, V: int) -> int:
    n = lib().fkl_logprob_workspace_size(T, d, V)
    if n == 0:
        raise FklError(1, "fkl_logprob_workspace_size", f"unsupported shape T={T} d={d} V={V}")
    return n


@functools.lru_cache(maxsize=1024)
def _backward_bytes(T: int, d: int, V: int, chunk: int, bf16: int) -> int:
    n = lib().fkl_logprob_backward_workspace_size(T, d, V, chunk, bf16)
    if n == 0:
        raise FklError(1, "fkl_logprob_backward_workspace_size", f"unsupported shape T={T} d={d} V={V} chunk={chunk}")
    return n


def _stats(t: Optional[torch.Tensor], T: int, device) -> Optional[torch.Tensor]:
    if t is not None and (t.dtype != torch.float32 or t.shape != (T, 2) or t.device != device or not t.is_contiguous()):
        raise ValueError(f"stats must be a contiguous float32 tensor of shape [{T}, 2] on {device}")
    return t


def _launch_forward(H, W, tokens, size, mask, tau, workspace, lse, stats):
    (T, d), V, device = H.shape, W.shape[0], H.device
    ws = _scratch(workspace, _forward_bytes(T, d, V), device)
    logprob = torch.empty(T, dtype=torch.float32, device=device)
    entropy = torch.empty(T, dtype=torch.float32, device=device)
    st = lib().fkl_logprob_forward_ex(H.data_ptr(), W.data_ptr(), tokens.data_ptr(), size, _address(mask), T, d, V,
                                      float(tau), logprob.data_ptr(), entropy.data_ptr(), _address(lse),
                                      _address(stats), ws.data_ptr(), ws.numel(), _stream(device))
    check(st, "fkl_logprob_forward_ex")
    return logprob, entropy


def logprob_forward(H: torch.Tensor, W: torch.Tensor, tokens: torch.Tensor, mask: Optional[torch.Tensor] = None,
                    tau: float = 1.0, workspace=None, stats: Optional[torch.Tensor] = None,
                    ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(logprob, entropy, lse), float32 [T], of ``tokens`` [T] under softmax(H W^T / tau); lse is that of every row,
    the masked ones included.  ``stats`` (float32 [T, 2], optional) receives each row's reference logit and the log of
    its sum, from which the backward knows q at any temperature.  A wait of the product that runs out makes
    all of them NaN, as a token outside [0, V) does its log-probability; ``read_status(workspace)`` tells."""
    size, mask = _operands(H, W, tokens, mask)
    T = H.shape[0]
    lse = torch.empty(T, dtype=torch.float32, device=H.device)
    logprob, entropy = _launch_forward(H, W, tokens, size, mask, tau, workspace, lse, _stats(stats, T, H.device))
    return logprob, entropy, lse


def _launch_backward(H, W, tokens, mask, logprob, entropy, lse, stats, grad_logprob, grad_entropy, tau, chunk, out, bf16,
                     flags, workspace):
    (T, d), V, device = H.shape, W.shape[0], H.device
    if T == 0 and out[1] is None:  # nothing to write, and no address to say so with
        return
    ws = _scratch(workspace, _backward_bytes(T, d, V, chunk, bf16), device)
    st = lib().fkl_logprob_backward_ex(
        H.data_ptr(), W.data_ptr(), tokens.data_ptr(), _TOKEN_BYTES[tokens.dtype], _address(mask), logprob.data_ptr(),
        entropy.data_ptr(), _address(lse), _address(stats), _address(grad_logprob), _address(grad_entropy), T, d, V,
        float(tau), chunk, bf16, flags, _address(out[0]), _address(out[1]), ws.data_ptr(), ws.numel(), _stream(device))
    check(st, "fkl_logprob_backward_ex")


def logprob_backward(H: torch.Tensor, W: torch.Tensor, tokens: torch.Tensor, mask: Optional[torch.Tensor],
                     logprob: torch.Tensor, entropy: torch.Tensor, lse: Optional[torch.Tensor],
                     grad_logprob: Optional[torch.Tensor] = None, grad_entropy: Optional[torch.Tensor] = None,
                     tau: float = 1.0, chunk: int = 2048, workspace=None,
                     out: Optional[Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]] = None,
                     accumulate: bool = False, grad_dtype: torch.dtype = torch.float32,
                     stats: Optional[torch.Tensor] = None,
                     ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """dH [T, d] and dW [V, d], the gradient of sum(grad_logprob * logprob + grad_entropy * entropy) (float32 [T]
    each; None = 0), in float32 or, with ``grad_dtype=torch.bfloat16``, in bfloat16 (fp32 sums rounded once).

    ``logprob``, ``entropy``, ``lse`` and ``stats`` are the forward's (with ``stats`` lse may be None).  Without ``stats``
    the probabilities come from lse, whose rounding is 2^-24 |lse| of them, and a row with |lse| above 32768 (low
    temperatures: logits of 30 below tau = 1e-3) has NaN gradients.  ``chunk`` bounds the buffer of the logits' gradient:
    at most max(chunk * V, 256 * T) bfloat16 values.  ``out`` gives the tensors to write, one of them None if it is not
    wanted (a frozen head: ``(dH, None)``); ``accumulate=True`` adds into them (float32)."""
    if grad_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("grad_dtype must be torch.float32 or torch.bfloat16")
    bf16 = grad_dtype == torch.bfloat16
    if accumulate and (bf16 or out is None):
        raise ValueError("accumulate=True adds into float32 gradients given in `out`")
    _, mask = _operands(H, W, tokens, mask)
    T, device = H.shape[0], H.device
    logprob, entropy = _floats(logprob, "logprob", T, device), _floats(entropy, "entropy", T, device)
    lse, stats = _floats(lse, "lse", T, device), _stats(stats, T, device)
    grad_logprob = _floats(grad_logprob, "grad_logprob", T, device)
    grad_entropy = _floats(grad_entropy, "grad_entropy", T, device)
    if out is None:
        out = tuple(torch.empty(t.shape, dtype=grad_dtype, device=device) for t in (H, W))
    for g, t in zip(out, (H, W)):
        if g is not None and (g.dtype != grad_dtype or g.shape != t.shape or not g.is_contiguous() or g.device != device):
            raise ValueError(f"out gradients must be contiguous {grad_dtype} {tuple(t.shape)} on {device}")
    flags = (FKL_ACCUMULATE_DH | FKL_ACCUMULATE_DW) if accumulate else 0
    _launch_backward(H, W, tokens, mask, logprob, entropy, lse, stats, grad_logprob, grad_entropy, tau, chunk, out,
                     int(bf16), flags, workspace)
    return out


def _fused_backward(ctx, grad_logprob, grad_entropy):
    H, W, tokens, mask, logprob, entropy, stats = ctx.saved_tensors
    if grad_logprob is None and grad_entropy is None:
        return None, None, None, None, None, None
    need = ctx.needs_input_grad
    out = (torch.empty_like(H) if need[0] else None, torch.empty_like(W) if need[1] else None)
    grad_logprob = None if grad_logprob is None else grad_logprob.contiguous()
    grad_entropy = None if grad_entropy is None else grad_entropy.contiguous()
    _launch_backward(H, W, tokens, mask, logprob, entropy, None, stats, grad_logprob, grad_entropy, ctx.tau, ctx.chunk,
                     out, 1, 0, None)
    return out[0], out[1], None, None, None, None


_fused_backward_once = once_differentiable(_fused_backward)


class _FusedLogprobs(torch.autograd.Function):
    """Saves the forward's scores and statistics; the backward recomputes the projection block by block."""

    @staticmethod
    def forward(ctx, H, W, tokens, mask, tau, chunk):
        size, mask = _operands(H, W, tokens, mask)
        _backward_bytes(H.shape[0], H.shape[1], W.shape[0], chunk, 1)  # refuses a chunk here, not in the backward
        stats = torch.empty((H.shape[0], 2), dtype=torch.float32, device=H.device)
        logprob, entropy = _launch_forward(H, W, tokens, size, mask, tau, None, None, stats)
        ctx.save_for_backward(H, W, tokens, mask, logprob, entropy, stats)
        ctx.tau, ctx.chunk = tau, chunk
        ctx.set_materialize_grads(False)
        return logprob, entropy

    @staticmethod
    def backward(ctx, *grads):
        return _fused_backward_once(ctx, *grads) if torch.is_grad_enabled() else _fused_backward(ctx, *grads)


def fused_logprobs(H: torch.Tensor, W: torch.Tensor, tokens: torch.Tensor, mask: Optional[torch.Tensor] = None,
                   tau: float = 1.0, chunk: int = 2048) -> Tuple[torch.Tensor, torch.Tensor]:
    """(logprob, entropy), float32 [T], of ``tokens`` [T] (int32 or int64) under softmax(H W^T / tau) for hidden
    states H [T, d] and LM head W [V, d] (bfloat16), without the [T, V] logits in memory; differentiable in H and W.

    ``tau`` is any finite number above 4.25e-39.  ``mask`` (uint8 or bool [T]) leaves tokens out: log-probability, entropy
    and gradient 0.  A token outside [0, V) in another row gives NaN there, and NaN gradients; so does a NaN among a
    row's logits (in ``token_logprobs`` it counts as -inf), in the row's scores, its dH and dW.  ``chunk`` bounds the
    backward's buffer of the logits' gradient: at most max(chunk * V, 256 * T) bfloat16 values."""
    if torch.is_grad_enabled() and (H.requires_grad or W.requires_grad):
        return _FusedLogprobs.apply(H, W, tokens, mask, tau, chunk)
    size, mask = _operands(H, W, tokens, mask)
    return _launch_forward(H, W, tokens, size, mask, tau, None, None, None)
