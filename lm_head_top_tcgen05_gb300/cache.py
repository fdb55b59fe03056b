"""The teacher cache in few bits (C ABI and format in include/fkl_cache.h).

    cache = quantize_cache(*teacher_topk(Ht, Wt, K=100), V=Wt.shape[0])    # 360 bytes a token instead of 800
    cache = teacher_cache(Ht, Wt, K=100)                                   # the same, in one call
    torch.save(cache.state(), path)
    loss = fused_kl(H, W, cache, mask=mask)                                # reads it

A logit is off by half a step of its 32 slots' range at most (in 8 bits 1/508 of the range, in 4 bits
1/28), their largest by nothing, and ids are kept whole.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from ._lib import FklError, check, lib
from .generate import _stream

__all__ = ["QuantizedCache", "quantize_cache", "dequantize_cache"]


def _words(K: int, V: int, bits: int) -> int:
    n = lib().fkl_cache_words(K, V, bits)
    if n == 0:
        raise FklError(1, "fkl_cache_words", f"need 1 <= K <= 1024, 1 <= V <= 2^30 and bits 4 or 8, not K={K} V={V} bits={bits}")
    return n


class QuantizedCache:
    """Records of T cached rows: ``data`` (int32 [T, words], contiguous) with the K, V and bits they were
    written with.  ``cache[a:b]`` are the rows of a micro-batch or shard, without a copy."""

    def __init__(self, data: torch.Tensor, K: int, V: int, bits: int):
        if data.dtype != torch.int32 or data.dim() != 2 or data.shape[1] != _words(K, V, bits) or not data.is_contiguous():
            raise ValueError(f"data must be a contiguous int32 tensor [T, {_words(K, V, bits)}]")
        self.data, self.K, self.V, self.bits = data, int(K), int(V), int(bits)

    def __len__(self) -> int:
        return self.data.shape[0]

    def __getitem__(self, rows: slice) -> "QuantizedCache":
        if not isinstance(rows, slice) or rows.step not in (None, 1):
            raise TypeError("a cache is indexed by a slice of consecutive rows")
        return QuantizedCache(self.data[rows], self.K, self.V, self.bits)

    def to(self, device, non_blocking: bool = False) -> "QuantizedCache":
        return QuantizedCache(self.data.to(device, non_blocking=non_blocking), self.K, self.V, self.bits)

    def state(self) -> dict:
        """What ``QuantizedCache(**state)`` makes the cache of again."""
        return {"data": self.data, "K": self.K, "V": self.V, "bits": self.bits}


def quantize_cache(topk_idx: torch.Tensor, topk_logits: torch.Tensor, V: int, bits: int = 8) -> QuantizedCache:
    """Packs a teacher cache (int32 ids and float32 logits [T, K], as ``teacher_topk`` gives them, any slot order) for a
    vocabulary of V ids into ``bits`` (8 or 4) a logit.

    -inf logits stay -inf, and so does one more than 4096 below its row's largest become.  An id outside
    [0, V) is read back as -1, and a row with a NaN or +inf as NaN, which the loss reports."""
    if not (topk_idx.is_cuda and topk_logits.is_cuda) or topk_idx.device != topk_logits.device:
        raise ValueError("topk_idx and topk_logits must be CUDA tensors on one device")
    if topk_idx.dtype != torch.int32 or topk_logits.dtype != torch.float32:
        raise TypeError("topk_idx must be int32 and topk_logits float32")
    if topk_idx.dim() != 2 or topk_logits.shape != topk_idx.shape or not (topk_idx.is_contiguous() and topk_logits.is_contiguous()):
        raise ValueError("topk_idx and topk_logits must be [T, K], contiguous")
    T, K = topk_idx.shape
    data = torch.empty((T, _words(K, V, bits)), dtype=torch.int32, device=topk_idx.device)
    st = lib().fkl_cache_pack(topk_idx.data_ptr(), topk_logits.data_ptr(), T, K, V, bits, data.data_ptr(),
                              _stream(topk_idx.device))
    check(st, "fkl_cache_pack")
    return QuantizedCache(data, K, V, bits)


def dequantize_cache(cache: QuantizedCache, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(topk_idx int32 [T, K], topk_logits float32 [T, K]) of a cache on the device, written to ``out`` if given."""
    data = cache.data
    if not data.is_cuda:
        raise ValueError("the cache must be on a CUDA device (cache.to(device))")
    T, K = data.shape[0], cache.K
    if out is None:
        out = (torch.empty((T, K), dtype=torch.int32, device=data.device),
               torch.empty((T, K), dtype=torch.float32, device=data.device))
    for t, dtype in zip(out, (torch.int32, torch.float32)):
        if t.dtype != dtype or t.shape != (T, K) or t.device != data.device or not t.is_contiguous():
            raise ValueError(f"out must be contiguous int32 and float32 tensors [{T}, {K}] on {data.device}")
    st = lib().fkl_cache_unpack(data.data_ptr(), T, K, cache.V, cache.bits, out[0].data_ptr(), out[1].data_ptr(),
                                _stream(data.device))
    check(st, "fkl_cache_unpack")
    return out
