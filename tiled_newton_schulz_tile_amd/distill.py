"""Distillation over torch tensors: himuon_top_logits and himuon_distill_loss of libhimuon.

top_logits gives what a teacher keeps of each token's distribution: its k largest logits, their
tokens and the log-sum-exp of the others.  distill_loss takes them and gives the
divergence to the student's softmax and, where it is asked for, its gradient with respect to the
student's logits, which a training program hands to torch (``logits.backward(got.dlogits)``; the
loss itself has no graph).  Formulas and conventions: include/himuon.h.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import (himuon_distill, himuon_distill_loss, himuon_distill_workspace, himuon_top, himuon_top_logits,
               himuon_top_workspace)
from .adamw import _empty, _launch
from .policy import _DTYPES, _leading, _row


class TopLogits(NamedTuple):
    value: object      # logits' dtype (N, k): the largest logits, from the largest
    index: object      # int64 (N, k): their tokens
    rest: object       # float32 (N): log-sum-exp of the others / temperature


def top_logits(logits, k: int, temperature: float = 1.0, stream=None) -> TopLogits:
    """The k largest logits (k up to 1024) of each row of the (N, V) float32 or bfloat16 CUDA tensor `logits` (unit column
    stride, any row stride; V up to 2^20), equal ones by index, and the log-sum-exp of the others over the temperature.
    stream: as for policy_loss."""
    N, V, ld = _logits(logits)
    dev = logits.device
    p = himuon_top(N, V, ld, k, logits.data_ptr(), None, None, None, k, _DTYPES[logits.dtype], temperature)
    need = himuon_top_workspace(p)

    def empty(size, dtype):
        return torch.empty(size, dtype=dtype, device=dev) if stream is None else _empty(torch, stream, size, dtype)

    value, index = empty((N, k), logits.dtype), empty((N, k), torch.int64)
    buf = empty((need // 4 + N,), torch.float32)   # workspace (whole words), rest
    p.value, p.index, p.rest = value.data_ptr(), index.data_ptr(), buf.data_ptr() + need
    if stream is not None:
        logits.record_stream(stream)
    _launch(torch, dev, stream, himuon_top_logits, p, buf.data_ptr(), need)
    return TopLogits(value, index, buf[need // 4:])


class DistillLoss(NamedTuple):
    loss: object       # float32, no dimensions: sum over rows of weight * kl
    kl: object         # float32 (N): divergence of each row
    dlogits: Optional[object]


def distill_loss(logits, value, index, weight, rest=None, temperature: float = 1.0, grad_scale: float = 1.0, dlogits=True,
                 stream=None) -> DistillLoss:
    """Divergence (and gradient) from a teacher's entries to the softmax of the (N, V) float32 or bfloat16 CUDA tensor
    `logits` (unit column stride, any row stride; V up to 2^20).

    value: (N, k) float32 or bfloat16, the teacher's logits of the tokens `index`, int64 (N, k), k up to 1024 (unit
    column stride, the same row stride); an entry whose index is outside [0, V) does not count.  weight: float32 (N); a
    row with weight 0 is left out.  rest: float32 (N), the log-sum-exp of the teacher's other logits / temperature, or
    None: the teacher's probabilities are those of its entries alone.  dlogits, stream: as for policy_loss; loss, kl and
    the workspace share one allocation of the call."""
    N, V, ld = _logits(logits)
    dev = logits.device
    if value.dim() != 2 or value.dtype not in _DTYPES or value.shape[0] != N or value.device != dev:
        raise ValueError(f"value must be a float32 or bfloat16 tensor of {N} rows on {dev}")
    k = value.shape[1]
    if index.dtype is not torch.int64 or index.shape != value.shape or index.device != dev or k < 1:
        raise ValueError("index must be an int64 tensor of value's shape (one column at least) and device")
    ld_top = _leading(value, "value", N, k)
    if _leading(index, "index", N, k) != ld_top:
        raise ValueError("index must have value's row stride")
    f32 = torch.float32
    rest_at = 0 if rest is None else _row(rest, f32, N, dev, "rest")
    weight_at = _row(weight, f32, N, dev, "weight")
    given = dlogits is not True
    if not given:
        dlogits = (torch.empty(N, V, dtype=logits.dtype, device=dev) if stream is None else
                   _empty(torch, stream, (N, V), logits.dtype))
    elif dlogits is False:
        dlogits = None
    elif dlogits is not None and (dlogits.shape != logits.shape or dlogits.dtype is not logits.dtype or
                                  dlogits.device != dev):
        raise ValueError("dlogits must have the shape, dtype and device of logits")
    p = himuon_distill(N, V, ld, _leading(dlogits, "dlogits", N, V) if dlogits is not None else 0, ld_top,
                       logits.data_ptr(), dlogits.data_ptr() if dlogits is not None else None, value.data_ptr(),
                       index.data_ptr(), rest_at, weight_at, None, None, k, _DTYPES[logits.dtype], _DTYPES[value.dtype],
                       temperature, grad_scale)
    need = himuon_distill_workspace(p)
    words = 4 + need // 4 + N   # loss, workspace (whole words), kl
    buf = torch.empty(words, dtype=f32, device=dev) if stream is None else _empty(torch, stream, (words,), f32)
    base = buf.data_ptr()
    p.loss, p.kl = base, base + 16 + need
    if stream is not None:
        for t in (logits, value, index, weight, rest, dlogits):
            if t is not None:
                t.record_stream(stream)
    _launch(torch, dev, stream, himuon_distill_loss, p, base + 16, need)
    if given and dlogits is not None:
        torch.autograd.graph.increment_version(dlogits)   # a backward pass that saved what stood here has to say so
    loss, _, kl = buf.split_with_sizes((1, 3 + need // 4, N))
    return DistillLoss(loss[0], kl, dlogits)


def _logits(logits):
    """(rows, columns, row stride) of a tensor of logits."""
    if logits.dim() != 2 or logits.dtype not in _DTYPES or not logits.is_cuda:
        raise ValueError("logits must be a 2-D float32 or bfloat16 CUDA tensor")
    N, V = logits.shape
    if V < 1:
        raise ValueError("logits must have at least one column")
    return N, V, _leading(logits, "logits", N, V)
