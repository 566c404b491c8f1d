"""The clipped policy loss over torch tensors: himuon_policy_loss of libhimuon.

One call gives the loss, its parts, the log probability of every sampled token and, where
it is asked for, the gradient with respect to the logits, which a training program hands
to torch (``logits.backward(got.dlogits)``; the loss itself has no graph).  Formulas and conventions: include/himuon.h.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import BF16, F32, himuon_policy, himuon_policy_loss, himuon_policy_workspace
from .adamw import _empty, _launch

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


class PolicyLoss(NamedTuple):
    stats: object      # float32 (4): loss; sums over rows of weight * (-min(u, c)), weight * kl, weight of clipped rows
    logp: object       # float32 (N): log probability of each row's label
    dlogits: Optional[object]

    @property
    def loss(self):
        return self.stats[0]


def policy_loss(logits, label, weight, advantage, old_logp=None, ref_logp=None, clip=(0.2, 0.2), kl_coef: float = 0.0,
                temperature: float = 1.0, grad_scale: float = 1.0, dlogits=True, stream=None) -> PolicyLoss:
    """Clipped policy loss (and gradient) of the (N, V) float32 or bfloat16 CUDA tensor `logits` (unit column stride,
    any row stride).

    label: int64 (N); weight, advantage, old_logp, ref_logp: float32 (N).  A row with weight 0 or a label outside
    [0, V) is left out.  old_logp None: the ratio is 1; ref_logp None: no KL term.  clip: the pair (low, high).
    dlogits: True allocates the gradient, False or None computes the forward pass alone, a tensor of logits' shape
    and dtype receives it (`logits` itself: in place).  Everything runs on `stream` (the current stream by default),
    whose work has to come after what made the arguments; stats, logp and the workspace share one allocation of the
    call.  With a `stream`, results are allocated on it and arguments are recorded on it (torch's record_stream)."""
    if logits.dim() != 2 or logits.dtype not in _DTYPES or not logits.is_cuda:
        raise ValueError("logits must be a 2-D float32 or bfloat16 CUDA tensor")
    N, V = logits.shape
    if V < 1:
        raise ValueError("logits must have at least one column")
    dev = logits.device
    ld = _leading(logits, "logits", N, V)
    f32 = torch.float32
    rows = (_row(label, torch.int64, N, dev, "label"), _row(weight, f32, N, dev, "weight"),
            _row(advantage, f32, N, dev, "advantage"),
            0 if old_logp is None else _row(old_logp, f32, N, dev, "old_logp"),
            0 if ref_logp is None else _row(ref_logp, f32, N, dev, "ref_logp"))
    given = dlogits is not True
    if not given:
        dlogits = (torch.empty(N, V, dtype=logits.dtype, device=dev) if stream is None else
                   _empty(torch, stream, (N, V), logits.dtype))
    elif dlogits is False:
        dlogits = None
    elif dlogits is not None and (dlogits.shape != logits.shape or dlogits.dtype is not logits.dtype or
                                  dlogits.device != dev):
        raise ValueError("dlogits must have the shape, dtype and device of logits")
    p = himuon_policy(N, V, ld, _leading(dlogits, "dlogits", N, V) if dlogits is not None else 0, logits.data_ptr(),
                      dlogits.data_ptr() if dlogits is not None else None, *rows, None, None,
                      _DTYPES[logits.dtype], clip[0], clip[1], kl_coef, temperature, grad_scale)
    need = himuon_policy_workspace(p)
    words = 4 + need // 4 + N   # stats, workspace (whole words), logp
    buf = torch.empty(words, dtype=f32, device=dev) if stream is None else _empty(torch, stream, (words,), f32)
    base = buf.data_ptr()
    p.stats, p.logp = base, base + 16 + need
    if stream is not None:
        for t in (logits, label, weight, advantage, old_logp, ref_logp, dlogits):
            if t is not None:
                t.record_stream(stream)
    _launch(torch, dev, stream, himuon_policy_loss, p, base + 16, need)
    if given and dlogits is not None:
        torch.autograd.graph.increment_version(dlogits)   # a backward pass that saved what stood here has to say so
    stats, _, logp = buf.split_with_sizes((4, need // 4, N))
    return PolicyLoss(stats, logp, dlogits)


def _row(t, dtype, N, dev, name):
    if t is None or t.dtype is not dtype or t.shape != (N,) or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {N} elements on {dev}")
    return t.data_ptr()


def _leading(t, name, N, V):
    if N <= 1:
        if V > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must have unit column stride")
        return V
    rows, cols = t.stride()
    if (V > 1 and cols != 1) or rows < V:
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")
    return rows
