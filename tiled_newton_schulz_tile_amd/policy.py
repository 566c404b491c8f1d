"""The clipped policy loss over torch tensors: himuon_policy_loss of libhimuon.

One call gives the loss, its parts, the log probability of every sampled token and, where
it is asked for, the gradient with respect to the logits, which a training program hands
to torch (``logits.backward(got.dlogits)``).  Formulas and conventions: include/himuon.h.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

from . import BF16, F32, himuon_policy, himuon_policy_loss, himuon_policy_workspace


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
    and dtype receives it (`logits` itself: in place).  Everything runs on `stream` (the current stream by default);
    the outputs and the workspace that the call allocates belong to that stream."""
    import torch
    if logits.dim() != 2 or logits.dtype not in (torch.float32, torch.bfloat16) or not logits.is_cuda:
        raise ValueError("logits must be a 2-D float32 or bfloat16 CUDA tensor")
    N, V = logits.shape
    if V < 1:
        raise ValueError("logits must have at least one column")
    dev = logits.device

    def ld_of(t, name):
        if (V > 1 and t.stride(1) != 1) or (N > 1 and t.stride(0) < V):
            raise ValueError(f"{name} must have unit column stride and rows that do not overlap")
        return t.stride(0) if N > 1 else V

    def row(t, dtype, name):
        if t is None:
            return 0
        if t.shape != (N,) or t.dtype != dtype or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of {N} elements on {dev}")
        return t.data_ptr()

    ld = ld_of(logits, "logits")
    for t, name in ((label, "label"), (weight, "weight"), (advantage, "advantage")):
        if t is None:
            raise ValueError(f"{name} is needed")
    ptrs = (row(label, torch.int64, "label"), row(weight, torch.float32, "weight"),
            row(advantage, torch.float32, "advantage"), row(old_logp, torch.float32, "old_logp"),
            row(ref_logp, torch.float32, "ref_logp"))
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.device(dev), torch.cuda.stream(s):
        if dlogits is True:
            dlogits = torch.empty(N, V, dtype=logits.dtype, device=dev)
        elif dlogits is False:
            dlogits = None
        if dlogits is not None and (dlogits.shape != logits.shape or dlogits.dtype != logits.dtype or
                                    dlogits.device != dev):
            raise ValueError("dlogits must have the shape, dtype and device of logits")
        logp = torch.empty(N, dtype=torch.float32, device=dev)
        stats = torch.empty(4, dtype=torch.float32, device=dev)
        p = himuon_policy(N, V, ld, ld_of(dlogits, "dlogits") if dlogits is not None else 0, logits.data_ptr(),
                          dlogits.data_ptr() if dlogits is not None else None, *ptrs, logp.data_ptr(),
                          stats.data_ptr(), F32 if logits.dtype == torch.float32 else BF16, clip[0], clip[1], kl_coef,
                          temperature, grad_scale)
        n = himuon_policy_workspace(p)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        himuon_policy_loss(p, ws.data_ptr(), n, s.cuda_stream)
    return PolicyLoss(stats, logp, dlogits)
