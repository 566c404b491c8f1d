"""Sampling tokens from logits over torch tensors: himuon_sample of libhimuon.

One call draws a token a row under temperature, top-k, top-p and min-p from random numbers that
the caller gives, and its log probability without the filters, which is what policy_loss takes as
old_logp.  Definitions and conventions: include/himuon.h.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import himuon_sample, himuon_sample_workspace, himuon_sampling
from .adamw import _empty, _launch
from .distill import _logits
from .policy import _DTYPES, _row


class Sampled(NamedTuple):
    token: object      # int64 (N); -1 for a row that has no distribution
    logp: object       # float32 (N): log of the token's probability under softmax(logits / temperature)
    kept: object       # float32 (N): the probability of all tokens that the filters kept


def sample(logits, uniform, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None) -> Sampled:
    """A token for each row of the (N, V) float32 or bfloat16 CUDA tensor `logits` (unit column stride, any row stride; V
    up to 2^20), from `uniform`, float32 (N) numbers in [0, 1).

    temperature (0: the largest logit), top_k (0: all), top_p (1: all) and min_p (0: all) are numbers for all rows or
    tensors of one a row, float32 (N) (top_k int32).  The filters apply one after the other, in this order; at least one
    token is kept.  stream: as for policy_loss; token, logp and kept share one allocation of the call."""
    N, V, ld = _logits(logits)
    dev = logits.device
    f32 = torch.float32
    settings, at = [], []
    for x, name, dtype, none in ((temperature, "temperature", f32, 1.0), (top_k, "top_k", torch.int32, 0),
                                 (top_p, "top_p", f32, 1.0), (min_p, "min_p", f32, 0.0)):
        each = isinstance(x, torch.Tensor)
        at.append(_row(x, dtype, N, dev, name) if each else None)
        settings.append(none if each else x)
    T, k, top_p_all, min_p_all = settings
    p = himuon_sampling(N, V, ld, logits.data_ptr(), _row(uniform, f32, N, dev, "uniform"), *at, None, None, None,
                        _DTYPES[logits.dtype], k if 0 < k < V else 0, T, top_p_all, min_p_all)
    need = himuon_sample_workspace(p)
    words = need // 8 + 2 * N   # workspace (whole words), token, logp and kept
    buf = torch.empty(words, dtype=torch.int64, device=dev) if stream is None else _empty(torch, stream, (words,), torch.int64)
    base = buf.data_ptr()
    p.token, p.logp, p.kept = base + need, base + need + 8 * N, base + need + 12 * N
    if stream is not None:
        for t in (logits, uniform, temperature, top_k, top_p, min_p):
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    _launch(torch, dev, stream, himuon_sample, p, base, need)
    _, token, rest = buf.split_with_sizes((need // 8, N, N))
    return Sampled(token, *rest.view(f32).split_with_sizes((N, N)))
