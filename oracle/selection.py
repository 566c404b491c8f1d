"""Plain fp64 reference of sampling from logits and of a row's top logits.  numpy only, row by row
from the definitions, no code shared with the GPU path."""
from __future__ import annotations

import numpy as np


def order(row):
    """Indices from the largest logit to the smallest, NaN first, equal ones by index."""
    row = np.asarray(row, np.float64) + 0.0
    return np.lexsort((np.arange(len(row)), -np.where(np.isnan(row), 0, row), ~np.isnan(row)))


def sample_row(row, uniform, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logp, kept, margin, cut): margin is the distance of uniform's place to the nearest border between
    tokens, cut that of top_p's target to the nearest sum that it is compared with, both over the sums they part."""
    row = np.asarray(row, np.float64) + 0.0
    V = len(row)
    T = float(temperature)
    if np.isnan(row).any() or row.max() == np.inf or row.max() == -np.inf or not (T == 0 or 2.0 ** -20 <= T <= 2.0 ** 20):
        return -1, np.nan, np.nan, np.inf, np.inf
    if T == 0:
        return int(order(row)[0]), 0.0, 1.0, np.inf, np.inf
    line = order(row)
    line = line[np.isfinite(row[line])]
    y = (row - row.max()) / T
    e = np.exp(y)
    sums = np.cumsum(e[line])
    n = len(line)
    if 1 <= top_k <= V:
        n = min(n, int(top_k))
    cut = np.inf
    if top_p < 1:
        target = max(float(top_p), 0.0) * sums[n - 1]
        cut = np.abs(sums[:n] - target).min() / sums[n - 1] if target > 0 else np.inf
        n = min(n, int((sums[:n] < target).sum()) + 1)
    n = min(n, max(1, int((e[line] >= min(float(min_p), 1.0)).sum())))
    keep = np.sort(line[:n])
    keep = keep[e[keep] > 0]
    sums = np.cumsum(e[keep])
    u = 0.0 if np.isnan(uniform) else min(max(float(uniform), 0.0), 1.0)
    target = u * sums[-1]
    at = min(int((sums <= target).sum()), len(keep) - 1)
    margin = np.abs(sums[:-1] - target).min() / sums[-1] if len(keep) > 1 else np.inf
    return int(keep[at]), float(y[keep[at]] - np.log(e.sum())), float(sums[-1] / e.sum()), margin, cut


def top_row(row, k, temperature=1.0):
    """(index, rest): the k largest, and the log-sum-exp of the others over the temperature."""
    row = np.asarray(row, np.float64) + 0.0
    line = order(row)
    others = row[line[k:]] / temperature
    if len(others) == 0 or others[0] == -np.inf:
        return line[:k], -np.inf
    if np.isnan(others[0]) or others[0] == np.inf:
        return line[:k], np.nan
    return line[:k], float(others[0] + np.log(np.exp(others - others[0]).sum()))
