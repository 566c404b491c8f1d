"""Pins of the fp64 reference of sampling and of top logits (CPU): hand-made rows, torch's sort, and
the shares that a grid of uniforms gives."""
import numpy as np
import pytest
import torch

from oracle import selection as S


def test_order_breaks_ties_by_index():
    assert list(S.order([1.0, 3.0, -0.0, 3.0, 0.0, np.nan, -np.inf, np.inf])) == [5, 7, 1, 3, 0, 2, 4, 6]
    z = np.random.default_rng(0).integers(-5, 5, 200).astype(float)
    assert list(S.order(z)) == torch.from_numpy(z).sort(descending=True, stable=True).indices.tolist()


@pytest.mark.parametrize("kw,keep", [
    (dict(), [0, 1, 2, 3]), (dict(top_k=2), [1, 2]), (dict(top_k=9), [0, 1, 2, 3]), (dict(top_p=0.5), [2]),
    (dict(top_p=0.51), [1, 2]), (dict(top_p=0.0), [2]), (dict(top_p=-1.0), [2]), (dict(top_p=1.0), [0, 1, 2, 3]),
    (dict(min_p=0.5), [1, 2]), (dict(min_p=2.0), [2]), (dict(top_k=3, top_p=0.6), [1, 2]),
    (dict(top_k=1, top_p=0.1), [2]), (dict(top_k=3, min_p=0.2), [0, 1, 2])])
def test_filters_by_hand(kw, keep):
    p = np.array([0.15, 0.25, 0.5, 0.1])       # sums in order: 0.5, 0.75, 0.9, 1
    row = np.log(p)
    n = 4000
    got = [S.sample_row(row, (i + 0.5) / n, **kw) for i in range(n)]
    share = p[keep] / p[keep].sum()
    count = np.bincount([g[0] for g in got], minlength=4)
    assert np.abs(count[keep] - n * share).max() <= 1 and count.sum() == count[keep].sum()
    assert all(abs(g[2] - p[keep].sum()) < 1e-12 and abs(g[1] - row[g[0]]) < 1e-12 for g in got)


def test_temperature_and_bad_rows():
    row = [1.0, 2.0, 2.0]
    assert S.sample_row(row, 0.99, temperature=0)[:3] == (1, 0.0, 1.0)
    lp = torch.log_softmax(torch.tensor(row, dtype=torch.float64) / 0.5, 0)
    t, logp, kept, _, _ = S.sample_row(row, 0.3, temperature=0.5)
    assert abs(logp - float(lp[t])) < 1e-12 and abs(kept - 1) < 1e-12
    for bad in ([np.nan, 1.0], [np.inf, 1.0], [-np.inf, -np.inf]):
        assert S.sample_row(bad, 0.5)[0] == -1
    assert S.sample_row(row, 0.5, temperature=np.nan)[0] == -1 and S.sample_row(row, 0.5, temperature=-1)[0] == -1
    assert S.sample_row([-np.inf, 0.0, -np.inf], 0.999)[0] == 1
    assert S.sample_row(row, np.nan)[0] == 0 and S.sample_row(row, 7.0)[0] == 2


def test_top_row():
    r = np.random.default_rng(1).standard_normal(50)
    index, rest = S.top_row(r, 7, 0.5)
    t = torch.from_numpy(r)
    assert index.tolist() == t.topk(7).indices.tolist()
    others = t.clone()
    others[index] = -np.inf
    assert abs(rest - float(torch.logsumexp(others / 0.5, 0))) < 1e-12
    assert S.top_row(r, 50)[1] == -np.inf
