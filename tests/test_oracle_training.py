"""Pins of the fp64 reference of the training-step operators (CPU): the policy loss's
gradient against central differences of its loss, its limits, AdamW against torch's, the
8-bit format against torch's e4m3 and the dithered rounding's mean."""
import numpy as np
import pytest
import torch

from oracle import training as T


def _rows(N, V, seed):
    r = np.random.default_rng(seed)
    z = 2 * r.standard_normal((N, V))
    label = r.integers(0, V, N)
    weight = r.random(N)
    weight[::5] = 0
    lp = z - np.log(np.exp(z).sum(1, keepdims=True))
    lp = lp[np.arange(N), label]
    return z, label, weight, r.standard_normal(N), lp - 0.2 * r.standard_normal(N), lp + 0.2 * r.standard_normal(N)


@pytest.mark.parametrize("V", [2, 5, 17])
@pytest.mark.parametrize("temperature", [1.0, 0.6])
@pytest.mark.parametrize("old,ref", [(True, True), (True, False), (False, True)])
def test_policy_gradient_is_the_difference_quotient(V, temperature, old, ref):
    N = 12
    z, y, w, A, o, r = _rows(N, V, 3 + V)
    kw = dict(old_logp=o if old else None, ref_logp=r if ref else None, clip=(0.2, 0.28), kl_coef=0.1,
              temperature=temperature)
    _, logp, grad = T.policy_loss(z, y, w, A, **kw)
    # old None: the ratio is exp(lp - (lp held constant)), so the differences hold lp where it was
    kd = dict(kw, old_logp=o if old else logp)
    h = 1e-4

    def loss_at(i, j, by):
        zz = z.copy()
        zz[i, j] += by
        return T.policy_loss(zz, y, w, A, **kd)[0][0]

    for i in range(N):
        for j in range(V):
            d = (8 * (loss_at(i, j, h) - loss_at(i, j, -h)) - (loss_at(i, j, 2 * h) - loss_at(i, j, -2 * h))) / (12 * h)
            # four-point differences: h^4 / 30 = 3e-18 times the fifth derivative, and a few 1e-16 |loss| / h of
            # cancellation, |loss| below 100
            assert abs(d - grad[i, j]) <= 2e-9 + 1e-10, (i, j, d, grad[i, j])


def test_policy_logp_is_torchs_log_softmax():
    z, y, w, A, o, r = _rows(9, 31, 5)
    _, logp, _ = T.policy_loss(z, y, w, A, temperature=0.7)
    want = torch.log_softmax(torch.from_numpy(z) / 0.7, 1).numpy()[np.arange(9), y]
    live = w != 0
    assert np.allclose(logp[live], want[live], rtol=1e-13, atol=1e-13) and not logp[~live].any()


def test_policy_clips_only_on_the_far_side():
    # ratio 1.5: clipped for a positive advantage, kept for a negative one; 0.5 the other way round
    z = np.zeros((4, 2))
    old = np.log(0.5) - np.log([1.5, 1.5, 0.5, 0.5])
    A = np.array([1.0, -1.0, 1.0, -1.0])
    s, _, g = T.policy_loss(z, [0] * 4, np.ones(4), A, old, clip=(0.2, 0.2))
    assert np.isclose(s[1], -(1.2 - 1.5 + 0.5 - 0.8)) and s[3] == 2
    assert not g[0].any() and not g[3].any() and g[1].any() and g[2].any()


@pytest.mark.parametrize("t", [1, 2, 100])
def test_adamw_is_torchs(t):
    r = np.random.default_rng(t)
    p = torch.nn.Parameter(torch.from_numpy(r.standard_normal(50)))
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.05)
    w, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for k in range(1, t + 1):
        g = r.standard_normal(50)
        p.grad = torch.from_numpy(g)
        opt.step()
        w, m, v = T.adamw(w, g, m, v, k, 3e-3, 0.9, 0.99, 1e-8, 0.05)
    assert np.allclose(p.detach().numpy(), w, rtol=1e-12, atol=1e-14)


def test_e4m3_values_are_torchs():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(T.e4m3_values(), want, equal_nan=True)


def test_pack8_gives_e4m3_neighbours_and_keeps_the_mean():
    r = np.random.default_rng(0)
    x = r.standard_normal(700) * np.exp(3 * r.standard_normal(700))
    grid = np.unique(np.abs(T.e4m3_values()[~np.isnan(T.e4m3_values())]))
    total, rounds = np.zeros(700), 400
    for k in range(rounds):
        q, s, _ = T.pack8(x, 0, int(r.integers(0, 2 ** 32)))
        assert np.isin(np.abs(q), grid).all()
        unit = np.repeat(s, T.BLOCK)[:700]
        y = np.abs(x) / unit
        lo = grid[np.maximum(np.searchsorted(grid, y * (1 + 1e-12), side="right") - 1, 0)]
        hi = grid[np.minimum(np.searchsorted(grid, y * (1 - 1e-12)), len(grid) - 1)]
        assert ((np.abs(q) == lo) | (np.abs(q) == hi)).all()
        total += q * unit
    gap = np.where(hi > lo, hi - lo, 0) * unit
    # a rounding's variance is at most gap^2 / 4: six standard deviations of the mean over the rounds
    assert (np.abs(total / rounds - x) <= 6 * gap / 2 / np.sqrt(rounds) + 1e-9 * np.abs(x)).all()


def test_pack8_edges():
    q, s, _ = T.pack8(np.zeros(300), 1, 7)
    assert not q.any() and not s.any() and s.size == 2
    q, s, _ = T.pack8(np.array([1.0, 1e-9, 0.0]), 1, 0)
    assert q[0] == 448 and q[1] == 2.0 ** -9 and q[2] == 0
    q, s, _ = T.pack8(np.array([2.0 ** -101]), 0, 0)
    assert not q.any() and not s.any()


def test_grad_norm_limits():
    assert T.grad_norm([np.array([3.0]), np.array([4.0])], 1.0)[0] == 5.0
    assert T.grad_norm([np.array([3e-9])], 1.0)[1] == 1.0
    assert np.isnan(T.grad_norm([np.array([np.inf])], 1.0)[1])


def test_pack8_leaves_elements_that_are_not_finite_alone():
    x = np.array([1.0, np.nan, -0.25, np.inf, 3e-3])
    for kind in (0, 1):
        y = np.abs(x) if kind else x
        q, s, _ = T.pack8(y, kind, 12345)
        want, unit, _ = T.pack8(np.where(np.isfinite(y), y, 0), kind, 12345)
        assert np.isnan(q[[1, 3]]).all() and np.array_equal(q[[0, 2, 4]], want[[0, 2, 4]]) and np.array_equal(s, unit)
