"""Pins of the fp64 reference of the distillation loss (CPU): its gradient against differences
of its loss, its limits, and torch's divergence."""
import numpy as np
import pytest
import torch

from oracle import training as T


def rows(N, V, k, seed, twice=False):
    r = np.random.default_rng(seed)
    z, teacher = 2 * r.standard_normal((N, V)), 2 * r.standard_normal((N, V))
    index = np.argsort(-teacher, 1)[:, :k].copy()
    value = np.take_along_axis(teacher, index, 1)
    if twice:
        index[:, -1] = index[:, 0]
    off = teacher.copy()
    np.put_along_axis(off, index, -np.inf, 1)
    weight = r.random(N) + 0.1
    weight[::5] = 0
    with np.errstate(all="ignore"):
        rest = np.log(np.exp(off).sum(1))
    return z, value, index, weight, rest


@pytest.mark.parametrize("V,k", [(2, 1), (5, 3), (5, 5), (17, 4)])
@pytest.mark.parametrize("temperature", [1.0, 0.6])
@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("twice", [False, True])
def test_distill_gradient_is_the_difference_quotient(V, k, temperature, rest, twice):
    z, value, index, weight, r = rows(6, V, k, V + k, twice and k > 1)
    index[2, -1] = -1
    if rest and k == V:
        r = np.full_like(r, -np.inf)   # no other token: nothing may be left for it
        index[2, -1] = index[2, 0]
    kw = dict(rest=r if rest else None, temperature=temperature)
    _, _, grad = T.distill_loss(z, value, index, weight, **kw)
    h = 1e-4
    for i in range(len(z)):
        for u in range(V):
            def at(by):
                y = z.copy()
                y[i, u] += by
                return T.distill_loss(y, value, index, weight, **kw)[0]
            d = (8 * (at(h) - at(-h)) - (at(2 * h) - at(-2 * h))) / (12 * h)
            # four-point differences: h^4 / 30 = 3e-18 times the fifth derivative (below 1e3 here), and a few 1e-16
            # |loss| / h of cancellation, |loss| below 100
            assert abs(d - grad[i, u]) <= 2e-9, (i, u, d, grad[i, u])


def test_distill_of_every_token_is_the_divergence():
    z, value, index, weight, _ = rows(7, 9, 9, 3)
    loss, kl, grad = T.distill_loss(z, value, index, weight)
    teacher = np.empty_like(value)
    np.put_along_axis(teacher, index, value, 1)
    zt = torch.from_numpy(z).requires_grad_()
    each = torch.nn.functional.kl_div(torch.log_softmax(zt, 1), torch.log_softmax(torch.from_numpy(teacher), 1),
                                      reduction="none", log_target=True).sum(1)
    total = (each * torch.from_numpy(weight)).sum()
    total.backward()
    assert np.allclose(kl[weight != 0], each.detach().numpy()[weight != 0], atol=1e-12) and abs(loss - float(total)) < 1e-12
    assert np.allclose(grad, zt.grad.numpy(), atol=1e-12)


def test_distill_limits():
    z, value, index, weight, r = rows(6, 11, 4, 8)
    weight[:] = 1
    teacher = np.full((6, 11), -np.inf)
    np.put_along_axis(teacher, index, value, 1)
    # a student that agrees with the teacher has no divergence and no gradient
    student = teacher.copy()
    others = ~np.isfinite(teacher)
    student[others] = np.repeat(r - np.log(7), 7)
    loss, kl, grad = T.distill_loss(student, value, index, weight, rest=r)
    assert np.abs(kl).max() < 1e-12 and np.abs(grad).max() < 1e-12
    # rest -inf is no rest; entries out of range do not count; nothing that counts: left out
    a = T.distill_loss(z, value, index, weight, rest=np.full(6, -np.inf))
    b = T.distill_loss(z, value, index, weight)
    assert np.allclose(a[1], b[1]) and np.allclose(a[2], b[2])
    index[0] = -1
    index[1] = 11
    loss, kl, grad = T.distill_loss(z, value, index, weight)
    assert kl[0] == kl[1] == 0 and not grad[:2].any()
    # a student without probability where the teacher has some
    z[2, index[2, 0]] = -np.inf
    loss, kl, grad = T.distill_loss(z, value, index, weight)
    assert kl[2] == np.inf and np.isfinite(grad[2]).all()
