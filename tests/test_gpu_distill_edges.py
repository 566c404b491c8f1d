"""himuon_distill_loss where the teacher's rest is all that it has, of any size, or almost nothing (MI355X only)."""
import numpy as np
import pytest
import torch

from oracle import training as T
from test_gpu_distill import make

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.distill import distill_loss  # noqa: E402

INF = float("inf")
# spans, and rows in blocks of one and of more waves
SIZES = [(3, 70001), (3, 700), (140, 1031), (140, 20000)]


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("N,V", SIZES)
@pytest.mark.parametrize("rest", [-1e12, 1e12, -3e30, 2e38, -3.3e38, 1e4])
@pytest.mark.parametrize("temperature", [1.7, 0.3, 1.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_rest_alone(N, V, rest, temperature, dtype):
    """A teacher whose entries are all -inf or far below its rest: the divergence is -log p_rest whatever the rest's size.
    fp32's error: a log probability's as in test_gpu_distill, for two of them; a gradient is weight / T times
    probabilities, each within twice its logarithm's error."""
    _need_gpu()
    logits, value, index, weight, r = make(N, V, 12, dtype, 9, masked=0.0, temperature=temperature)
    value.fill_(-INF)
    if rest > 0:
        value[1::2] = 5.0
    r.fill_(rest)
    weight[:] = 1.0
    weight[4:] = 0.0
    got = distill_loss(logits, value, index, weight, rest=r, temperature=temperature)
    fwd = distill_loss(logits, value, index, weight, rest=r, temperature=temperature, dlogits=False)
    host = [x.double().cpu().numpy() for x in (logits, value)] + [index.cpu().numpy()]
    loss, kl, grad = T.distill_loss(*host, weight.double().cpu().numpy(), r.double().cpu().numpy(), temperature)
    live = min(N, 4)
    assert (kl[:live] > 1e-3).all()
    y = host[0][:live] / temperature
    tol = 2 * (2.0 ** -22 * (1 + np.abs(y - y.max(1, keepdims=True)).max()) + 2.0 ** -24 * (V / 512 + 24))
    for k in (got.kl, fwd.kl):
        assert (np.abs(k.double().cpu().numpy() - kl)[:live] <= tol + 2.0 ** -24 * kl[:live]).all()
    half = 2.0 ** -8 if dtype is torch.bfloat16 else 0.0
    p = np.exp(y - y.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    others = np.ones_like(p, bool)
    np.put_along_axis(others, host[2][:live], False, 1)
    p_rest = (p * others).sum(1, keepdims=True)
    size = (p + p / p_rest) / temperature
    error = np.abs(got.dlogits.double().cpu().numpy() - grad)[:live]
    assert (error <= 2 * tol * size + half * np.abs(grad[:live]) + 1e-37).all()


@pytest.mark.parametrize("N,V", SIZES)
@pytest.mark.parametrize("below", [60.0, 110.0, 600.0])
def test_a_small_rest_where_the_student_has_none(N, V, below):
    """A rest of any probability that is a number in 64 bits has an infinite divergence from a student without one, as a
    named token has; the gradient is finite.  One of no probability has none."""
    _need_gpu()
    logits, value, index, weight, r = make(N, V, 12, torch.float32, 9, masked=0.0)
    named = torch.zeros(N, V, dtype=torch.bool, device="cuda").scatter_(1, index, True)
    logits.masked_fill_(~named, -INF)
    value[:, 11] = value[:, 0] - below
    r[:] = value[:, 0] - below
    r[2] = -INF
    for grad in (True, False):
        got = distill_loss(logits, value, index, weight, rest=r, dlogits=grad)
        assert (got.kl[:2] == INF).all() and torch.isfinite(got.kl[2])
        assert (got.kl[3:] == INF).all() and (not grad or torch.isfinite(got.dlogits).all())
    logits[0, index[0, 11]], r[0] = -INF, -INF    # (the named one)
    assert distill_loss(logits, value, index, weight, rest=r).kl[0] == INF
