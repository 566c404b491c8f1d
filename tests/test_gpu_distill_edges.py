"""himuon_distill_loss where the teacher's rest is all that it has, of any size, or almost nothing, rows that are cut into
spans on several streams and in graphs, and the largest use of LDS (MI355X only)."""
import numpy as np
import pytest
import torch

from oracle import training as T
from test_gpu_distill import both, make

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


FEW = [(8, 131077), (31, 70001)]   # rows that are cut into spans, with a gradient and without


def test_two_calls_at_once_with_spans():
    """Calls on two streams share nothing: tickets, spans and entries neither."""
    _need_gpu()
    sets = [make(N, V, 30, torch.bfloat16, N) for N, V in FEW]

    def run(a, s=None):
        return [x for g in (True, False) for x in distill_loss(*a[:4], rest=a[4], dlogits=g, stream=s) if x is not None]

    for logits, value, *_ in sets:
        p = hm.himuon_distill(rows=logits.shape[0], vocab=logits.shape[1], ld_logits=logits.shape[1],
                              ld_dlogits=logits.shape[1], ld_top=30, k=30, dtype=hm.BF16, value_dtype=hm.BF16, temperature=1.0,
                              grad_scale=1.0, logits=16, dlogits=32)
        assert hm.himuon_distill_workspace(p) > 0
    want = [run(a) for a in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[run(a, s) for a, s in zip(sets, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        for x, y in zip(pair, want):
            assert all(torch.equal(a, b) for a, b in zip(x, y))


@pytest.mark.parametrize("N,V", FEW)
@pytest.mark.parametrize("grad", [True, False])
def test_spans_on_another_stream_and_in_a_graph(N, V, grad):
    _need_gpu()
    logits, value, index, weight, rest = make(N, V, 30, torch.bfloat16, 21)

    def run(stream=None):
        return [x for x in distill_loss(logits, value, index, weight, rest=rest, dlogits=grad, stream=stream) if x is not None]

    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = run(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for n in range(3):
        logits.mul_(1 + 0.25 * n)
        weight.add_(0.01 * n)
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


@pytest.mark.parametrize("N", [33, 70])
@pytest.mark.parametrize("V", [1 << 20, (1 << 20) - 3])
def test_largest_vocabulary_in_fp32(N, V):
    """The largest bitmap of named tokens (a bit a logit beyond the held ones) and the most entries, in LDS together."""
    _need_gpu()
    args = make(2, V, 1024, torch.float32, 2, masked=0.0)
    args = tuple(t.repeat(-(-N // 2), *[1] * (t.dim() - 1))[:N].contiguous() for t in args)
    args[2][1, 3::5] = torch.arange(V - len(args[2][1, 3::5]), V)   # (tokens of the row's last vectors)
    args[3][2:] = 0
    both(args)
