"""himuon_sample and himuon_top_logits on the paths that use their workspace (rows that blocks of one and two waves leave to a
second launch) on several streams and in graphs, a rest beside masked logits, and how many rows the comparisons with the
reference take in (MI355X only)."""
import math

import numpy as np
import pytest
import torch

from oracle import selection as S
from test_gpu_select import check_sample, rows_of

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.distill import top_logits  # noqa: E402
from tiled_newton_schulz_tile_amd.sampling import sample  # noqa: E402

DEV = "cuda"
INF = float("inf")


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def overflowing(N, V, seed):
    """fp32 rows for one (4200) or two (2100) waves each: equal ones, nearly flat ones and, one in four, ordinary ones."""
    logits, uniform = rows_of(N, V, torch.float32, seed)
    logits[0::4] = 0.5
    logits[1::4] *= 0.01
    logits[3::4] *= 0.1
    return logits, uniform


def run(logits, uniform, stream=None):
    return (*sample(logits, uniform, top_k=50, stream=stream), *sample(logits, uniform, min_p=1e-6, stream=stream),
            *sample(logits, uniform, top_k=200, top_p=0.9, stream=stream), *top_logits(logits, 50, stream=stream))


@pytest.mark.parametrize("N,V", [(4200, 1031), (2100, 9001)])
def test_rows_that_overflow_match_the_reference(N, V):
    _need_gpu()
    logits, uniform = overflowing(N, V, 3)
    some = torch.arange(0, N, N // 16 + 1)
    got = run(logits, uniform)
    for at, kw in ((0, dict(top_k=50)), (3, dict(min_p=1e-6)), (6, dict(top_k=200, top_p=0.9))):
        few = [x[some] for x in got[at:at + 3]]
        ties = int((some % 4 == 0).sum()) if "top_p" in kw else 0   # (of 200 equal logits 180 sum to 0.9 exactly)
        assert check_sample(logits[some], uniform[some], few, **kw) >= len(some) - 2 - ties
        assert ties == 0 or (few[2][(some % 4 == 0).to(DEV)].cpu() == torch.tensor(180 / V)).all()
    for n in some.tolist():
        want, lse = S.top_row(logits[n].double().cpu().numpy(), 50)
        assert (got[10][n].cpu().numpy() == want).all() and abs(float(got[11][n]) - lse) <= 2.0 ** -18


def test_two_calls_at_once_with_second_launches():
    """Calls on two streams share nothing, their row marks neither."""
    _need_gpu()
    sets = [overflowing(N, V, N) for N, V in ((4200, 1031), (2100, 9001))]
    want = [run(*a) for a in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[run(*a, s) for a, s in zip(sets, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        for x, y in zip(pair, want):
            assert all(torch.equal(a, b) for a, b in zip(x, y))


@pytest.mark.parametrize("N,V", [(4200, 1031), (2100, 9001)])
def test_second_launches_in_a_graph(N, V):
    _need_gpu()
    logits, uniform = overflowing(N, V, 5)
    run(logits, uniform)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(logits, uniform)
    for n in range(3):
        logits.copy_(logits.roll(n, 0) * (1 - 0.25 * n))   # (other rows overflow)
        uniform.mul_(0.7)
        want = run(logits, uniform)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


@pytest.mark.parametrize("N,V", [(12, 1100), (12, 40000), (12, 150001), (300, 9001), (2100, 9001), (4200, 1100)])
@pytest.mark.parametrize("mask", ["lowest", -1e30, -1e4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rest_of_rows_that_are_masked(N, V, mask, dtype):
    """A few ordinary logits among masked ones, at the row's beginning, its end or anywhere: while some of them are
    left the rest is theirs alone.  Its logarithm is fp32: the largest is rounded over T, a few powers are added.  A power
    is taken relative to a logit between the rest's largest and the row's (further than 2^-60 of its power, from the rest's
    largest itself): the distance, log2(e) / T and their product are each rounded at 2^-24, so the power is off by
    3 ln 2 2^-24 of the octaves that it is away, 3 2^-24 of the distance over T."""
    _need_gpu()
    g = torch.Generator().manual_seed(V)
    low = torch.tensor(torch.finfo(dtype).min if mask == "lowest" else mask, dtype=dtype).item()
    logits = torch.full((N, V), low, dtype=dtype)
    at = torch.stack([torch.randperm(V, generator=g)[:7] for _ in range(N)])
    at[1::3], at[2::3] = torch.arange(7), torch.arange(V - 7, V)
    few = (3 * torch.randn(N, 7, generator=g)).to(dtype)
    logits.scatter_(1, at, few)
    logits = logits.to(DEV)
    few = few.double().sort(1, descending=True).values
    for T in (1.0, 0.3, 20.0):
        for k in (1, 2, 6):
            got = top_logits(logits, k, temperature=T)
            others = torch.cat([few[:, k:] / T, torch.full((N, V - 7), float(low), dtype=torch.float64)[:, :1] / T], 1)
            others[:, -1] += math.log(V - 7)
            want = others.logsumexp(1)
            away = ((few[:, 0] - few[:, k]) / T).clamp(max=60 * math.log(2) + math.log(V))
            tol = 2.0 ** -22 * (others[:, 0].abs() + 4 + math.log(V)) + 3 * 2.0 ** -24 * away
            assert ((got.rest.double().cpu() - want).abs() <= tol).all(), (T, k)
            assert torch.equal(got.value.double().cpu(), few[:, :k])
        got = top_logits(logits, 7, temperature=T)   # (nothing is left but the masked ones)
        want = float(low) / T + math.log(V - 7)
        if abs(want) < 3.4e38:
            assert (abs(got.rest.double().cpu() - want) <= 2.0 ** -22 * (abs(float(low)) / T + 4 + math.log(V))).all(), T


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_largest_vocabulary_compares_its_rows(dtype):
    """Sharp rows of 2^20 tokens, whose borders are further apart than the sums' errors."""
    _need_gpu()
    V, N = 1 << 20, 6
    logits, uniform = rows_of(N, V, dtype, 4, 1.5)
    for kw in (dict(), dict(top_p=0.9), dict(top_p=0.3), dict(top_k=100), dict(min_p=1e-3), dict(top_k=1000, top_p=0.8)):
        assert check_sample(logits, uniform, sample(logits, uniform, **kw), **kw) >= N - 1, kw


@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (61, 7)])
@pytest.mark.parametrize("N,V", [(9, 97), (9, 33000), (130, 4099)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_compare_their_rows(N, V, pad, offset, dtype):
    _need_gpu()
    logits, uniform = rows_of(N, V, dtype, V + pad, pad=pad, offset=offset)
    for kw in (dict(), dict(top_k=30, top_p=0.95), dict(top_p=0.9), dict(min_p=0.02)):
        got = sample(logits, uniform, **kw)
        assert check_sample(logits[:9], uniform[:9], [x[:9] for x in got], **kw) >= 8
    masked = logits.clone()
    masked[:, V // 3:] = -INF
    for kw in (dict(), dict(top_k=9), dict(top_p=0.9), dict(min_p=0.01), dict(temperature=0.0)):
        got = sample(masked, uniform, **kw)
        assert check_sample(masked[:9], uniform[:9], [x[:9] for x in got], **kw) >= 8
        assert (got.token < V // 3).all()


@pytest.mark.parametrize("N,V", [(12, 40000), (300, 9001), (1100, 9001), (2100, 9001), (4200, 9001), (300, 600)])
@pytest.mark.parametrize("low", [-60.0, -20.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rest_of_rows_whose_largest_come_late(N, V, low, dtype):
    """Every wave begins with logits far below the others'.  The rest's own largest is about as large as the row's, so its
    powers have no distance to speak of: rounding it over T, a thread's V / 256 terms (at least) and a join of ten levels
    are all."""
    _need_gpu()
    g = torch.Generator().manual_seed(V)
    z = torch.randn(N, V, generator=g)
    turn = 256 * (4 if dtype is torch.float32 else 8)
    z[:, (torch.arange(V) // turn) % 5 != 4] += low
    z[:, -V // 8:] -= torch.where(z[:, -V // 8:] < low / 2, low, 0.0)
    logits = z.to(dtype).to(DEV)
    z = logits.double().cpu().sort(1, descending=True).values
    for T in (1.0, 0.5):
        for k in (1, 5, 60):
            got = top_logits(logits, k, temperature=T)
            want = (z[:, k:] / T).logsumexp(1)
            tol = 2.0 ** -22 * (z[:, k].abs() / T + 2 + math.log(V)) + 2.0 ** -24 * (V / 256 + 24)
            tol += 3 * 2.0 ** -24 * (z[:, 0] - z[:, k]) / T
            error = (got.rest.double().cpu() - want).abs()
            assert (error <= tol).all(), (T, k, float((error / tol).max()))
            assert torch.equal(got.value.double().cpu(), z[:, :k])


@pytest.mark.parametrize("N,V", [(12, 40000), (300, 9001), (1100, 9001), (2100, 9001), (4200, 9001), (300, 600)])
@pytest.mark.parametrize("low", [-60.0, -20.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_log_probabilities_of_rows_whose_largest_come_late(N, V, low, dtype):
    """Every wave begins with logits far below the others'; the tolerances are those of other rows."""
    _need_gpu()
    g = torch.Generator().manual_seed(V)
    z = torch.randn(N, V, generator=g)
    turn = 256 * (4 if dtype is torch.float32 else 8)
    z[:, (torch.arange(V) // turn) % 5 != 4] += low
    z[:, -V // 8:] -= torch.where(z[:, -V // 8:] < low / 2, low, 0.0)
    logits, uniform = z.to(dtype).to(DEV), torch.rand(N, generator=g).to(DEV)
    some = torch.arange(0, N, N // 12 + 1)
    for kw in (dict(top_k=1), dict(top_k=5), dict(top_k=60), dict(min_p=0.9), dict(min_p=0.5), dict(top_k=40, top_p=0.8)):
        got = sample(logits, uniform, **kw)
        assert check_sample(logits[some], uniform[some], [x[some] for x in got], **kw) >= len(some) - 1


@pytest.mark.parametrize("N,V", [(12, 40000), (300, 9001), (1100, 9001), (2100, 9001), (4200, 9001)])
@pytest.mark.parametrize("low", [-60.0, -30.0])
def test_log_probabilities_beside_a_few_late_logits(N, V, low):
    """The same with four large logits at the row's end, one of which is kept: the others' powers are nearly all that
    the log probability has besides."""
    _need_gpu()
    g = torch.Generator().manual_seed(N)
    z = torch.randn(N, V, generator=g) + low
    z[:, [V - 700, V - 300, V - 9, V - 2]] = torch.rand(N, 4, generator=g)
    logits, uniform = z.to(DEV), torch.rand(N, generator=g).to(DEV)
    some = torch.arange(0, N, N // 100 + 1)
    for kw in (dict(top_k=1), dict(top_k=2), dict(min_p=0.95)):
        got = sample(logits, uniform, **kw)
        assert check_sample(logits[some], uniform[some], [x[some] for x in got], **kw) >= len(some) - 1
