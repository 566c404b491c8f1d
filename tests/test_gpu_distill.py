"""himuon_distill_loss against the fp64 reference (MI355X only): vocabularies from one token to
2^20, entries from one to 1024, named twice, out of range or of -inf, with and without the rest,
students that give the rest almost nothing, row strides, unaligned starts, rows left out with
garbage in them, in-place gradients, other streams and graph replays."""
import numpy as np
import pytest
import torch

from oracle import training as T

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.distill import distill_loss  # noqa: E402

DEV = "cuda"
INF = float("inf")


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(N, V, k, dtype, seed, pad=0, offset=0, masked=0.2, temperature=1.0, spread=2.5, value_dtype=None, top_pad=0):
    """Device inputs: student logits ((N, V) view of rows V + pad apart, `offset` elements into memory), and the entries
    of a teacher that is not far from it."""
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(N, V, generator=g) * spread
    t = (t + 0.3 * torch.randn(N, V, generator=g) ** 3).to(value_dtype or dtype)
    z = (0.8 * t.float() + 0.5 * torch.randn(N, V, generator=g)).to(dtype)
    buf = torch.full((offset + N * (V + pad),), float("nan"), dtype=dtype, device=DEV)
    logits = buf[offset:].view(N, V + pad)[:, :V]
    logits.copy_(z)
    v, i = t.float().topk(k, dim=1)
    others = t.double().scatter(1, i, -INF) / temperature
    rest = torch.logsumexp(others, 1).float()
    value = torch.zeros(N, k + top_pad, dtype=t.dtype, device=DEV)[:, :k]
    index = torch.zeros(N, k + top_pad, dtype=torch.int64, device=DEV)[:, :k]
    value.copy_(v)
    index.copy_(i)
    weight = torch.rand(N, generator=g) + 0.1
    weight[torch.rand(N, generator=g) < masked] = 0
    return logits, value, index, weight.to(DEV), rest.to(DEV)


def check(args, got, rest=True, temperature=1.0, grad_scale=1.0):
    """Outputs within the error of the fp32 formulas.  A token's log probability: the distance to the largest logit is
    rounded at 2^-24 of its value, a thread sums V / 512 terms (at least) one after the other and a join of nine levels
    follows; exp2, log2 and the products are within 2^-22 together.  The teacher's have k / 64 terms a lane instead, and
    value / temperature is rounded at 2^-23 of itself before the distance is taken.  A probability's relative error is
    that of its logarithm twice (its own and the sum's).  The divergence adds k / 64 + 8 rounded terms; a gradient entry
    carries the errors of its probabilities times their size, and its type's rounding."""
    logits, value, index, weight, r = args
    z, v, w = (x.double().cpu().numpy() for x in (logits, value, weight))
    i = index.cpu().numpy()
    r = r.double().cpu().numpy() if rest else None
    loss, kl, grad = T.distill_loss(z, v, i, w, rest=r, temperature=temperature, grad_scale=grad_scale)
    N, V = z.shape
    k = i.shape[1]
    gkl = got.kl.double().cpu().numpy()
    gz = None if got.dlogits is None else got.dlogits.double().cpu().numpy()
    half = 2.0 ** -8 if logits.dtype == torch.bfloat16 else 0.0
    total = 0.0
    for n in range(N):
        counts = (i[n] >= 0) & (i[n] < V)
        x = v[n][counts] / temperature
        if rest:
            x = np.append(x, r[n])
        if w[n] == 0 or not (x > -np.inf).any():
            assert gkl[n] == 0 and (gz is None or not gz[n].any())
            continue
        y = z[n] / temperature
        with np.errstate(all="ignore"):
            lp = y - y.max() - np.log(np.exp(y - y.max()).sum())
            lq = x - x.max() - np.log(np.exp(x - x.max()).sum())
            q, p = np.exp(lq), np.exp(lp)
            s = 2.0 ** -22 * (1 + np.where(np.isfinite(lp), np.abs(lp), 0)) + 2.0 ** -24 * (V / 512 + 24)
            t = (2.0 ** -22 * (1 + np.where(q > 0, np.abs(lq), 0)) + 2.0 ** -24 * (k / 64 + 24)
                 + 2.0 ** -22 * np.abs(x[np.isfinite(x)]).max())
            others = np.ones(V, bool)
            others[i[n][counts]] = False
            lps, ss = lp[i[n][counts]], s[i[n][counts]]
            share, pull = np.zeros(V), np.zeros(V)
            if rest:
                top = y[others].max() if others.any() else -np.inf
                e = np.exp(y[others] - top) if np.isfinite(top) else np.zeros(others.sum())
                lps = np.append(lps, top - y.max() + np.log(e.sum()) + lp.max())
                ss = np.append(ss, s[others].min() if others.any() else 0)
                if e.sum() > 0:
                    share[others] = q[-1] * e / e.sum()
            on = q > 0
            gap = np.abs(lq[on] - lps[on])
            tol = (q[on] * (ss[on] + t[on] + gap * 2 * t[on])).sum() + 2.0 ** -24 * (k / 64 + 8) * (q[on] * gap).sum()
        if not np.isfinite(kl[n]):
            assert gkl[n] == kl[n]
        else:
            assert abs(gkl[n] - kl[n]) <= tol, (n, gkl[n], kl[n], tol)
        total += w[n] * tol + 2.0 ** -22 * abs(w[n] * kl[n])
        if gz is None:
            continue
        for a, b in zip(i[n][counts], q):
            pull[a] += b
        c = abs(grad_scale * w[n] / temperature)
        bound = c * (p * (2 * s + 2.0 ** -20) + pull * (2 * t.max() + 2.0 ** -20)
                     + share * (4 * s + 2 * t.max() + 2.0 ** -20)) + half * np.abs(grad[n]) + 1e-37
        off = np.abs(gz[n] - grad[n]) > bound
        assert not off.any(), (n, np.flatnonzero(off)[:5], gz[n][off][:5], grad[n][off][:5], bound[off][:5])
    if np.isfinite(loss):
        assert abs(float(got.loss) - loss) <= total + 1e-30
    else:
        assert float(got.loss) == loss


def both(args, rest=True, **kw):
    logits, value, index, weight, r = args
    r = r if rest else None
    got = distill_loss(logits, value, index, weight, rest=r, **kw)
    check(args, got, rest, **kw)
    fwd = distill_loss(logits, value, index, weight, rest=r, dlogits=False, **kw)
    assert fwd.dlogits is None
    check(args, fwd, rest, **kw)
    return got


@pytest.mark.parametrize("V", [1, 2, 7, 9, 64, 257, 1000, 4104, 8195, 16384, 32003, 50257, 131073, 150001])
@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_distill_matches_reference(V, rest, dtype):
    _need_gpu()
    both(make(5 if V > 10000 else 21, V, min(V, 20), dtype, V, temperature=0.8), rest, temperature=0.8, grad_scale=3.0)


@pytest.mark.parametrize("V", [255, 1024, 2049, 4097, 8192, 16385, 32768, 50257, 65537, 131071, 131080, 150001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_distill_many_rows(V, dtype):
    """More rows than the path that cuts rows into spans takes: every size of row that a block holds in registers, and
    rows past it; forward alone, with the gradient, and in place."""
    _need_gpu()
    args = make(131, V, 33, dtype, V, pad=1, masked=0.93)
    args[3][130] = 0.5
    got = both(args, V % 2 == 0, temperature=1.3)
    z = args[0].clone()
    again = distill_loss(z, *args[1:4], rest=args[4] if V % 2 == 0 else None, temperature=1.3, dlogits=z)
    assert again.dlogits is z and torch.equal(z, got.dlogits) and torch.equal(again.kl, got.kl)


@pytest.mark.parametrize("k", [1, 2, 63, 64, 65, 200, 1000, 1024])
@pytest.mark.parametrize("N,V", [(3, 1024), (3, 40000), (140, 1031), (140, 20000)])
def test_distill_entries(N, V, k):
    _need_gpu()
    both(make(N, V, k, torch.bfloat16, k, masked=0.8 if N > 100 else 0.0, value_dtype=torch.float32, top_pad=k % 3))


@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 5), (61, 7)])
@pytest.mark.parametrize("N,V", [(9, 97), (9, 33000), (130, 4099)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_distill_strides_and_alignments(N, V, pad, offset, dtype):
    _need_gpu()
    args = make(N, V, 17, dtype, V + pad, pad=pad, offset=offset, masked=0.5, top_pad=pad)
    logits, value, index, weight, rest = args
    buf = torch.full((N, V + 2 * pad + 1), 7.0, dtype=dtype, device=DEV)
    got = distill_loss(logits, value, index, weight, rest=rest, dlogits=buf[:, pad:pad + V])
    check(args, got)
    assert (buf[:, :pad] == 7).all() and (buf[:, pad + V:] == 7).all()   # nothing beside the rows


@pytest.mark.parametrize("N,V", [(6, 600), (6, 33001), (6, 140001), (140, 600), (140, 9001), (140, 140001)])
@pytest.mark.parametrize("rest", [True, False])
def test_distill_entries_that_repeat_or_do_not_count(N, V, rest):
    _need_gpu()
    args = make(N, V, 40, torch.float32, 5, masked=0.95 if N > 100 else 0.0)
    logits, value, index, weight, r = args
    weight[:6] = 0.5
    index[0, 3:] = -1                       # fewer entries
    index[1, 1::2] = index[1, 0::2]         # every token twice
    index[2, :] = index[2, 0]               # one token, forty times
    index[3, 0], index[3, 1] = V, -(1 << 40)
    index[3, 2] = (1 << 32) + 5             # not token 5
    value[4, 7:] = -INF
    index[5, 20:] = V - 1                   # the row's last token, many times
    got = both(args, rest)
    assert torch.equal(distill_loss(logits, value, index, weight, rest=r if rest else None).dlogits, got.dlogits)
    # a teacher without anything: left out (with a rest it still has that)
    index[0] = -1
    value[1] = -INF
    r[0] = -INF
    got = both(args, rest)
    assert got.kl[0] == 0 and not got.dlogits[0].any() and (rest or not got.dlogits[1].any())


@pytest.mark.parametrize("N,V", [(7, 700), (7, 40000), (140, 700), (140, 20000), (140, 140001)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_distill_rests_of_all_sizes(N, V, dtype):
    """Students that give the tokens which the teacher did not name almost nothing, nothing, or almost everything."""
    _need_gpu()
    args = make(N, V, 12, dtype, 9, masked=0.95 if N > 100 else 0.0)
    logits, value, index, weight, rest = args
    weight[:7] = 1.0
    named = torch.zeros(N, V, dtype=torch.bool, device=DEV).scatter_(1, index, True)
    for n, by in enumerate((-30.0, -80.0, -200.0, 60.0, 300.0)):
        logits[n] += torch.where(named[n], 0.0, by).to(dtype)
    logits[5].masked_fill_(~named[5], -INF)     # nothing: an infinite divergence, a finite gradient
    logits[6].masked_fill_(~named[6], torch.finfo(dtype).min)
    got = both(args)
    assert got.kl[5] == INF and torch.isfinite(got.dlogits).all()
    rest[5] = -INF                              # unless the teacher has nothing there, too
    assert torch.isfinite(both(args).kl[:6]).all()
    both(args, False)


@pytest.mark.parametrize("N,V", [(8, 513), (8, 40000), (140, 513), (140, 30000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_distill_rows_left_out_hide_their_contents(N, V, dtype):
    _need_gpu()
    args = make(N, V, 9, dtype, 4, masked=0.0)
    logits, value, index, weight, rest = args
    off = [1, 2, 4]
    weight[off] = 0
    logits[1], value[2], rest[4] = float("nan"), float("nan"), INF
    index[4] = 1 << 50
    got = distill_loss(logits, value, index, weight, rest=rest)
    assert not got.kl[off].any() and not got.dlogits[off].any() and torch.isfinite(got.loss)
    keep = [n for n in range(N) if n not in off]
    part = distill_loss(*(t[keep].contiguous() for t in args[:4]), rest=rest[keep].contiguous())
    assert torch.equal(part.kl, got.kl[keep]) and torch.equal(part.dlogits, got.dlogits[keep])
    weight.zero_()
    got = distill_loss(logits, value, index, weight, rest=rest)
    assert got.loss == 0 and not got.kl.any() and not got.dlogits.any()


@pytest.mark.parametrize("N,V", [(9, 600), (9, 33001), (140, 600), (140, 33001), (140, 140001)])
@pytest.mark.parametrize("rest", [True, False])
def test_distill_infinite_and_nan(N, V, rest):
    _need_gpu()
    args = make(N, V, 16, torch.float32, 8, masked=0.0)
    logits, value, index, weight, r = args
    n_rest = r if rest else None
    logits[0, index[0, 3]] = -INF
    got = distill_loss(logits, value, index, weight, rest=n_rest)
    assert got.kl[0] == INF and torch.isfinite(got.dlogits).all() and got.loss == INF
    logits[0, index[0, 3]] = 0
    want = distill_loss(logits, value, index, weight, rest=n_rest)
    logits[1, V - 1] = float("nan")
    logits[2, 0] = INF
    logits[3] = -INF
    logits[4, index[4, 0]] = float("nan")
    value[5, 2] = float("nan")
    value[6, 2] = INF
    bad = list(range(1, 7))
    if rest:
        r[7], r[8] = float("nan"), INF
        bad += [7, 8]
    got = distill_loss(logits, value, index, weight, rest=n_rest)
    assert torch.isnan(got.kl[bad]).all() and torch.isnan(got.dlogits[bad]).any(1).all() and torch.isnan(got.loss)
    good = [n for n in range(N) if n not in bad]
    assert torch.equal(got.kl[good], want.kl[good]) and torch.equal(got.dlogits[good], want.dlogits[good])


def test_distill_gradient_is_the_difference_quotient():
    """The gradient from the kernel (fp32) against central differences of the reference's loss in fp64."""
    _need_gpu()
    args = make(5, 37, 6, torch.float32, 11, masked=0.0, temperature=1.3)
    logits, value, index, weight, rest = args
    got = distill_loss(logits, value, index, weight, rest=rest, temperature=1.3).dlogits.double().cpu().numpy()
    z, v, w, r = (x.double().cpu().numpy() for x in (logits, value, weight, rest))
    h = 1e-4
    for n in range(5):
        for u in range(37):
            zp, zm = z.copy(), z.copy()
            zp[n, u] += h
            zm[n, u] -= h
            d = (T.distill_loss(zp, v, index.cpu().numpy(), w, rest=r, temperature=1.3)[0]
                 - T.distill_loss(zm, v, index.cpu().numpy(), w, rest=r, temperature=1.3)[0]) / (2 * h)
            # h^2 / 6 third derivatives (a few units), and the kernel's fp32
            assert abs(d - got[n, u]) <= 1e-7 + 2e-5 * abs(d) + 1e-6


@pytest.mark.parametrize("N", [2, 131])
@pytest.mark.parametrize("V", [1 << 20, (1 << 20) - 3])
def test_distill_largest_vocabulary(N, V):
    _need_gpu()
    args = make(3, V, 1024, torch.bfloat16, 2, masked=0.0)
    args = tuple(t.repeat(-(-N // 3), *[1] * (t.dim() - 1))[:N].contiguous() for t in args)
    args[3][3:] = 0
    both(args)
    with pytest.raises(hm.HiMuonError):
        distill_loss(torch.zeros(1, (1 << 20) + 1, device=DEV), *(t[:1] for t in args[1:4]))


def test_distill_no_rows_and_many_rows():
    _need_gpu()
    e = torch.zeros(0, device=DEV)
    got = distill_loss(torch.zeros(0, 100, device=DEV), torch.zeros(0, 5, device=DEV),
                       torch.zeros(0, 5, dtype=torch.int64, device=DEV), e)
    assert got.loss == 0 and got.kl.shape == (0,) and got.dlogits.shape == (0, 100)
    N, V, k = (1 << 21) + 3, 9, 2                       # more rows than a launch holds
    g = torch.Generator(device=DEV).manual_seed(1)
    z = torch.randn(N, V, device=DEV, generator=g).bfloat16()
    value = torch.randn(N, k, device=DEV, generator=g)
    index = torch.randint(-1, V, (N, k), device=DEV, generator=g)
    weight, rest = torch.rand(N, device=DEV, generator=g), torch.randn(N, device=DEV, generator=g)
    got = distill_loss(z, value, index, weight, rest=rest)
    for a in (slice(N - 300, N), slice(1000, 1300)):
        one = distill_loss(z[a], value[a], index[a], weight[a], rest=rest[a])
        assert torch.equal(one.kl, got.kl[a]) and torch.equal(one.dlogits, got.dlogits[a])
    want = float((weight.double() * got.kl.double()).sum())
    assert abs(float(got.loss) - want) <= 2.0 ** -23 * abs(want)


def test_distill_offsets_past_32_bits():
    """Rows whose element offset does not fit 32 bits (a row stride into a large buffer)."""
    _need_gpu()
    N, V, ld = 5, 1003, (1 << 30) + 7
    buf = torch.zeros((N - 1) * ld + V, dtype=torch.bfloat16, device=DEV)
    view = torch.as_strided(buf, (N, V), (ld, 1))
    small, *args = make(N, V, 6, torch.bfloat16, 3, masked=0.0)
    view.copy_(small)
    want = distill_loss(small, *args[:3], rest=args[3])
    got = distill_loss(view, *args[:3], rest=args[3], dlogits=view)
    assert torch.equal(got.kl, want.kl) and torch.equal(got.dlogits, want.dlogits)


@pytest.mark.parametrize("N,V", [(64, 5001), (140, 5001)])
def test_distill_on_another_stream_and_in_a_graph(N, V):
    _need_gpu()
    logits, value, index, weight, rest = make(N, V, 30, torch.bfloat16, 21)
    want = distill_loss(logits, value, index, weight, rest=rest)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = distill_loss(logits, value, index, weight, rest=rest, stream=s)
    s.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = distill_loss(logits, value, index, weight, rest=rest)
    for n in range(3):
        logits.mul_(1 + 0.25 * n)
        weight.add_(0.01 * n)
        want = distill_loss(logits, value, index, weight, rest=rest)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(held, want):
            assert torch.equal(x, y)


def test_distill_two_calls_at_once():
    """Calls on two streams share nothing."""
    _need_gpu()
    sets = [make(N, V, 30, torch.bfloat16, N) for N, V in ((64, 50001), (100, 20001))]
    want = [distill_loss(*a[:4], rest=a[4]) for a in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[distill_loss(*a[:4], rest=a[4], stream=s) for a, s in zip(sets, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        for x, y in zip(pair, want):
            assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_distill_wrapper_refusals():
    _need_gpu()
    z, value, index, weight, rest = make(4, 10, 3, torch.float32, 1)
    ok = dict(logits=z, value=value, index=index, weight=weight, rest=rest)
    distill_loss(**ok)
    for bad in [dict(logits=z.t()), dict(logits=z.half()), dict(logits=z[0]), dict(logits=z.cpu()), dict(value=value[:3]),
                dict(value=value.half()), dict(value=value.t()), dict(index=index.int()), dict(index=index[:, :2]),
                dict(value=value[:, :0], index=index[:, :0]), dict(weight=weight[:3]), dict(weight=None),
                dict(rest=rest.double()), dict(rest=rest[:1]), dict(index=index.cpu()),
                dict(index=torch.zeros(4, 6, dtype=torch.int64, device=DEV)[:, :3]),
                dict(dlogits=torch.empty(4, 11, device=DEV)), dict(dlogits=torch.empty(4, 10, device=DEV).bfloat16())]:
        with pytest.raises(ValueError):
            distill_loss(**(ok | bad))
    for bad in [dict(temperature=0.0), dict(temperature=INF), dict(temperature=float("nan")), dict(grad_scale=INF),
                dict(value=torch.zeros(4, 1025, device=DEV), index=torch.zeros(4, 1025, dtype=torch.int64, device=DEV))]:
        with pytest.raises(hm.HiMuonError):
            distill_loss(**(ok | bad))
