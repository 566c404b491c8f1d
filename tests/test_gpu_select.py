"""himuon_sample and himuon_top_logits against the fp64 reference (MI355X only): vocabularies from
one token to 2^20, sharp and flat rows, rows of equal logits, every filter alone and together, one
setting for all rows or one a row, masks, bad rows, row strides, unaligned starts, other streams and
graph replays."""
import math

import numpy as np
import pytest
import torch

from oracle import selection as S

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.distill import top_logits  # noqa: E402
from tiled_newton_schulz_tile_amd.sampling import sample  # noqa: E402

DEV = "cuda"
INF = float("inf")
NAN = float("nan")


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rows_of(N, V, dtype, seed, scale=1.0, pad=0, offset=0):
    """(N, V) view of device rows V + pad apart, `offset` elements into memory, NaN around them."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, V, generator=g)
    z = ((2.5 * z + 0.35 * z ** 3) * scale).to(dtype)
    buf = torch.full((offset + N * (V + pad),), NAN, dtype=dtype, device=DEV)
    logits = buf[offset:].view(N, V + pad)[:, :V]
    logits.copy_(z)
    return logits, torch.rand(N, generator=g).to(DEV)


def setting(x, n):
    return x[n].item() if torch.is_tensor(x) else x


def check_sample(logits, uniform, got, **kw):
    """Tokens are the reference's.  A border may fall the other way only where it is as near as the error of the sums:
    2^-44 for the draw (V terms within 2^-51, added in fp64), and V 2^-(mass bits + 1), mass bits = 62 - bits of V, for
    top_p's, which is taken from sums of multiples of 2^-mass bits.  The log probability and the kept share are fp64
    rounded to fp32, but for the sum over all tokens: where no border hangs on it, those below the filters' bound (none of
    them is the largest) enter it in fp32.  Such a power is within 2^-23 of itself, and an exponent of x is rounded
    when the distance is taken and when it is multiplied, 2^-24 |x| each, so the power by ln 2 2^-23 |x|; eight are
    added at a time (3 levels of 2^-24).  top_p's border shifted by one token moves the kept share by that token, so
    rows with such a border are not compared."""
    z = logits.double().cpu().numpy()
    u = uniform.cpu().numpy()
    V = z.shape[1]
    near = V * 2.0 ** -(63 - V.bit_length())
    compared = 0
    token, logp, kept = (x.double().cpu().numpy() for x in got)
    for n in range(len(z)):
        want = S.sample_row(z[n], u[n], **{k: setting(x, n) for k, x in kw.items()})
        if want[0] < 0:
            assert token[n] == -1 and np.isnan(logp[n]) and np.isnan(kept[n])
            continue
        if want[3] <= 2.0 ** -44 or want[4] <= near:
            continue
        compared += 1
        assert token[n] == want[0], (n, token[n], want)
        x = (z[n] - z[n].max()) / (setting(kw.get("temperature", 1.0), n) or 1.0) / math.log(2)
        x = np.delete(x, x.argmax())
        x = x[x > -100]
        e = np.exp2(x)
        near32 = (e * (2.0 ** -23 + 3 * 2.0 ** -24 + math.log(2) * 2.0 ** -23 * np.abs(x))).sum() / (1 + e.sum())
        assert abs(logp[n] - want[1]) <= 2.0 ** -23 * abs(want[1]) + 2.0 ** -40 + near32, (n, logp[n], want)
        assert abs(kept[n] - want[2]) <= (2.0 ** -23 + near32) * want[2], (n, kept[n], want)
    return compared


FILTERS = [dict(), dict(top_k=1), dict(top_k=50), dict(top_k=700), dict(top_p=0.3), dict(top_p=0.95), dict(top_p=0.9999),
           dict(min_p=0.1), dict(min_p=1e-4), dict(top_k=50, top_p=0.9), dict(top_k=3000, top_p=0.8, min_p=0.01),
           dict(top_k=20, min_p=0.05), dict(top_p=0.9, min_p=0.02), dict(top_p=0.0), dict(min_p=1.0)]


@pytest.mark.parametrize("V", [1, 2, 7, 64, 257, 1000, 2048, 4104, 8195, 16384, 32003, 50257, 131072, 131075, 150001])
@pytest.mark.parametrize("scale", [1.0, 0.15])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_matches_reference(V, scale, dtype):
    _need_gpu()
    N = 4 if V > 10000 else 16
    logits, uniform = rows_of(N, V, dtype, V, scale)
    compared = 0
    for kw in FILTERS:
        kw = dict(temperature=0.8, **kw)
        compared += check_sample(logits, uniform, sample(logits, uniform, **kw), **kw)
    assert compared >= 0.9 * N * len(FILTERS)


def settings_of(N, seed):
    g = torch.Generator().manual_seed(seed)
    pick = lambda *x: torch.tensor(x)[torch.randint(0, len(x), (N,), generator=g)].to(DEV)  # noqa: E731
    return dict(temperature=pick(0.0, 0.3, 1.0, 2.0), top_k=pick(0, 0, 1, 40, 1000, 1 << 30).int(),
                top_p=pick(1.0, 1.0, 0.5, 0.9, 0.99, 0.0), min_p=pick(0.0, 0.0, 0.001, 0.05, 2.0))


@pytest.mark.parametrize("N,V", [(200, 300), (300, 5003), (150, 32003), (70, 131072), (140, 131075)])
@pytest.mark.parametrize("scale", [1.0, 0.1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_settings_of_their_own(N, V, scale, dtype):
    """Many rows, each with its own settings; each row is what a call with its numbers for all rows gives."""
    _need_gpu()
    logits, uniform = rows_of(N, V, dtype, N + V, scale, pad=3, offset=1)
    kw = settings_of(N, V)
    got = sample(logits, uniform, **kw)
    assert check_sample(logits[:64], uniform[:64], [x[:64] for x in got], **{k: x[:64] for k, x in kw.items()}) >= 50
    for n in (0, 1, N - 1):
        one = sample(logits[n:n + 1], uniform[n:n + 1], **{k: x[n].item() for k, x in kw.items()})
        assert all(torch.equal(a, b[n:n + 1]) for a, b in zip(one, got))
    again = sample(logits, uniform, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("V,n", [(9, 4096), (500, 8192), (20000, 4096)])
@pytest.mark.parametrize("kw", [dict(), dict(top_k=5), dict(top_p=0.7), dict(min_p=0.3)])
def test_sample_shares(V, n, kw):
    """A grid of uniforms over one row gives every kept token its share to within one draw of each end."""
    _need_gpu()
    logits, _ = rows_of(1, V, torch.float32, 3)
    u = (torch.arange(n, device=DEV) + 0.5) / n
    got = sample(logits.expand(n, V).contiguous(), u, **kw)
    count = torch.bincount(got.token, minlength=V).cpu().double().numpy()
    row = logits[0].double().cpu().numpy()
    p = np.exp(row - row.max())
    line = S.order(row)
    keep = len(line)
    if "top_k" in kw:
        keep = kw["top_k"]
    if "top_p" in kw:
        keep = int((np.cumsum(p[line]) < kw["top_p"] * p.sum()).sum()) + 1
    if "min_p" in kw:
        keep = int((p >= kw["min_p"]).sum())
    keep = line[:keep]
    share = p[keep] / p[keep].sum()
    assert np.abs(count[keep] - n * share).max() <= 1 + 1e-6 and count.sum() == count[keep].sum()


@pytest.mark.parametrize("N,V", [(11, 1000), (11, 40000), (11, 150001), (140, 1000), (300, 40000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_equal_logits(N, V, dtype):
    """Rows of one value, of two, and with equal logits at every border: ties go by index."""
    _need_gpu()
    g = torch.Generator().manual_seed(1)
    logits = torch.zeros(N, V, dtype=dtype, device=DEV)
    logits[1::2] = torch.randint(0, 3, (V,), generator=g).to(DEV, dtype)
    logits[2] = -0.0
    logits[2, ::2] = 0.0                         # -0 equals 0
    logits[3] = torch.finfo(dtype).min           # masked alike: uniform
    logits[4, 1:] = torch.finfo(dtype).min       # one token left
    logits[5, : V - 1] = -INF
    uniform = torch.rand(N, generator=g).to(DEV)
    uniform[6], uniform[7], uniform[8], uniform[9] = 0.0, 1.0 - 2.0 ** -24, 1.0, NAN
    for kw in (dict(), dict(top_k=37), dict(top_p=0.37), dict(top_p=0.5), dict(top_k=V // 2 + 1, top_p=0.31), dict(min_p=0.9),
               dict(temperature=0.0), dict(temperature=1e-3), dict(temperature=1e4, top_p=0.77)):
        got = sample(logits, uniform, **kw)
        check_sample(logits[:12], uniform[:12], [x[:12] for x in got], **kw)
        assert got.token[4] == 0 and got.token[5] == V - 1
    got = sample(logits, uniform, temperature=0.0)
    assert got.token[0] == got.token[2] == got.token[3] == 0


@pytest.mark.parametrize("N,V", [(12, 700), (12, 40000), (12, 150001), (150, 700), (300, 40000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_masks_and_bad_rows(N, V, dtype):
    _need_gpu()
    logits, uniform = rows_of(N, V, dtype, V + 1)
    want = sample(logits, uniform, top_p=0.9)
    logits[0, V // 3:] = -INF
    logits[1, V // 3:] = torch.finfo(dtype).min
    logits[2, 3] = NAN
    logits[3, V - 1] = INF
    logits[4] = -INF
    logits[5, 0] = -NAN
    logits[6, :] = -INF
    logits[6, [5, V - 2]] = 1.0                  # fewer tokens than top_k
    for kw in (dict(), dict(top_k=9), dict(top_p=0.9), dict(top_k=600, top_p=0.5), dict(min_p=0.01), dict(temperature=0.0)):
        got = sample(logits, uniform, **kw)
        check_sample(logits[:12], uniform[:12], [x[:12] for x in got], **kw)
        assert (got.token[2:6] == -1).all() and torch.isnan(got.logp[2:6]).all() and torch.isnan(got.kept[2:6]).all()
    got = sample(logits, uniform, top_p=0.9)
    assert torch.equal(got.token[7:], want.token[7:]) and torch.equal(got.logp[7:], want.logp[7:])
    T = torch.ones(N, device=DEV)
    T[7], T[8], T[9], T[10], T[11] = NAN, -1.0, INF, 2.0 ** -30, 1e30
    got = sample(logits, uniform, temperature=T)
    assert (got.token[7:12] == -1).all() and torch.isnan(got.logp[7:12]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_takes_what_policy_loss_takes(dtype):
    """logp is policy_loss's log probability of the token at the same temperature."""
    _need_gpu()
    from tiled_newton_schulz_tile_amd.policy import policy_loss
    N, V = 40, 32003
    logits, uniform = rows_of(N, V, dtype, 8)
    one = torch.ones(N, device=DEV)
    got = sample(logits, uniform, temperature=0.7, top_p=0.9)
    lp = policy_loss(logits, got.token, one, one, temperature=0.7, dlogits=False).logp
    # (fp32's error there, as in its own tests)
    assert ((lp - got.logp).abs() <= 2.0 ** -22 * (2 + lp.abs()) + 2.0 ** -24 * (V / 512 + 24)).all()


def check_top(logits, k, got, temperature=1.0):
    """Indices and values are the reference's.  The rest: the largest logit over T is rounded at 2^-23 of itself; the
    distance to it at 2^-23 of its value, which weighs at most log V in the mean, a thread adds V / 256 terms (at least)
    and a join of ten levels follows."""
    z = logits.double().cpu().numpy()
    V = z.shape[1]
    value, index, rest = got.value.double().cpu().numpy(), got.index.cpu().numpy(), got.rest.double().cpu().numpy()
    for n in range(len(z)):
        want, lse = S.top_row(z[n], k, temperature)
        assert (index[n] == want).all(), (n, index[n][index[n] != want][:5], want[index[n] != want][:5])
        assert np.array_equal(value[n], z[n][want], equal_nan=True)
        if not np.isfinite(lse):
            assert np.array_equal(rest[n], lse, equal_nan=True)
            continue
        others = np.delete(z[n], want) / temperature
        tol = 2.0 ** -22 * (np.abs(others[np.isfinite(others)]).max() + 2 + math.log(V)) + 2.0 ** -24 * (V / 256 + 24)
        assert abs(rest[n] - lse) <= tol, (n, rest[n], lse, tol)


@pytest.mark.parametrize("V", [1, 2, 9, 64, 257, 1000, 2049, 4104, 8195, 16384, 32003, 50257, 131072, 131075, 150001])
@pytest.mark.parametrize("N", [3, 140])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_top_matches_reference(V, N, dtype):
    _need_gpu()
    logits, _ = rows_of(N, V, dtype, V + N, pad=1)
    for k in sorted({1, min(V, 20), min(V, 64), min(V, 100), min(V, 1024)}):
        got = top_logits(logits, k, temperature=0.7)
        check_top(logits[:8], k, TopOf(got, 8), 0.7)
        again = top_logits(logits, k, temperature=0.7)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


class TopOf:
    def __init__(self, got, n):
        self.value, self.index, self.rest = (x[:n] for x in got)


@pytest.mark.parametrize("N,V", [(13, 1100), (13, 40000), (13, 150001), (140, 1100), (140, 40000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_top_ties_masks_and_nan(N, V, dtype):
    _need_gpu()
    g = torch.Generator().manual_seed(2)
    logits, _ = rows_of(N, V, dtype, 5, scale=0.05)
    logits[0] = 0
    logits[1] = torch.randint(0, 3, (V,), generator=g).to(DEV, dtype)
    logits[2] = -0.0
    logits[2, ::3] = 0.0
    logits[3] = -INF
    logits[4] = -INF
    logits[4, V // 2:V // 2 + 30] = 1.0
    logits[5, 7:] = torch.finfo(dtype).min
    logits[6, [3, V - 1]] = NAN
    logits[7, [4, V - 2]] = INF
    logits[8, 11] = -NAN
    logits[9] = NAN
    logits[10] = torch.arange(V).flip(0).to(DEV, dtype)      # sorted: the largest together
    logits[11] = torch.arange(V).to(DEV, dtype)
    logits[12] = INF
    for k in (1, 2, 33, 64, 500, 1024):
        check_top(logits[:13], k, TopOf(top_logits(logits, k), 13))


@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 5), (61, 7)])
@pytest.mark.parametrize("N,V", [(9, 97), (9, 33000), (130, 4099)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_select_strides_and_alignments(N, V, pad, offset, dtype):
    _need_gpu()
    logits, uniform = rows_of(N, V, dtype, V + pad, pad=pad, offset=offset)
    kw = dict(top_k=30, top_p=0.95)
    check_sample(logits[:9], uniform[:9], [x[:9] for x in sample(logits, uniform, **kw)], **kw)
    check_top(logits[:9], 30, TopOf(top_logits(logits, 30), 9))


def test_select_largest_vocabulary():
    _need_gpu()
    V = 1 << 20
    for dtype, scale in ((torch.bfloat16, 1.0), (torch.float32, 0.2)):
        logits, uniform = rows_of(2, V, dtype, 1, scale)
        for kw in (dict(), dict(top_p=0.9), dict(top_k=100)):
            check_sample(logits, uniform, sample(logits, uniform, **kw), **kw)
        for k in (10, 1024):
            check_top(logits, k, top_logits(logits, k))
    big = torch.zeros(1, V + 1, device=DEV)
    for call in (lambda: sample(big, big[0, :1]), lambda: top_logits(big, 1)):
        with pytest.raises(hm.HiMuonError):
            call()


def test_select_offsets_past_32_bits():
    """Rows whose element offset does not fit 32 bits (a row stride into a large buffer)."""
    _need_gpu()
    N, V, ld = 5, 1003, (1 << 30) + 7
    buf = torch.zeros((N - 1) * ld + V, dtype=torch.bfloat16, device=DEV)
    view = torch.as_strided(buf, (N, V), (ld, 1))
    small, uniform = rows_of(N, V, torch.bfloat16, 3)
    view.copy_(small)
    for a, b in zip(sample(view, uniform, top_p=0.9), sample(small, uniform, top_p=0.9)):
        assert torch.equal(a, b)
    for a, b in zip(top_logits(view, 40), top_logits(small, 40)):
        assert torch.equal(a, b)


def test_select_no_rows_and_many_rows():
    _need_gpu()
    e = torch.zeros(0, 50, device=DEV)
    assert [x.numel() for x in sample(e, e[:, 0])] == [0, 0, 0]
    got = top_logits(e, 3)
    assert got.value.shape == got.index.shape == (0, 3) and got.rest.shape == (0,)
    N, V = (1 << 21) + 3, 9                              # more rows than a launch holds
    g = torch.Generator(device=DEV).manual_seed(1)
    z = torch.randn(N, V, device=DEV, generator=g).bfloat16()
    u = torch.rand(N, device=DEV, generator=g)
    k = torch.randint(0, 9, (N,), device=DEV, generator=g).int()
    got, most = sample(z, u, top_k=k, top_p=0.9), top_logits(z, 4)
    for a in (slice(N - 300, N), slice(1000, 1300)):
        assert all(torch.equal(x, y[a]) for x, y in zip(sample(z[a], u[a], top_k=k[a], top_p=0.9), got))
        assert all(torch.equal(x, y[a]) for x, y in zip(top_logits(z[a], 4), most))


@pytest.mark.parametrize("N,V", [(1, 32000), (64, 5001), (140, 5001), (8, 140001)])
def test_select_on_another_stream_and_in_a_graph(N, V):
    _need_gpu()
    logits, uniform = rows_of(N, V, torch.bfloat16, 21)
    kw = dict(temperature=0.9, top_k=100, top_p=0.97, min_p=0.001)

    def run(stream=None):
        return (*sample(logits, uniform, stream=stream, **kw), *sample(logits, uniform, top_p=0.9, stream=stream),
                *sample(logits, uniform, stream=stream), *top_logits(logits, 50, stream=stream))

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
        logits.mul_(1 - 0.25 * n)
        uniform.mul_(0.7)
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_select_two_calls_at_once():
    """Calls on two streams share nothing."""
    _need_gpu()
    sets = [rows_of(N, V, torch.bfloat16, N) for N, V in ((48, 50001), (100, 20001))]

    def run(a, s=None):
        return (*sample(*a, top_p=0.9, stream=s), *sample(*a, top_k=40, stream=s), *top_logits(a[0], 64, stream=s))

    want = [run(a) for a in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[run(a, s) for a, s in zip(sets, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        for x, y in zip(pair, want):
            assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_select_wrapper_refusals():
    _need_gpu()
    z, u = rows_of(4, 10, torch.float32, 1)
    for bad in [dict(logits=z.t()), dict(logits=z.half()), dict(logits=z[0]), dict(uniform=u[:3]), dict(uniform=u.double()),
                dict(uniform=u.cpu()), dict(temperature=u.double()), dict(top_k=u), dict(top_p=u[:2]),
                dict(min_p=torch.ones(8, device=DEV)[::2])]:
        with pytest.raises(ValueError):
            sample(**(dict(logits=z, uniform=u) | bad))
    for bad in [dict(temperature=-1.0), dict(temperature=NAN), dict(temperature=1e9), dict(top_p=NAN), dict(min_p=NAN)]:
        with pytest.raises(hm.HiMuonError):
            sample(z, u, **bad)
    for bad in [dict(k=0), dict(k=11), dict(k=-1), dict(k=3, temperature=0.0)]:
        with pytest.raises(hm.HiMuonError):
            top_logits(z, **bad)
    with pytest.raises(ValueError):
        top_logits(z.t(), 1)


@pytest.mark.parametrize("N", [3, 300, 2100, 4200])
@pytest.mark.parametrize("k", [1, 50, 216, 217, 640, 641, 1024])
@pytest.mark.parametrize("way", ["up", "down", "mixed"])
def test_ordered_rows(N, k, way):
    """Rows that rise, fall or do neither, for every number of waves a row: rising ones raise a list's bound all the
    way, and in ordered ones a single stretch has all that is kept.  Logits are all different in fp32, so torch's top k is the
    only right one.  rest: each power is within 2^-23 (1 + ln 2 |x|) of itself, x below 30 octaves where it counts, so
    the sum within 2^-18 and three levels of 2^-24, its logarithm by as much, and that is rounded."""
    _need_gpu()
    V = 9001
    g = torch.Generator().manual_seed(k)
    z = (torch.randperm(V, generator=g).double() / V * 20 - 10).float().expand(N, V).contiguous().cuda()
    if way != "mixed":
        z = z.sort(1, descending=way == "down").values.contiguous()
    z += (torch.arange(N) % 7).float()[:, None].cuda()   # (rounds, but an order of steps of 2e-3 stays)
    got = top_logits(z, k, temperature=0.9)
    want = z.topk(k, 1)
    assert torch.equal(got.value, want.values) and torch.equal(got.index, want.indices)
    rest = (z.double().scatter(1, want.indices, -INF) / 0.9).logsumexp(1)
    assert ((got.rest - rest).abs() <= 2.0 ** -17 + 2.0 ** -23 * rest.abs()).all()
    u = torch.rand(N, generator=g).cuda()
    for kw in (dict(top_k=k), dict(top_p=0.9), dict(min_p=0.05), dict(top_k=k, top_p=0.5, min_p=1e-4, temperature=3.0)):
        drawn = sample(z, u, **kw)
        some = torch.arange(0, N, max(1, N // 5))
        assert check_sample(z[some], u[some], [x[some] for x in drawn], **kw) == len(some)
