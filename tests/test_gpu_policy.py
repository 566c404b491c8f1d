"""himuon_policy_loss against the fp64 reference (MI355X only): vocabularies from one token
to sizes past a block's first sweep, odd ones, row strides, unaligned starts, masked rows
with garbage in them, logits of -inf, missing log probabilities, in-place gradients, other
streams and graph replays."""
import numpy as np
import pytest
import torch

from oracle import training as T

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.policy import policy_loss  # noqa: E402

DEV = "cuda"
VOCABS = [1, 2, 7, 8, 9, 31, 64, 257, 1000, 4095, 4104, 8195, 16384, 32003, 50257, 131072, 131073, 150001]


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(N, V, dtype, seed, pad=0, offset=0, masked=0.3, spread=2.5):
    """Device inputs of one call; logits are a (N, V) view of rows V + pad apart, `offset` elements into memory."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, V, generator=g) * spread
    z = (z + 0.3 * torch.randn(N, V, generator=g) ** 3).to(dtype)
    buf = torch.full((offset + N * (V + pad),), float("nan"), dtype=dtype, device=DEV)
    logits = buf[offset:].view(N, V + pad)[:, :V]
    logits.copy_(z)
    label = torch.randint(0, V, (N,), generator=g)
    weight = torch.rand(N, generator=g) + 0.1
    weight[torch.rand(N, generator=g) < masked] = 0
    lp = torch.log_softmax(z.double(), 1).gather(1, label[:, None])[:, 0]
    old = (lp + 0.2 * torch.randn(N, generator=g)).float()
    ref = (lp + 0.2 * torch.randn(N, generator=g)).float()
    adv = torch.randn(N, generator=g)
    return logits, [t.to(DEV) for t in (label, weight, adv, old, ref)]


def check(logits, rest, got, dtype, **kw):
    """Outputs within the error of the fp32 formulas.  A row's log probability: the largest logit distance is rounded
    at 2^-24 of its value, a thread sums V / 512 terms (at least) one after the other and a join of nine levels
    follows; exp2, log2 and the two products are within 2^-22 together.  The ratio and the KL term add their own
    exponents' errors.  A gradient entry carries those errors times its size, and its type's rounding."""
    label, weight, adv, old, ref = rest
    kw = dict(kw)
    z = logits.double().cpu().numpy()
    a = [None if x is None else x.double().cpu().numpy() for x in (weight, adv, kw.pop("old", old), kw.pop("ref", ref))]
    stats, lp, grad = T.policy_loss(z, label.cpu().numpy(), *a, **kw)
    V = z.shape[1]
    temp = kw.get("temperature", 1.0)
    tol = 2.0 ** -22 * (1 + np.abs(lp)) + 2.0 ** -24 * (V / 512 + 24)
    live = np.isfinite(lp) & (a[0] != 0) & (label.cpu().numpy() >= 0) & (label.cpu().numpy() < V)
    glp = got.logp.double().cpu().numpy()
    assert (np.abs(glp - lp)[live] <= tol[live]).all(), np.abs(glp - lp)[live].max()
    assert not glp[~live & ~np.isnan(lp)].any()
    d = np.zeros_like(lp) if a[3] is None else np.where(live, a[3] - lp, 0)
    rho = np.ones_like(lp) if a[2] is None else np.where(live, np.exp(np.where(live, lp - a[2], 0)), 0)
    size = a[0] * (np.abs(rho * a[1]) + (np.abs(kw.get("kl_coef", 0.0)) + 1) * (np.exp(d) + np.abs(d) + 1))
    size = np.where(live, size, 0)
    assert (np.abs(got.stats.double().cpu().numpy() - stats) <= (size * (2 * tol + 2.0 ** -20)).sum() + 1e-30).all()
    if got.dlogits is None:
        return
    gz = got.dlogits.double().cpu().numpy()
    assert np.isfinite(gz[live]).all() and not gz[~live & ~np.isnan(lp)].any()
    with np.errstate(all="ignore"):
        p = np.exp(z / temp - (z / temp).max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    p[np.arange(len(p)), np.where(live, label.cpu().numpy(), 0)] += 1
    scale = (size * np.abs(kw.get("grad_scale", 1.0)) / temp)[:, None] * p
    bound = scale * (4 * tol + 2.0 ** -20)[:, None] + np.abs(grad) * (2.0 ** -8 if dtype == torch.bfloat16 else 0) + 1e-37
    off = np.abs(gz - grad)[live] > bound[live]
    assert not off.any(), (off.sum(), np.abs(gz - grad)[live].max())


@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_policy_matches_reference(V, dtype):
    _need_gpu()
    N = 7 if V > 10000 else 33
    logits, rest = make(N, V, dtype, V, masked=0.2)
    kw = dict(clip=(0.2, 0.28), kl_coef=0.05, temperature=0.8, grad_scale=3.0)
    label, weight, adv, old, ref = rest
    got = policy_loss(logits, label, weight, adv, old, ref, **kw)
    check(logits, rest, got, dtype, **kw)
    fwd = policy_loss(logits, label, weight, adv, old, ref, dlogits=False, **kw)
    assert fwd.dlogits is None
    check(logits, rest, fwd, dtype, **kw)


@pytest.mark.parametrize("N,V", [(1, 32000), (3, 65537), (40, 5000), (300, 1000), (1025, 129), (5000, 40), (600, 32003)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_policy_row_counts(N, V, dtype):
    _need_gpu()
    logits, rest = make(N, V, dtype, N + V)
    label, weight, adv, old, ref = rest
    got = policy_loss(logits, label, weight, adv, old, None)
    check(logits, rest, got, dtype, ref=None)
    again = policy_loss(logits, label, weight, adv, old, None)
    for x, y in zip(got, again):
        assert torch.equal(x, y)   # fixed orders of summation


@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 5), (64, 0), (61, 7)])
@pytest.mark.parametrize("V", [97, 4099, 33000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_policy_strides_and_alignments(V, pad, offset, dtype):
    _need_gpu()
    logits, rest = make(9, V, dtype, V + pad + offset, pad=pad, offset=offset, masked=0.0)
    label, weight, adv, old, ref = rest
    buf = torch.full((9, V + 2 * pad + 1), 7.0, dtype=dtype, device=DEV)
    out = buf[:, pad:pad + V]
    got = policy_loss(logits, label, weight, adv, old, ref, kl_coef=0.1, dlogits=out)
    check(logits, rest, got, dtype, kl_coef=0.1)
    assert (buf[:, :pad] == 7).all() and (buf[:, pad + V:] == 7).all()   # nothing beside the rows


@pytest.mark.parametrize("V", [1000, 32003, 131072, 150001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_policy_gradient_in_place(V, dtype):
    _need_gpu()
    logits, rest = make(6, V, dtype, V, pad=3)
    label, weight, adv, old, ref = rest
    want = policy_loss(logits, label, weight, adv, old, ref, kl_coef=0.1)
    z = logits.clone()
    got = policy_loss(z, label, weight, adv, old, ref, kl_coef=0.1, dlogits=z)
    assert got.dlogits is z and torch.equal(z, want.dlogits) and torch.equal(got.logp, want.logp)


@pytest.mark.parametrize("V", [513, 40000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_policy_masked_rows_hide_their_contents(V, dtype):
    _need_gpu()
    logits, rest = make(8, V, dtype, 4, masked=0.0)
    label, weight, adv, old, ref = rest
    logits[1] = float("nan")
    weight[1] = 0
    logits[2] = float("inf")
    label[2] = -100
    label[3] = V
    old[4] = float("nan")
    weight[4] = 0
    adv[5] = float("inf")
    label[5] = -1
    got = policy_loss(logits, label, weight, adv, old, ref, kl_coef=0.1)
    off = [1, 2, 3, 4, 5]
    assert not got.logp[off].any() and not got.dlogits[off].any() and torch.isfinite(got.stats).all()
    keep = [0, 6, 7]
    part = policy_loss(logits[keep].contiguous(), *(t[keep].contiguous() for t in (label, weight, adv, old, ref)), kl_coef=0.1)
    assert torch.equal(part.logp, got.logp[keep]) and torch.equal(part.dlogits, got.dlogits[keep])
    assert torch.equal(part.stats, got.stats)
    weight.zero_()
    got = policy_loss(logits, label, weight, adv, old, ref)
    assert not got.stats.any() and not got.logp.any() and not got.dlogits.any()


@pytest.mark.parametrize("V", [600, 33001, 140001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_policy_infinite_logits(V, dtype):
    _need_gpu()
    logits, rest = make(9, V, dtype, 8, masked=0.0)
    label, weight, adv, old, ref = rest
    logits[:, V // 3:] = float("-inf")               # tokens that may not be sampled
    logits[:, 5] = float("-inf")
    logits[6, : V - 1] = float("-inf")                # one token left, in the row's last place
    logits[6, V - 1] = 2.0
    label.fill_(1)
    label[6] = V - 1
    lowest = torch.finfo(dtype).min
    logits[7, V // 3:] = lowest                       # a mask of the type's lowest value
    old.fill_(-3.0)
    ref.fill_(-3.5)
    got = policy_loss(logits, label, weight, adv, old, ref, kl_coef=0.02)
    check(logits, rest, got, dtype, kl_coef=0.02)
    assert got.logp[6] == 0 and not got.dlogits[:6, V // 3:].any()
    # NaN and +inf among the logits, and nothing but -inf, give NaN in their own row
    logits[0, V - 1] = float("nan")
    logits[1, 0] = float("inf")
    logits[2] = float("-inf")
    got = policy_loss(logits, label, weight, adv, old, ref)
    assert torch.isnan(got.logp[:3]).all() and torch.isfinite(got.logp[3:]).all()
    assert torch.isnan(got.dlogits[:3]).any(1).all() and torch.isfinite(got.dlogits[3:]).all()
    assert torch.isnan(got.stats[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_policy_on_policy_and_large_logits(dtype):
    """Without old log probabilities the ratio is 1 and nothing is clipped; logits far from zero."""
    _need_gpu()
    logits, rest = make(16, 3001, dtype, 2, masked=0.0)
    logits.add_(200.0)
    logits[3].mul_(50.0)
    label, weight, adv, old, ref = rest
    label[3] = logits[3].float().argmax()
    got = policy_loss(logits, label, weight, adv)
    check(logits, rest, got, dtype, old=None, ref=None)
    assert got.stats[3] == 0


def test_policy_gradient_is_the_difference_quotient():
    """The gradient from the kernel (fp32) against central differences of the reference's loss in fp64."""
    _need_gpu()
    logits, rest = make(5, 37, torch.float32, 11, masked=0.0)
    label, weight, adv, old, ref = rest
    kw = dict(clip=(0.2, 0.28), kl_coef=0.1, temperature=1.3)
    got = policy_loss(logits, label, weight, adv, old, ref, **kw).dlogits.double().cpu().numpy()
    z = logits.double().cpu().numpy()
    a = [label.cpu().numpy()] + [x.double().cpu().numpy() for x in (weight, adv, old, ref)]
    h = 1e-4
    for i in range(5):
        for j in range(0, 37, 3):
            zp, zm = z.copy(), z.copy()
            zp[i, j] += h
            zm[i, j] -= h
            d = (T.policy_loss(zp, *a, **kw)[0][0] - T.policy_loss(zm, *a, **kw)[0][0]) / (2 * h)
            # h^2 / 6 third derivatives (a few units), and the kernel's fp32
            assert abs(d - got[i, j]) <= 1e-7 + 2e-5 * abs(d) + 1e-6


def test_policy_no_rows():
    _need_gpu()
    z = torch.zeros(0, 100, device=DEV)
    e = torch.zeros(0, device=DEV)
    got = policy_loss(z, torch.zeros(0, dtype=torch.int64, device=DEV), e, e)
    assert not got.stats.any() and got.logp.shape == (0,) and got.dlogits.shape == (0, 100)


def test_policy_offsets_past_32_bits():
    """Rows whose element offset does not fit 32 bits (a row stride into a large buffer)."""
    _need_gpu()
    N, V, ld = 5, 1003, (1 << 30) + 7
    buf = torch.zeros(N - 1, ld, dtype=torch.bfloat16, device=DEV).view(-1)
    buf = torch.cat([buf, torch.zeros(V, dtype=torch.bfloat16, device=DEV)])
    view = torch.as_strided(buf, (N, V), (ld, 1))
    small, rest = make(N, V, torch.bfloat16, 3, masked=0.0)
    view.copy_(small)
    label, weight, adv, old, ref = rest
    want = policy_loss(small, label, weight, adv, old, ref)
    got = policy_loss(view, label, weight, adv, old, ref, dlogits=view)
    assert torch.equal(got.logp, want.logp) and torch.equal(got.dlogits, want.dlogits)


def test_policy_on_another_stream_and_in_a_graph():
    _need_gpu()
    logits, rest = make(64, 5001, torch.bfloat16, 21)
    label, weight, adv, old, ref = rest
    want = policy_loss(logits, label, weight, adv, old, ref, kl_coef=0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = policy_loss(logits, label, weight, adv, old, ref, kl_coef=0.1, stream=s)
    s.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = policy_loss(logits, label, weight, adv, old, ref, kl_coef=0.1)
    for k in range(3):
        logits.add_(0.25 * k)
        old.sub_(0.01 * k)
        want = policy_loss(logits, label, weight, adv, old, ref, kl_coef=0.1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(held, want):
            assert torch.equal(x, y)


def test_policy_wrapper_refusals():
    _need_gpu()
    z, rest = make(4, 10, torch.float32, 1)
    label, weight, adv, old, ref = rest
    for bad in [dict(logits=z.t()), dict(logits=z.half()), dict(logits=z[0]), dict(label=label.int()),
                dict(weight=weight[:3]), dict(old_logp=old.double()), dict(advantage=None),
                dict(dlogits=torch.empty(4, 11, device=DEV)), dict(dlogits=torch.empty(4, 10, device=DEV).bfloat16()),
                dict(weight=weight.cpu())]:
        args = dict(logits=z, label=label, weight=weight, advantage=adv, old_logp=old) | bad
        with pytest.raises(ValueError):
            policy_loss(**args)
    for bad in [dict(clip=(-0.1, 0.2)), dict(clip=(1.1, 0.2)), dict(clip=(0.2, float("inf"))), dict(kl_coef=float("nan")),
                dict(temperature=0.0), dict(temperature=float("inf")), dict(grad_scale=float("nan"))]:
        with pytest.raises(hm.HiMuonError):
            policy_loss(z, label, weight, adv, old, **bad)


@pytest.mark.parametrize("V", [255, 1024, 2049, 4097, 8192, 16385, 32768, 32777, 50257, 65537, 131071, 131080, 150001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_policy_more_rows_than_are_split(V, dtype):
    """More rows than the path that cuts rows into spans takes: every size of row that a block holds in registers,
    and rows past it; forward alone, with the gradient, and in place."""
    _need_gpu()
    logits, rest = make(133, V, dtype, V, pad=1, masked=0.9)
    label, weight, adv, old, ref = rest
    weight[132] = 0.5
    kw = dict(clip=(0.2, 0.28), kl_coef=0.05, temperature=1.2)
    got = policy_loss(logits, label, weight, adv, old, ref, **kw)
    check(logits, rest, got, dtype, **kw)
    fwd = policy_loss(logits, label, weight, adv, old, ref, dlogits=False, **kw)
    check(logits, rest, fwd, dtype, **kw)
    z = logits.clone()
    policy_loss(z, label, weight, adv, old, ref, dlogits=z, **kw)
    assert torch.equal(z, got.dlogits)


@pytest.mark.parametrize("V", [3000, 40000, 140001])
def test_policy_extreme_rows_among_many(V):
    """Rows of -inf, of the lowest value, with NaN or +inf, on the paths for many rows."""
    _need_gpu()
    logits, rest = make(140, V, torch.float32, 5, masked=0.9)
    label, weight, adv, old, ref = rest
    weight[:8] = 1.0
    old[:8], ref[:8] = -3.0, -3.5
    label[:8] = 1
    logits[0, V // 3:] = float("-inf")
    logits[1, V // 3:] = torch.finfo(torch.float32).min
    logits[2] = torch.finfo(torch.float32).min          # every token masked alike: a uniform row
    logits[3] = float("-inf")
    logits[3, 1] = -5.0
    got = policy_loss(logits, label, weight, adv, old, ref)
    assert abs(float(got.logp[2]) + np.log(V)) <= 2.0 ** -21 * np.log(V) + 2.0 ** -24 * (V / 512 + 24)
    assert float(got.logp[3]) == 0
    logits[2].zero_()
    again = policy_loss(logits, label, weight, adv, old, ref)
    assert torch.equal(got.logp, again.logp) and torch.equal(got.dlogits, again.dlogits)
    check(logits, rest, got, torch.float32)
    logits[4, 7], logits[5, V - 1] = float("nan"), float("inf")
    logits[6] = float("-inf")
    got = policy_loss(logits, label, weight, adv, old, ref)
    assert torch.isnan(got.logp[4:7]).all() and torch.isfinite(got.logp[:4]).all()
    assert torch.isnan(got.dlogits[4:7]).any(1).all() and torch.isfinite(got.dlogits[:4]).all()


@pytest.mark.parametrize("V", [1001, 20000, 128256, 140001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_policy_large_gradient_equals_its_parts(V, dtype):
    """A gradient past the caches' size has the bits of the same rows in smaller calls."""
    _need_gpu()
    N = max(400, (40 << 20) // (V * 2))
    logits, rest = make(400, V, dtype, 12)
    logits = logits.repeat(-(-N // 400), 1)[:N]
    rest = [t.repeat(-(-N // 400))[:N] for t in rest]
    label, weight, adv, old, ref = rest
    got = policy_loss(logits, label, weight, adv, old, ref, kl_coef=0.1)
    n = 140
    part = policy_loss(logits[:n], *(t[:n] for t in rest), kl_coef=0.1)
    assert torch.equal(part.logp, got.logp[:n]) and torch.equal(part.dlogits, got.dlogits[:n])
    fwd = policy_loss(logits, label, weight, adv, old, ref, kl_coef=0.1, dlogits=False)
    assert torch.equal(fwd.stats, got.stats) or V > 65536   # (long rows are summed in another order without a gradient)
    reps = N // 400
    for k in range(1, reps):
        assert torch.equal(got.dlogits[400 * k:400 * (k + 1)], got.dlogits[:400])


def test_policy_more_rows_than_a_launch_holds():
    _need_gpu()
    N, V = (1 << 21) + 3, 9
    g = torch.Generator(device=DEV).manual_seed(1)
    z = torch.randn(N, V, device=DEV, generator=g).bfloat16()
    label = torch.randint(-1, V, (N,), device=DEV, generator=g)
    weight, adv = torch.rand(N, device=DEV, generator=g), torch.randn(N, device=DEV, generator=g)
    got = policy_loss(z, label, weight, adv)
    for part in (slice(N - 300, N), slice(1000, 1300)):
        one = policy_loss(z[part], label[part], weight[part], adv[part])
        assert torch.equal(one.logp, got.logp[part]) and torch.equal(one.dlogits, got.dlogits[part])
    live = label >= 0
    assert abs(float(got.stats[1]) + float((weight * adv)[live].double().sum())) <= 1e-6 * float((weight * adv.abs())[live].sum())


@pytest.mark.parametrize("N,V", [(4, 500), (4, 40000), (140, 40000), (140, 140001)])
def test_policy_infinite_kl_that_does_not_count(N, V):
    """A sampled token that the policy now gives probability 0: with kl_coef 0 the KL sum is infinite, the loss and
    the gradient are not."""
    _need_gpu()
    logits, rest = make(N, V, torch.float32, 31, masked=0.0)
    label, weight, adv, old, ref = rest
    logits[0, label[0]] = float("-inf")
    ref[1] = 500.0                          # exp(ref - lp) past fp32
    got = policy_loss(logits, label, weight, adv, old, ref)
    assert torch.isfinite(got.stats[[0, 1, 3]]).all() and not torch.isfinite(got.stats[2])
    assert torch.isfinite(got.dlogits).all() and got.logp[0] == float("-inf")
    want = policy_loss(logits, label, weight, adv, old)
    assert torch.equal(got.dlogits, want.dlogits) and torch.equal(got.stats[:2], want.stats[:2])
