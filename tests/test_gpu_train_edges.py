"""Calls of the training step's operators at the edges of what their documentation allows
(MI355X only): gradients in the place of the logits for many blocks a row, calls on another
stream than the current one, and gradients from subnormal ones to those whose squares overflow."""
import numpy as np
import pytest
import torch

from oracle import training as T

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.adamw import AdamW, GradNorm, adamw_moments, adamw_state  # noqa: E402
from tiled_newton_schulz_tile_amd.policy import policy_loss  # noqa: E402
from test_gpu_adamw import check8  # noqa: E402

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def policy_inputs(N, V, dtype, seed, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    logits = (2.5 * rand(N, V + pad)).to(dtype)[:, :V]
    label = torch.randint(0, V, (N,), device=DEV, generator=g)
    label[:5] = torch.tensor([0, V - 1, V // 8 * 8 - 1, min(V - 1, V // 8 * 8), V // 2], device=DEV)
    lp = torch.log_softmax(logits.double(), 1).gather(1, label[:, None])[:, 0].float()
    weight = torch.rand(N, device=DEV, generator=g) + 0.1
    weight[::7] = 0
    return logits, (label, weight, rand(N), lp + 0.2 * rand(N), lp + 0.2 * rand(N))


@pytest.mark.parametrize("N,V", [(6, 150001), (64, 4099), (65, 50257), (100, 32003), (128, 16391), (128, 128256),
                                 (128, 150001)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_policy_few_rows_in_place_equal_their_own_buffer(N, V, dtype):
    """Rows that are cut into spans, as many blocks as the chip holds at once and more, labels in every place: a
    gradient written over the logits has the bits of one with a buffer of its own, and so have the terms and sums."""
    _need_gpu()
    logits, rest = policy_inputs(N, V, dtype, N + V, pad=3)
    kw = dict(clip=(0.2, 0.28), kl_coef=0.1, temperature=0.9)
    want = policy_loss(logits, *rest, **kw)
    z = logits.clone()
    got = policy_loss(z, *rest, dlogits=z, **kw)
    assert torch.equal(got.logp, want.logp) and torch.equal(got.stats, want.stats)
    assert torch.equal(z, want.dlogits)


def pool_stream(t):
    """The stream whose pool of torch's allocator a tensor's memory belongs to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not torch's memory")


def reused(nbytes, ptr):
    """Whether one of the next allocations of that many bytes on the current stream gets the address `ptr`."""
    held = [torch.empty(nbytes, dtype=torch.uint8, device=DEV) for _ in range(8)]
    return any(t.data_ptr() == ptr for t in held)


def test_results_belong_to_the_stream_that_writes_them():
    """Memory of the current stream's pool may still be used by kernels pending there: what a call on another stream
    writes is allocated on that one."""
    _need_gpu()
    logits, rest = policy_inputs(12, 1001, F32, 1)
    G = torch.randn(1000, device=DEV)
    norm = GradNorm([G])
    want, n = policy_loss(logits, *rest), norm.compute(1.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, m = policy_loss(logits, *rest, stream=s), norm.compute(1.0, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for t in (got.stats, got.logp, got.dlogits, m):
        assert pool_stream(t) == s.cuda_stream
    for t in (want.stats, want.dlogits, n):
        assert pool_stream(t) == torch.cuda.current_stream().cuda_stream
    for x, y in zip((*got, m), (*want, n)):
        assert torch.equal(x, y)


def test_policy_arguments_outlive_a_call_on_another_stream():
    """Logits that the caller lets go of while a call on another stream has yet to read them are not handed out."""
    _need_gpu()
    logits, rest = policy_inputs(32, 40000, F32, 2)
    want = policy_loss(logits, *rest)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = logits.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    got = policy_loss(z, *rest, stream=s)
    ptr, nbytes = z.data_ptr(), z.numel() * 4
    del z
    assert not reused(nbytes, ptr)
    torch.cuda.synchronize()
    assert torch.equal(got.dlogits, want.dlogits) and torch.equal(got.stats, want.stats)


@pytest.mark.parametrize("given", [True, False])
def test_descriptors_and_workspaces_outlive_steps_on_another_stream(given):
    """The device table of an AdamW, the workspace of a GradNorm and gradients that were replaced, all made on one
    stream and let go of while work on another has yet to read them, are not handed out; given: the stream is an
    argument, or the current one at the call."""
    _need_gpu()
    sizes = [1000 + k for k in range(20)]
    W = [torch.randn(n, device=DEV) for n in sizes]
    G = [torch.randn(n, device=DEV) for n in sizes]
    V, sw, sv = [w.clone() for w in W], [adamw_state(w) for w in W], [adamw_state(w) for w in W]
    AdamW([(v, g, *t) for v, g, t in zip(V, G, sv)]).step(1e-2, 1)
    want = GradNorm(G).compute(1.0)
    old = [g.clone() for g in G]
    opt, norm = AdamW([(w, g, *t) for w, g, t in zip(W, old, sw)]), GradNorm(old)
    table, ws = opt._table.data_ptr(), norm._ws.data_ptr()
    sizes_of = opt._table.numel(), norm._ws.numel()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        if not given:
            opt.step(1e-2, 1)
            got = norm.compute(1.0)
    if given:
        opt.step(1e-2, 1, stream=s)
        got = norm.compute(1.0, stream=s)
    last = [g.data_ptr() for g in old[-2:]]
    opt.set_grads([*old[:-1], G[-1]], stream=s)   # (for the next step there)
    norm.set_grads([*old[:-1], G[-1]])
    del old
    assert not reused(sizes[-1] * 4, last[1])
    del opt, norm
    assert not reused(sizes[-2] * 4, last[0])
    assert not reused(sizes_of[0], table) and not reused(sizes_of[1], ws)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for w, v in zip(W, V):
        assert torch.equal(w, v)


@pytest.mark.parametrize("given", [True, False])
def test_factors_outlive_calls_on_another_stream(given):
    """A factor that a step has yet to read, and a result's place that a norm has yet to write, are not handed out."""
    _need_gpu()
    W, G = torch.zeros(100, device=DEV), torch.ones(100, device=DEV)
    opt, norm = AdamW([(W, G, *adamw_state(W))]), GradNorm([G])
    s = torch.cuda.Stream()
    factor, out = torch.full((1,), float("nan"), device=DEV), torch.zeros(2, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        if not given:
            opt.step(0.5, 1, scale=factor)
            norm.compute(1.0, out=out)
    if given:
        opt.step(0.5, 1, scale=factor, stream=s)
        norm.compute(1.0, out=out, stream=s)
    ptrs = factor.data_ptr(), out.data_ptr()
    del factor, out
    held = [torch.ones(1, device=DEV) for _ in range(16)]
    assert not {t.data_ptr() for t in held} & set(ptrs)
    torch.cuda.synchronize()
    assert not W.any() and all(t == 1 for t in held)


@pytest.mark.parametrize("count", [2, 20])
def test_adamw_needs_gradients_after_they_were_dropped(count):
    """(with descriptors in the arguments and in a table)"""
    _need_gpu()
    W = [torch.zeros(100, device=DEV) for _ in range(count)]
    G = [torch.ones(100, device=DEV) for _ in range(count)]
    opt = AdamW([(w, g, *adamw_state(w)) for w, g in zip(W, G)])
    opt.step(0.5, 1)
    opt.drop_grads()
    with pytest.raises(RuntimeError):
        opt.step(0.5, 2)
    assert all((w == -0.5).all() for w in W)
    opt.set_grads(G)
    opt.step(0.5, 2)
    assert all(((w + 1).abs() < 1e-6).all() for w in W)


@pytest.mark.parametrize("wt,gt", [(F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("big", [1e25, -3e30, 6e37, 3e38])
def test_adamw8_gradient_whose_square_overflows(wt, gt, big):
    """A finite gradient whose weighted square is past fp32: its root is not, so the states hold it, its own weight
    takes the step of the formulas, and its block's other weights stay finite, in this step and in later ones."""
    _need_gpu()
    n = 1000
    g = torch.Generator().manual_seed(5)
    W, G = torch.randn(n, generator=g).to(wt).to(DEV), torch.randn(n, generator=g).to(gt).to(DEV)
    G[300] = big
    state = adamw_state(W, 8)
    opt = AdamW([(W, G, *state)], betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
    for t, dither in ((1, (7, 8)), (2, (0xFFFF1234, 3)), (3, (1 << 31, 1 << 30))):
        before = [x.clone() for x in opt.tensors[0]]
        opt.step(1e-2, t, dither=dither)
        assert torch.isfinite(W.float()).all() and all(torch.isfinite(s.float()).all() for s in state)
        if abs(big) < 2.0 ** 126:   # (the reciprocal of a root past that is subnormal: its weight may keep still)
            check8(before, opt.tensors[0], t, 1e-2, 0.9, 0.999, 1e-8, 0.1, 1.0, dither)
        if t == 1:
            assert abs(float(state[3][1]) * 448 / (0.001 ** 0.5 * abs(float(G[300]))) - 1) < 1e-5   # the block's scale
            G[300] = 0.5


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("n", [1000, 300, 1])
def test_adamw8_element_that_is_not_finite_stays_alone(bad, n):
    """As with states in 32 bits, a gradient that is not finite and is not skipped takes its own weight and states,
    and nothing else: the others are those of a step without it, in this step and in later ones."""
    _need_gpu()
    g = torch.Generator().manual_seed(6)
    at = n // 3
    W = torch.randn(n, generator=g).to(DEV)
    V = W.clone()
    sw, sv = adamw_state(W, 8), adamw_state(V, 8)
    G = [torch.randn(n, generator=g).to(DEV) for _ in range(3)]
    H = [x.clone() for x in G]
    G[1][at] = bad
    for x in H:
        x[at] = 0   # (an element that is not finite does not set its block's scale)
    a, b = AdamW([(W, G[0], *sw)]), AdamW([(V, H[0], *sv)])
    G[0][at] = 0
    rest = torch.arange(n, device=DEV) != at
    for t in (1, 2, 3):
        a.set_grads([G[t - 1]])
        b.set_grads([H[t - 1]])
        a.step(1e-2, t, dither=(t, 9))
        b.step(1e-2, t, dither=(t, 9))
        assert torch.equal(W[rest], V[rest])
        for x, y in zip(sw[:2], sv[:2]):
            assert torch.equal(x.view(torch.uint8)[rest], y.view(torch.uint8)[rest])
        assert torch.equal(sw[2], sv[2]) and torch.equal(sw[3], sv[3])
        if t > 1:
            assert torch.isnan(W[at]) and all(torch.isnan(m[at]) for m in adamw_moments(sw))


@pytest.mark.parametrize("dtype,V", [(BF16, 1001), (BF16, 8000), (BF16, 20000), (BF16, 50257), (BF16, 100001),
                                     (F32, 1001), (F32, 9000), (F32, 30001), (F32, 57000)])
def test_policy_gradient_past_the_caches_equals_a_cached_one(dtype, V):
    """Every kernel for rows that a block holds, with stores past the L2s (a gradient above 32 MB) and with cached
    ones (a part of its rows below that), gives the same bits."""
    _need_gpu()
    row = V * (2 if dtype == BF16 else 4)
    n = 130   # (more rows than are cut into spans)
    N = max(2 * n, int(32e6 / row) + 10)
    assert N * row > 32e6 >= n * row
    logits, rest = policy_inputs(N, V, dtype, V)
    got = policy_loss(logits, *rest, kl_coef=0.1)
    for part in (slice(0, n), slice(N - n, N)):
        one = policy_loss(logits[part], *(t[part] for t in rest), kl_coef=0.1)
        assert torch.equal(one.logp, got.logp[part]) and torch.equal(one.dlogits, got.dlogits[part])


def states8_in_fp32(g, code, unit, dither, beta1=0.9, beta2=0.999):
    """The documented 8-bit states after a step: numpy float32, every operation rounded on its own.  Returns the codes
    and scales of m and r."""
    f = np.float32
    table = T.e4m3_values().astype(f)
    n = g.size
    with np.errstate(all="ignore"):
        old = [table[c] * np.repeat(u, T.BLOCK)[:n] for c, u in zip(code, unit)]
        m = f(beta1) * old[0] + f(1 - beta1) * g
        v = f(beta2) * (old[1] * old[1]) + f(1 - beta2) * g * g
        gs, rs = g * f(2.0 ** -66), old[1] * f(2.0 ** -66)
        large = f(beta2) * (rs * rs) + f(1 - beta2) * gs * gs
        past = np.isinf(v) & np.isfinite(large)
        r = np.where(past, np.minimum(np.sqrt(large) * f(2.0 ** 66), np.finfo(f).max), np.sqrt(v))
        out = []
        for k, x in enumerate((m, r)):
            lost = ~np.isfinite(x)
            x = np.where(lost, f(0), x)
            peak = np.abs(np.concatenate([x, np.zeros(-n % T.BLOCK, f)])).reshape(-1, T.BLOCK).max(1)
            held = peak >= f(2.0 ** -100)
            inv = np.repeat(np.where(held, f(1) / peak * f(448), f(0)), T.BLOCK)[:n]
            seq = ((np.arange(n, dtype=np.uint64) * T.MULT[k] + dither[k]) % 2 ** 32 >> np.uint64(16)).astype(np.uint32)
            bits = (np.abs(x) * inv * f(2.0 ** -120)).view(np.uint32)
            c = np.minimum((bits + (seq << np.uint32(4)) + np.uint32(8)) >> np.uint32(20), 126)
            c = np.maximum(c, x != 0) if k else c | (np.signbit(x) * np.uint32(128))
            c = np.where(lost, 0x7f, np.where(inv > 0, c, 0)).astype(np.uint8)
            out.append((c, np.where(held, peak * f(1 / 448), f(0))))
    return out


@pytest.mark.parametrize("spread", [2, 30, 150])
@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("n", [256, 20001])
def test_adamw8_states_over_the_range_of_fp32(spread, gt, n):
    """Bit for bit, with gradients and scales from subnormal ones to the largest, zeros, and some that are not finite,
    in blocks of one size (spread 2) or of many."""
    _need_gpu()
    for seed in range(4):
        rng = np.random.default_rng(100 * spread + seed)
        middle = np.repeat(rng.uniform(-145, 127, -(-n // T.BLOCK)), T.BLOCK)[:n]
        size = np.clip(middle + rng.uniform(-spread, spread, n), -149, 127.9)
        g = torch.from_numpy((np.sign(rng.standard_normal(n)) * 2.0 ** size * (rng.random(n) > 0.05)).astype(np.float32))
        if seed == 3:
            g[::997] = float("nan")
            g[1::1499] = float("inf")
        G = g.to(gt).to(DEV)
        blocks = -(-n // T.BLOCK)
        code = [rng.integers(0, 127, n).astype(np.uint8) for _ in range(2)]
        code[0] |= (rng.integers(0, 2, n) * 128).astype(np.uint8)
        unit = [(2.0 ** rng.uniform(-145, 119, blocks) * (rng.random(blocks) > 0.1)).astype(np.float32) for _ in range(2)]
        dither = [int(x) for x in rng.integers(0, 2 ** 32, 2)]
        state = [torch.from_numpy(c.copy()).to(DEV).view(torch.float8_e4m3fn) for c in code]
        scale = [torch.from_numpy(u.copy()).to(DEV) for u in unit]
        W = torch.zeros(n, device=DEV)
        AdamW([(W, G, *state, *scale)]).step(1e-3, 7, dither=dither)
        want = states8_in_fp32(G.float().cpu().numpy(), code, unit, dither)
        for got, s, (c, u) in zip(state, scale, want):
            assert np.array_equal(s.cpu().numpy(), u), (seed, np.nonzero(s.cpu().numpy() != u)[0][:5])
            got = got.view(torch.uint8).cpu().numpy()
            assert np.array_equal(got, c), (seed, np.nonzero(got != c)[0][:5], got[got != c][:5], c[got != c][:5])
