"""himuon_adamw_step (32-bit and 8-bit states) and himuon_grad_norm against the fp64
reference (MI355X only): one element to tensors of many chunks, more tensors than one
launch holds, empty tensors, unaligned views, every combination of types, skipped steps,
the 8-bit format byte by byte, other streams and graph replays."""
import numpy as np
import pytest
import torch

from oracle import training as T

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.adamw import AdamW, GradNorm, adamw_moments, adamw_state  # noqa: E402

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
SIZES = [1, 2, 3, 4, 5, 63, 64, 255, 256, 257, 1023, 4095, 4096, 4097, 20001]


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def place(x, dtype, offset):
    buf = torch.zeros(x.numel() + offset, dtype=dtype, device=DEV)
    v = buf[offset:]
    v.copy_(x)
    return v


def tensors32(sizes, wt, gt, seed, offset=0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for n in sizes:
        m = 0.1 * torch.randn(n, generator=g)
        v = (0.2 * torch.rand(n, generator=g) + 0.01) ** 2
        out.append((place(torch.randn(n, generator=g), wt, offset), place(torch.randn(n, generator=g), gt, offset),
                    place(m, F32, offset), place(v, F32, offset)))
    return out


def np64(*ts):
    return [t.double().cpu().numpy() for t in ts]


def check32(before, after, t, lr, beta1, beta2, eps, wd, scale):
    """Per element: two fused multiply-adds and the products in them are within 3 * 2^-24 of the terms' sizes; the
    step's root, reciprocal, constants and products within 2^-20 of the step; bf16 weights round once more."""
    w0, g0, m0, v0 = np64(*before)
    w1, m1, v1 = np64(after[0], after[2], after[3])
    w, m, v = T.adamw(w0, g0, m0, v0, t, lr, beta1, beta2, eps, wd, scale)
    if np.isnan(scale):
        assert (w1 == w0).all() and (m1 == m0).all() and (v1 == v0).all()
        return
    tm = 2.0 ** -22 * (np.abs(beta1 * m0) + np.abs((1 - beta1) * g0 * scale)) + 1e-44
    tv = 2.0 ** -21 * v + 1e-44
    assert (np.abs(m1 - m) <= tm).all() and (np.abs(v1 - v) <= tv).all()
    den = np.sqrt(v / (1 - beta2 ** t)) + eps
    step = lr / (1 - beta1 ** t) * np.abs(m) / den
    tol = step * 2.0 ** -19 + lr / (1 - beta1 ** t) * tm / den + 2.0 ** -22 * np.abs(w0) + 1e-38
    if after[0].dtype == BF16:
        tol = tol + np.abs(w) * 2.0 ** -8
    assert (np.abs(w1 - w) <= tol).all(), (np.abs(w1 - w) / tol).max()


@pytest.mark.parametrize("wt", [F32, BF16])
@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_adamw32_matches_reference(wt, gt, offset):
    _need_gpu()
    ts = tensors32(SIZES, wt, gt, 5 + offset, offset)
    opt = AdamW(ts, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1)
    scale = torch.tensor([0.7], device=DEV)
    for t in (1, 2, 1000):
        before = [[x.clone() for x in q] for q in ts]
        opt.step(3e-3, t, scale=scale)
        for b, a in zip(before, ts):
            check32(b, a, t, 3e-3, 0.9, 0.99, 1e-6, 0.1, float(scale[0]))
            assert torch.equal(b[1], a[1])


def test_adamw32_many_tensors_and_decays():
    """More tensors than one launch takes, empty ones among them, each with its own decay."""
    _need_gpu()
    sizes = [(37 * k) % 611 for k in range(333)]
    ts = tensors32(sizes, F32, F32, 9)
    decay = [0.01 * (k % 5) for k in range(333)]
    before = [[x.clone() for x in q] for q in ts]
    AdamW(ts, weight_decay=decay).step(1e-2, 3)
    for b, a, wd in zip(before, ts, decay):
        check32(b, a, 3, 1e-2, 0.9, 0.999, 1e-8, wd, 1.0)


def test_adamw32_packed_bucket():
    """Tensors packed without gaps into one buffer: nothing beside a tensor is written."""
    _need_gpu()
    sizes = [1, 3, 4097, 2, 255, 5000, 1]
    one = tensors32([sum(sizes)], BF16, BF16, 6)[0]
    two = [x.clone() for x in one]
    AdamW([one]).step(1e-3, 2)
    at, ts = 0, []
    for n in sizes:
        ts.append(tuple(x[at:at + n] for x in two))
        at += n
    AdamW(ts).step(1e-3, 2)
    for a, b in zip(one, two):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_skips_a_gradient_that_is_not_finite(bits):
    _need_gpu()
    W = torch.randn(5000, device=DEV)
    G = torch.randn(5000, device=DEV)
    G[77] = float("inf")
    opt = AdamW([(W, G, *adamw_state(W, bits))])
    before = [x.clone() for x in opt.tensors[0]]
    factor = GradNorm([G]).compute(1.0)
    assert torch.isnan(factor[1])
    opt.step(1e-2, 1, scale=factor[1:])
    for a, b in zip(before, opt.tensors[0]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_adamw32_extremes():
    """Zero gradients and states, gradients whose squares leave fp32, and a NaN that stays where it is."""
    _need_gpu()
    n = 4096
    G = torch.zeros(n, device=DEV)
    G[1], G[2], G[3], G[4] = 1e25, 1e-30, float("nan"), -1e-20
    W = torch.ones(n, device=DEV)
    m, v = adamw_state(W)
    AdamW([(W, G, m, v)], eps=1e-8).step(0.1, 1)
    w = W.cpu()
    assert torch.isnan(w[3]) and torch.isfinite(w[torch.arange(n) != 3]).all()
    assert w[0] == 1 and w[1] == 1            # v overflows: the step is zero, as in the formula
    assert abs(float(w[2]) - 1) <= 1e-6       # far below eps
    assert (w[5:] == 1).all()


def tensors8(sizes, wt, gt, seed, offset=0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for n in sizes:
        q = []
        for kind in (0, 1):
            x = torch.randn(n, generator=g) * torch.exp(torch.randn(n, generator=g))
            x = x.abs() if kind else x
            val, scale, _ = T.pack8(0.1 * x.double().numpy(), kind, 99)
            code = torch.from_numpy(val).float().to(torch.float8_e4m3fn)
            buf = torch.zeros(n + offset, dtype=torch.uint8, device=DEV)
            buf[offset:] = code.view(torch.uint8).to(DEV)
            q.append((buf[offset:].view(torch.float8_e4m3fn), torch.from_numpy(scale).float().to(DEV)))
        out.append((place(torch.randn(n, generator=g), wt, offset), place(torch.randn(n, generator=g), gt, offset),
                    q[0][0], q[1][0], q[0][1], q[1][1]))
    return out


def check8(before, after, t, lr, beta1, beta2, eps, wd, scale, dither):
    """Weights as with fp32 states of the values that the codes stand for; every code is the reference's, or its
    neighbour where the dithered magnitude is within the fp32 formulas' error of the turning point: 2^-19 of a
    magnitude of at most 16 gaps."""
    w0, g0, ms, rs = np64(before[0], before[1], before[4], before[5])
    codes = [before[k].view(torch.uint8).cpu().numpy() for k in (2, 3)]
    m0, r0 = T.unpack8(codes[0], ms), T.unpack8(codes[1], rs)
    w, m, v = T.adamw(w0, g0, m0, r0 ** 2, t, lr, beta1, beta2, eps, wd, scale)
    w1 = after[0].double().cpu().numpy()
    den = np.sqrt(v / (1 - beta2 ** t)) + eps
    tm = 2.0 ** -21 * (np.abs(beta1 * m0) + np.abs((1 - beta1) * g0 * scale)) + 1e-44
    step = lr / (1 - beta1 ** t) * np.abs(m) / den
    tol = step * 2.0 ** -18 + lr / (1 - beta1 ** t) * tm / den + 2.0 ** -22 * np.abs(w0) + 1e-38
    if after[0].dtype == BF16:
        tol = tol + np.abs(w) * 2.0 ** -8
    assert (np.abs(w1 - w) <= tol).all(), (np.abs(w1 - w) / tol).max()
    table = T.e4m3_values()
    for kind, x, err in ((0, m, tm), (1, np.sqrt(v), np.sqrt(v) * 2.0 ** -20)):
        val, unit, margin = T.pack8(x, kind, dither[kind])
        got = table[after[2 + kind].view(torch.uint8).cpu().numpy()]
        gunit = after[4 + kind].double().cpu().numpy()
        assert (np.abs(gunit - unit) <= 2.0 ** -20 * unit + 1e-38).all()
        each = np.repeat(unit, T.BLOCK)[:x.size]
        with np.errstate(all="ignore"):
            y = np.where(each > 0, np.abs(x) / each, 0)
            near = np.where(each > 0, err / each, 0)
        gap = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
        slack = 16 * 2.0 ** -19 + near / gap
        same = got == val
        # (a magnitude next to a power of two may be taken on either side of it: the gap doubles there)
        assert (same | ((margin <= slack) & (np.abs(got - val) <= 2 * gap)) | (np.abs(np.log2(np.maximum(y, 1e-30)) -
                np.round(np.log2(np.maximum(y, 1e-30)))) <= 2.0 ** -18)).all()
        assert same.mean() > 0.99 or x.size < 300


@pytest.mark.parametrize("wt", [F32, BF16])
@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_adamw8_matches_reference(wt, gt, offset):
    _need_gpu()
    ts = tensors8(SIZES, wt, gt, 15 + offset, offset)
    opt = AdamW(ts, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1)
    scale = torch.tensor([0.7], device=DEV)
    for t, dither in ((1, (0, 0)), (2, (0xFFFFFFFF, 0x12345678)), (1000, (0xDEADBEEF, 0x80000000))):
        before = [[x.clone() for x in q] for q in ts]
        opt.step(3e-3, t, scale=scale, dither=dither)
        for b, a in zip(before, ts):
            check8(b, a, t, 3e-3, 0.9, 0.99, 1e-6, 0.1, float(scale[0]), dither)


def test_adamw8_many_tensors():
    _need_gpu()
    sizes = [(37 * k) % 611 for k in range(200)]
    ts = tensors8([n for n in sizes if n], F32, BF16, 3)
    before = [[x.clone() for x in q] for q in ts]
    AdamW(ts).step(1e-2, 3, dither=(5, 6))
    for b, a in zip(before, ts):
        check8(b, a, 3, 1e-2, 0.9, 0.999, 1e-8, 0.0, 1.0, (5, 6))


def test_adamw8_every_code_survives():
    """A step that leaves the moments as they are (zero gradient, betas rounding to 1 - tiny cannot: beta 0.5 and
    doubled scales instead) keeps every e4m3 code: halving moments halves the scale and nothing else."""
    _need_gpu()
    code = torch.arange(256, dtype=torch.uint8, device=DEV)
    code[127] = code[255] = 0            # the NaN codes
    W, G = torch.zeros(256, device=DEV), torch.zeros(256, device=DEV)
    r = (torch.arange(256, device=DEV) % 127).to(torch.uint8)
    r[r == 0] = 126
    one = torch.ones(1, device=DEV)
    m8, r8 = code.clone().view(torch.float8_e4m3fn), r.clone().view(torch.float8_e4m3fn)
    ms, rs = one.clone(), one.clone()
    AdamW([(W, G, m8, r8, ms, rs)], betas=(0.5, 0.25), eps=1e-8).step(0.0, 1, dither=(123456789, 987654321))
    want = code.clone()
    want[code == 128] = 0                # minus zero becomes zero
    assert torch.equal(m8.view(torch.uint8), want) and torch.equal(r8.view(torch.uint8), r)
    assert float(ms) == 0.5 and float(rs) == 0.5


def test_adamw8_zero_blocks_and_tiny_blocks():
    _need_gpu()
    n = 1024
    W = torch.randn(n, device=DEV)
    G = torch.zeros(n, device=DEV)
    G[256:512] = 1e-35
    G[512] = 3.0
    state = adamw_state(W, 8)
    w0 = W.clone()
    AdamW([(W, G, *state)], weight_decay=0.0).step(0.1, 1, dither=(1, 2))
    m, v = adamw_moments(state)
    assert torch.equal(W[:256], w0[:256]) and torch.equal(W[513:], w0[513:])
    assert not m[:512].any() and not v[:512].any() and float(m[512]) > 0 and not m[513:].any()
    assert abs(float(w0[512] - W[512]) - 0.1) < 1e-5


def test_adamw8_follows_adamw32_over_many_steps():
    """200 steps on a quadratic: 8-bit states follow the fp32 run (the dithered rounding is unbiased; rounding each
    moment to nearest would hold the second moment still)."""
    _need_gpu()
    g = torch.Generator().manual_seed(1)
    n = 8192
    target = torch.randn(n, generator=g).to(DEV)
    W32, W8 = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    G32, G8 = torch.empty_like(W32), torch.empty_like(W8)
    s32, s8 = adamw_state(W32), adamw_state(W8, 8)
    a, b = AdamW([(W32, G32, *s32)]), AdamW([(W8, G8, *s8)])
    rng = np.random.default_rng(0)
    for t in range(1, 201):
        noise = 0.3 * torch.randn(n, generator=g).to(DEV)
        G32.copy_(W32 - target + noise)
        G8.copy_(W8 - target + noise)
        a.step(1e-2, t)
        b.step(1e-2, t, dither=[int(x) for x in rng.integers(0, 2 ** 32, 2)])
    e32, e8 = float((W32 - target).norm() / target.norm()), float((W8 - target).norm() / target.norm())
    assert e32 < 0.5 and abs(e8 - e32) < 0.05
    _, v = adamw_moments(s8)
    assert 0.8 < float((v.sum() / s32[1].sum())) < 1.25


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 3], SIZES, [100_003, 1, 7_000_001], [(13 * k) % 97 for k in range(450)]])
@pytest.mark.parametrize("offset", [0, 1])
def test_grad_norm_matches_reference(sizes, dtype, offset):
    _need_gpu()
    g = torch.Generator().manual_seed(3)
    ts = [place(torch.randn(n, generator=g), dtype, offset) for n in sizes]
    norm, factor = T.grad_norm([t.double().cpu().numpy() for t in ts], 2.0)
    op = GradNorm(ts)
    got = op.compute(2.0)
    # squares and sums in fp64, one rounding to fp32
    assert abs(float(got[0]) - norm) <= 2.0 ** -23 * norm and abs(float(got[1]) - factor) <= 2.0 ** -23 * factor
    assert torch.equal(op.compute(2.0), got)


def test_grad_norm_range():
    _need_gpu()
    big = torch.full((1000,), 3e38, device=DEV)
    got = GradNorm([big]).compute(1.0)
    assert torch.isinf(got[0]) and float(got[1]) == pytest.approx(1 / (3e38 * 1000 ** 0.5), rel=1e-5)   # norm past fp32
    small = torch.full((4,), 1e-42, device=DEV)
    assert float(GradNorm([small]).compute(1.0)[0]) == pytest.approx(2e-42, rel=1e-2)
    for x in (float("inf"), float("nan")):
        big[999] = x
        assert torch.isnan(GradNorm([torch.ones(3, device=DEV), big]).compute(1.0)[1])
    zero = GradNorm([torch.zeros(9, device=DEV)]).compute(0.5)
    assert float(zero[0]) == 0 and float(zero[1]) == 1


def test_adamw_offsets_past_32_bits():
    """A tensor whose last elements lie past 2^32 bytes and 2^31 elements."""
    _need_gpu()
    n = (1 << 31) + 4099
    W = torch.zeros(n, dtype=BF16, device=DEV)
    G = torch.zeros(n, dtype=BF16, device=DEV)
    state = adamw_state(W, 8)
    G[-3:] = 1.0
    G[5] = -1.0
    AdamW([(W, G, *state)]).step(0.5, 1)
    assert W[-3:].tolist() == [-0.5] * 3 and float(W[5]) == 0.5 and int((W != 0).sum()) == 4
    norm = GradNorm([G]).compute(1.0)
    assert float(norm[0]) == 2.0
    del state
    m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    AdamW([(W, G, m, v)]).step(0.5, 1)
    assert W[-3:].tolist() == [-1.0] * 3 and float(W[5]) == 1.0 and int((W != 0).sum()) == 4


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_on_another_stream_and_in_a_graph(bits):
    _need_gpu()
    sizes = [300, 5000, 7]
    make = (lambda: tensors32(sizes, F32, BF16, 4)) if bits == 32 else (lambda: tensors8(sizes, F32, BF16, 4))
    a, b = make(), make()
    norm_a, norm_b = GradNorm([t[1] for t in a]), GradNorm([t[1] for t in b])
    opt_a, opt_b = AdamW(a), AdamW(b)
    torch.cuda.synchronize()

    def same():
        for x, y in zip(a, b):
            for s, t in zip(x, y):
                assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))

    opt_a.step(1e-2, 1, scale=norm_a.compute(0.5)[1:], dither=(3, 4))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        opt_b.step(1e-2, 1, scale=norm_b.compute(0.5)[1:], dither=(3, 4))
    torch.cuda.synchronize()
    same()
    out = torch.zeros(2, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm_b.compute(0.5, out=out)
        opt_b.step(1e-2, 2, scale=out[1:], dither=(5, 6))
    for k in range(3):
        for x, y in zip(a, b):
            x[1].add_(0.1)
            y[1].add_(0.1)
        opt_a.step(1e-2, 2, scale=norm_a.compute(0.5)[1:], dither=(5, 6))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same()


def test_wrapper_refusals():
    _need_gpu()
    W, G = torch.zeros(16, device=DEV), torch.zeros(16, device=DEV)
    m, v = adamw_state(W)
    s8 = adamw_state(W, 8)
    for bad in [[], [(W, G, m)], [(W, G, m, v.bfloat16())], [(W, G[:8], m, v)], [(W.half(), G, m, v)], [(W.cpu(), G, m, v)],
                [(W, G, *s8[:3], s8[3][:0])], [(W, G, m, v), (W, G, *s8)], [(W.view(4, 4).t(), G, m, v)],
                [(W, G, m, v), (W, G.bfloat16(), m, v)]]:
        with pytest.raises(ValueError):
            AdamW(bad)
    with pytest.raises(ValueError):
        AdamW([(W, G, m, v)], weight_decay=[0.1, 0.2])
    opt = AdamW([(W, G, m, v)])
    for bad in [dict(lr=float("nan"), t=1), dict(lr=0.1, t=0)]:
        with pytest.raises(hm.HiMuonError):
            opt.step(**bad)
    with pytest.raises(ValueError):
        opt.step(0.1, 1, scale=torch.ones(1))
    with pytest.raises(ValueError):
        opt.set_grads([G[:8]])
    for bad in [[], [W, G.bfloat16()], [W.view(4, 4).t()], [W.half()]]:
        with pytest.raises(ValueError):
            GradNorm(bad)
    with pytest.raises(hm.HiMuonError):
        GradNorm([G]).compute(float("inf"))
    with pytest.raises(ValueError):
        GradNorm([G]).compute(1.0, out=torch.zeros(3, device=DEV))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_table_equals_arguments(bits):
    """The descriptors in a device table (what AdamW uses for many tensors) give the bits of those in the arguments,
    and set_grads reaches the table."""
    _need_gpu()
    sizes = [(37 * k) % 2111 + 1 for k in range(150)]
    make = tensors32 if bits == 32 else tensors8
    a, b = make(sizes, F32, F32, 8), make(sizes, F32, F32, 8)
    opt = AdamW(a, weight_decay=0.1)
    assert opt._table is not None
    opt.step(1e-2, 1, dither=(7, 8))
    stream = torch.cuda.current_stream().cuda_stream
    opt_b = AdamW(b, weight_decay=0.1)
    hm.himuon_adamw_step(opt_b._c, opt_b.cfg, 1, 1e-2, 0, (7, 8), 0, stream)
    new = [torch.randn(n, generator=torch.Generator().manual_seed(n)).to(DEV) for n in sizes]
    opt.set_grads(new)
    opt.step(1e-2, 2, dither=(9, 10))
    for t, g in zip(b, new):
        t[1].copy_(g)
    hm.himuon_adamw_step(opt_b._c, opt_b.cfg, 2, 1e-2, 0, (9, 10), 0, stream)
    for x, y in zip(a, b):
        for k in range(len(x)):
            if k != 1:
                assert torch.equal(x[k].view(torch.uint8), y[k].view(torch.uint8))


@pytest.mark.parametrize("gt", [F32, BF16])
def test_adamw8_states_are_those_of_the_formulas_in_fp32(gt):
    """The 8-bit states bit for bit: numpy float32 operations (each correctly rounded) in the documented order."""
    _need_gpu()
    f = np.float32
    sizes = [1, 255, 256, 5001, 70000]
    ts = tensors8(sizes, F32, gt, 77)
    opt = AdamW(ts, betas=(0.9, 0.999))
    scale = torch.tensor([0.37], device=DEV)
    table = T.e4m3_values().astype(f)
    for t, dither in ((1, (11, 0xFEDCBA98)), (2, (0x9ABCDEF0, 5))):
        before = [[x.clone() for x in q] for q in ts]
        opt.step(1e-3, t, scale=scale, dither=dither)
        for b, a in zip(before, ts):
            n = b[0].numel()
            g = b[1].float().cpu().numpy() * f(0.37)
            m_unit, r_unit = (np.repeat(x.cpu().numpy(), T.BLOCK)[:n] for x in b[4:])
            m = table[b[2].view(torch.uint8).cpu().numpy()] * m_unit
            r = table[b[3].view(torch.uint8).cpu().numpy()] * r_unit
            m = f(0.9) * m + f(1 - 0.9) * g
            r = np.sqrt(f(0.999) * (r * r) + f(1 - 0.999) * g * g)
            for k, x in enumerate((m, r)):
                i = np.arange(n, dtype=np.uint64)
                d = ((i * T.MULT[k] + dither[k]) % 2 ** 32 >> np.uint64(16)).astype(np.uint32) << np.uint32(4) | np.uint32(8)
                pad = np.zeros(-n % T.BLOCK, f)
                peak = np.abs(np.concatenate([x, pad])).reshape(-1, T.BLOCK).max(1)
                inv = np.repeat(f(1) / peak * f(448), T.BLOCK)[:n]
                y = np.abs(x) * inv
                low = np.where(y < f(2 ** -6), f(2 ** -6), f(0))
                y = (((y + low).view(np.uint32) + d) & np.uint32(0xFFF00000)).view(f) - low
                y = np.clip(y, f(2 ** -9) if k else f(0), f(448)) * np.sign(x)
                assert np.array_equal(table[a[2 + k].view(torch.uint8).cpu().numpy()], y)
                assert np.array_equal(a[4 + k].cpu().numpy(), peak * f(1 / 448))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("wt,gt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
def test_adamw_large_call_equals_small_calls(bits, wt, gt):
    """A call of many bytes (which goes past the caches) gives the bits of calls on its tensors one by one."""
    _need_gpu()
    g = torch.Generator(device=DEV).manual_seed(3)
    sizes = [4_000_003, 3, 4_000_000, 3_999_744]
    a = []
    for n in sizes:
        W = torch.randn(n, device=DEV, generator=g).to(wt)
        a.append((W, torch.randn(n, device=DEV, generator=g).to(gt), *adamw_state(W, bits)))
    b = [tuple(x.clone() for x in t) for t in a]
    for t in (1, 2):
        AdamW(a, weight_decay=0.1).step(1e-2, t, dither=(t, 5))
        for x in b:
            AdamW([x], weight_decay=0.1).step(1e-2, t, dither=(t, 5))
    for x, y in zip(a, b):
        for s, u in zip(x, y):
            assert torch.equal(s.view(torch.uint8), u.view(torch.uint8))


def test_grad_norm_of_nothing():
    _need_gpu()
    got = GradNorm([torch.zeros(0, device=DEV), torch.zeros(0, device=DEV)]).compute(0.5)
    assert got.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_subnormal_second_moments(bits):
    """Gradients whose squares are subnormal in fp32, and an eps below their roots: the first step is lr times the
    sign, as the formula says, within what a subnormal of 2^-149's multiples resolves: v = 1e-3 g^2 lies within 1 %
    of a multiple of 2^-149 for these g, so its root is within 1 %."""
    _need_gpu()
    unit = 2.0 ** -149
    v = torch.arange(100, 1124, dtype=torch.float64) * unit
    G = torch.sqrt(v / (1 - 0.999)).float().to(DEV)
    W = torch.zeros(1024, device=DEV)
    state = adamw_state(W, bits)
    AdamW([(W, G, *state)], eps=1e-30).step(1e-2, 1, dither=(1, 2))
    assert ((W + 1e-2).abs() <= 1e-2 * 0.01).all()
