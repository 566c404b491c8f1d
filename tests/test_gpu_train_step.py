"""The training step around HiMuon on the GPU (MI355X only): AdamWOptimizer against torch's
AdamW, its parameter groups, late gradients and saved states, the clip factor through
HiMuonOptimizer, and the example that runs the loss, the norm, HiMuon and AdamW together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.adamw import GradNorm, adamw_moments  # noqa: E402
from tiled_newton_schulz_tile_amd.optim import AdamWOptimizer, HiMuonOptimizer  # noqa: E402

DEV = "cuda"
SHAPES = [(7,), (300, 170), (1,), (64, 3, 3), (5000,)]


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def params(seed, dtype=torch.float32, shapes=SHAPES):
    g = torch.Generator().manual_seed(seed)
    return [torch.nn.Parameter(torch.randn(s, generator=g).to(dtype).to(DEV)) for s in shapes]


def set_grads(ps, seed):
    g = torch.Generator().manual_seed(seed)
    for p in ps:
        p.grad = torch.randn(p.shape, generator=g).to(p.dtype).to(DEV)


def test_adamw_optimizer_is_torchs():
    """Ten steps with two groups, new gradient tensors each step, a changed lr and a parameter whose gradient comes
    late: parameters stay within the two fp32 computations' rounding (2^-20 of the steps' sum, and of the weight)."""
    _need_gpu()
    a, b = params(1), params(1)
    make = lambda cls, ps: cls([{"params": ps[:3], "weight_decay": 0.0}, {"params": ps[3:], "lr": 3e-3}],  # noqa: E731
                               lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    mine, theirs = make(AdamWOptimizer, a), make(torch.optim.AdamW, b)
    for step in range(10):
        for opt, ps in ((mine, a), (theirs, b)):
            set_grads(ps, 100 + step)
            if step < 3:
                ps[1].grad = None
            opt.param_groups[0]["lr"] = 1e-2 / (1 + step)
            opt.step()
            opt.zero_grad()
    for p, q in zip(a, b):
        assert ((p - q).abs() <= 2.0 ** -20 * (0.1 + q.abs())).all()


def test_adamw_optimizer_bf16_and_strided_gradients():
    _need_gpu()
    a, b = params(2, torch.bfloat16, [(33, 65)]), params(2, torch.bfloat16, [(33, 65)])
    mine, other = AdamWOptimizer(a, lr=1e-2, weight_decay=0.0), AdamWOptimizer(b, lr=1e-2, weight_decay=0.0)
    for step in range(3):
        g = torch.randn(65, 33, generator=torch.Generator().manual_seed(step)).bfloat16().to(DEV)
        a[0].grad, b[0].grad = g.t(), g.t().contiguous()   # a gradient whose rows are its parameter's columns
        mine.step()
        other.step()
        assert torch.equal(a[0], b[0])
    assert not torch.equal(a[0], params(2, torch.bfloat16, [(33, 65)])[0])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_adamw_optimizer_saved_states_resume_bit_for_bit(bits, dtype):
    _need_gpu()
    a = params(3, dtype)
    one = AdamWOptimizer(a, lr=1e-2, state_bits=bits, seed=5)
    for step in range(3):
        set_grads(a, step)
        one.step()
    b = [torch.nn.Parameter(p.detach().clone()) for p in a]
    two = AdamWOptimizer(b, lr=1e-2, state_bits=bits, seed=99)
    two.load_state_dict(one.state_dict())
    for step in range(3, 6):
        for opt, ps in ((one, a), (two, b)):
            set_grads(ps, step)
            opt.step()
    for p, q in zip(a, b):
        assert torch.equal(p, q)
        for s, t in zip(one.state[p]["adamw"], two.state[q]["adamw"]):
            assert s.dtype == t.dtype and torch.equal(s.view(torch.uint8), t.view(torch.uint8))
    with pytest.raises(ValueError):
        AdamWOptimizer(b, state_bits=40 - bits).load_state_dict(one.state_dict())


def test_adamw_optimizer_8_bit_moments_track_32_bit():
    """The moments after 50 steps of the same gradients, on average over 100 000 elements: the dithered rounding
    keeps m's mean (its spread is a few per cent of |m|: the sum's error is below 1 % of the sum of magnitudes) and
    raises v's by the variance of the root's rounding, a few per cent."""
    _need_gpu()
    a, b = params(4, shapes=[(100_000,)]), params(4, shapes=[(100_000,)])
    x, y = AdamWOptimizer(a, lr=1e-3), AdamWOptimizer(b, lr=1e-3, state_bits=8)
    for step in range(50):
        for opt, ps in ((x, a), (y, b)):
            set_grads(ps, step)
            opt.step()
    m, v = adamw_moments(x.state[a[0]]["adamw"])
    m8, v8 = adamw_moments(y.state[b[0]]["adamw"])
    assert float((m8 - m).sum().abs() / m.abs().sum()) < 0.01
    assert 0.95 < float(v8.sum() / v.sum()) < 1.15
    x, y, w = (p.detach() for p in (a[0], b[0], params(4, shapes=[(100_000,)])[0]))
    assert float((y - x).norm() / (x - w).norm()) < 0.2


def test_optimizer_refuses():
    _need_gpu()
    for bad in [[torch.nn.Parameter(torch.zeros(3))], [torch.nn.Parameter(torch.zeros(4, 4, device=DEV).t()[1:])],
                [torch.nn.Parameter(torch.zeros(3, device=DEV).half())]]:
        with pytest.raises(ValueError):
            AdamWOptimizer(bad)
    with pytest.raises(ValueError):
        AdamWOptimizer(params(1), state_bits=16)
    ps = params(1, shapes=[(64, 64), (64,)])
    set_grads(ps, 1)
    opt = HiMuonOptimizer(ps, tile=64)
    with pytest.raises(ValueError):
        opt.step(grad_scale=torch.ones(1, device=DEV))   # torch's AdamW takes no factor
    opt.close()


@pytest.mark.parametrize("bits", [32, 8])
def test_clip_factor_through_himuon_optimizer(bits):
    """A factor on the device equals gradients scaled beforehand; NaN leaves AdamW's parameters and states, and
    HiMuon's momentum decays as for a zero gradient."""
    _need_gpu()
    shapes = [(300, 170), (128, 512), (77,), (5000,)]
    a, b = params(6, shapes=shapes), params(6, shapes=shapes)
    make = lambda ps: HiMuonOptimizer(ps, lr=0.02, tile=64, state_dtype=torch.float32,  # noqa: E731
                                      precision=hm.PREC_F32,
                                      fallback=lambda q: AdamWOptimizer(q, lr=1e-2, state_bits=bits, seed=1))
    x, y = make(a), make(b)
    for step in range(3):
        set_grads(a, step)
        set_grads(b, step)
        factor = torch.full((2,), 0.25, device=DEV)   # a power of two: scaling beforehand is exact
        x.step(grad_scale=factor[1:])
        for p in b:
            p.grad.mul_(0.25)
        y.step()
        for p, q in zip(a, b):
            assert torch.equal(p, q)
    set_grads(a, 9)
    a[0].grad[3, 3] = float("inf")
    before = [p.detach().clone() for p in a]
    moment = x.momentum(a[0]).clone()
    got = GradNorm([p.grad for p in a]).compute(1.0)
    x.step(grad_scale=got[1:])
    assert torch.isnan(got[1]) and all(torch.isfinite(p).all() for p in a)
    for p, q in list(zip(a, before))[2:]:
        assert torch.equal(p, q)
    assert torch.equal(x.momentum(a[0]), moment * 0.95)
    x.close()
    y.close()


@pytest.mark.parametrize("bits", [32, 8])
def test_example_learns_by_reward(bits):
    _need_gpu()
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "policy_finetune.py")
    spec = importlib.util.spec_from_file_location("policy_finetune", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    first, last = mod.train(steps=50, state_bits=bits, log=None)
    assert last > 2 * first


def test_adamw_optimizer_follows_moved_parameters():
    """A parameter whose storage is replaced between steps is updated where it is now."""
    _need_gpu()
    a, b = params(7), params(7)
    x, y = AdamWOptimizer(a, lr=1e-2), AdamWOptimizer(b, lr=1e-2)
    for step in range(4):
        if step == 2:
            old = a[1].data
            a[1].data = old.clone()
            old.fill_(5.0)
        set_grads(a, step)
        set_grads(b, step)
        x.step()
        y.step()
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    assert (old == 5).all()


def test_adamw_set_grads_and_graphs():
    """Gradients of a call with a device table are set before a graph is captured (inside, set_grads refuses and the
    capture goes on); the replays take them."""
    _need_gpu()
    from tiled_newton_schulz_tile_amd.adamw import AdamW, adamw_state
    sizes = [100 + k for k in range(20)]
    g = torch.Generator().manual_seed(0)
    W = [torch.randn(n, generator=g).to(DEV) for n in sizes]
    V = [w.clone() for w in W]
    G1, G2 = ([torch.randn(n, generator=g).to(DEV) for n in sizes] for _ in range(2))
    sw, sv = [adamw_state(w) for w in W], [adamw_state(v) for v in V]
    opt = AdamW([(w, x, *s) for w, x, s in zip(W, G1, sw)])
    ref = AdamW([(v, x, *s) for v, x, s in zip(V, G2, sv)])
    opt.set_grads(G2)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError):
            opt.set_grads(G1)
        opt.step(1e-2, 1)
    for _ in range(3):
        graph.replay()
        ref.step(1e-2, 1)
        torch.cuda.synchronize()
        for w, v in zip(W, V):
            assert torch.equal(w, v)
