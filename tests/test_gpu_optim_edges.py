"""AdamWOptimizer and HiMuonOptimizer where a training program does the unusual (MI355X only):
states that are replaced, refused factors."""
import pytest
import torch

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.optim import AdamWOptimizer, HiMuonOptimizer  # noqa: E402

DEV = "cuda"
SHAPES = [(7,), (300, 170), (1,), (64, 3, 3), (5000,)]


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def params(seed, shapes=SHAPES):
    g = torch.Generator().manual_seed(seed)
    return [torch.nn.Parameter(torch.randn(s, generator=g).to(DEV)) for s in shapes]


def set_grads(ps, seed):
    g = torch.Generator().manual_seed(seed)
    for p in ps:
        p.grad = torch.randn(p.shape, generator=g).to(DEV)


def same_states(x, a, y, b):
    for p, q in zip(a, b):
        assert torch.equal(p, q) and x.state[p]["step"] == y.state[q]["step"]
        for s, t in zip(x.state[p]["adamw"], y.state[q]["adamw"]):
            assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_optimizer_takes_states_that_were_replaced(bits):
    """A program that clears the optimizer's state starts anew with it, and not with the moments of before."""
    _need_gpu()
    a = params(1)
    x = AdamWOptimizer(a, lr=1e-2, state_bits=bits)
    for step in range(2):
        set_grads(a, step)
        x.step()
    b = [torch.nn.Parameter(p.detach().clone()) for p in a]
    y = AdamWOptimizer(b, lr=1e-2, state_bits=bits)
    y._random.setstate(x._random.getstate())
    x.state.clear()
    for step in range(2, 4):
        set_grads(a, step)
        set_grads(b, step)
        x.step()
        y.step()
        same_states(x, a, y, b)


def bad_factors():
    one = torch.ones(1, device=DEV)
    return [0.5, one.double(), one.cpu(), one[:0], one.bfloat16()]


@pytest.mark.parametrize("which", range(5))
def test_refused_factor_changes_nothing(which):
    _need_gpu()
    bad = bad_factors()[which]
    ps = params(2, [(300, 170), (128, 64), (77,)])
    opt = HiMuonOptimizer(ps, lr=0.02, tile=64, fallback=lambda q: AdamWOptimizer(q, lr=1e-2))
    set_grads(ps, 0)
    opt.step()
    set_grads(ps, 1)
    before = [p.detach().clone() for p in ps] + [opt.momentum(p).clone() for p in ps[:2]]
    with pytest.raises(ValueError):
        opt.step(grad_scale=bad)
    with pytest.raises(ValueError):
        opt.fallback.step(grad_scale=bad)
    torch.cuda.synchronize()
    for x, y in zip(before, [*ps, *(opt.momentum(p) for p in ps[:2])]):
        assert torch.equal(x, y)
    assert opt.step_count == 1 and opt.fallback.state[ps[2]]["step"] == 1
    opt.close()
