"""AdamWOptimizer and HiMuonOptimizer where a training program does the unusual (MI355X only):
states that are replaced, refused factors, parameters whose gradients come and go, copies,
skipped steps, refused states, and what autograd has to know of writes that it does not make."""
import copy

import pytest
import torch

from oracle import training as T

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.optim import AdamWOptimizer, HiMuonOptimizer  # noqa: E402
from tiled_newton_schulz_tile_amd.policy import policy_loss  # noqa: E402

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


def test_parameters_whose_gradients_come_and_go():
    """Another set of parameters at nearly every step (routed experts): what the optimizer keeps for its calls stays
    bounded, and the parameters are torch's (within the two fp32 computations' rounding, as in a usual run)."""
    _need_gpu()
    shapes = [(40 + k,) for k in range(12)]
    a, b = params(3, shapes), params(3, shapes)
    x, y = AdamWOptimizer(a, lr=1e-2, weight_decay=0.1), torch.optim.AdamW(b, lr=1e-2, weight_decay=0.1)
    g = torch.Generator().manual_seed(0)
    sets = set()
    for step in range(60):
        take = torch.rand(12, generator=g) < 0.5
        sets.add(tuple(take.tolist()))
        for opt, ps in ((x, a), (y, b)):
            set_grads(ps, step)
            for p, t in zip(ps, take.tolist()):
                if not t:
                    p.grad = None
            opt.step()
    assert len(sets) > 50 and len(x._engines) <= 32
    for p, q in zip(a, b):
        assert ((p - q).abs() <= 2.0 ** -20 * (0.6 + q.abs())).all()


def test_many_groups_keep_their_descriptors():
    _need_gpu()
    ps = params(8, [(5,)] * 50)
    opt = AdamWOptimizer([{"params": [p]} for p in ps], lr=1e-2)
    kept = []
    for step in range(3):
        set_grads(ps, step)
        opt.step()
        kept.append({key: held[0] for key, held in opt._engines.items()})
    assert len(kept[0]) == 50 and all(k == kept[0] for k in kept)


@pytest.mark.parametrize("bits", [32, 8])
def test_copied_optimizer_goes_on_alone(bits):
    _need_gpu()
    a = params(4)
    x = AdamWOptimizer(a, lr=1e-2, state_bits=bits, seed=3)
    for step in range(2):
        set_grads(a, step)
        x.step()
    y = copy.deepcopy(x)
    b = y.param_groups[0]["params"]
    assert all(p is not q for p, q in zip(a, b))
    for step in range(2, 4):
        set_grads(a, step)
        set_grads(b, step)
        x.step()
        y.step()
        same_states(x, a, y, b)
    assert all(s.data_ptr() != t.data_ptr() for p, q in zip(a, b)
               for s, t in zip(x.state[p]["adamw"], y.state[q]["adamw"]))


def test_autograd_sees_the_gradient_written_over_logits():
    """A backward pass that saved the logits (a tanh cap keeps its output) raises torch's error and does not take the
    gradient for them; logits that nothing saved may be written over."""
    _need_gpu()
    g = torch.Generator().manual_seed(0)
    z = torch.randn(6, 50, generator=g).to(DEV).requires_grad_()
    label, w, adv = torch.arange(6, device=DEV), torch.ones(6, device=DEV), torch.ones(6, device=DEV)
    logits = torch.tanh(z)
    got = policy_loss(logits.detach(), label, w, adv, dlogits=logits.detach())
    with pytest.raises(RuntimeError):
        logits.backward(got.dlogits)
    logits = z * 2
    want = policy_loss(logits.detach(), label, w, adv).dlogits
    got = policy_loss(logits.detach(), label, w, adv, dlogits=logits.detach())
    logits.backward(got.dlogits)
    assert torch.equal(z.grad, want * 2)
    with torch.inference_mode():   # (tensors without a version)
        t = z.detach().clone()
        assert torch.equal(policy_loss(t, label, w, adv, dlogits=t).dlogits, policy_loss(z.detach(), label, w, adv).dlogits)


def test_autograd_sees_a_step():
    _need_gpu()
    p = torch.nn.Parameter(torch.ones(100, device=DEV))
    opt = AdamWOptimizer([p], lr=1e-2)
    loss = (p * p).sum()
    p.grad = torch.ones(100, device=DEV)
    opt.step()
    with pytest.raises(RuntimeError):
        loss.backward()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_skipped_step_counts_and_changes_nothing_else(bits):
    """The step after a skipped first one is the formula's with t = 2 on zero moments, within the kernel's 2^-18 of
    the step and 2^-22 of the weight."""
    _need_gpu()
    p = torch.nn.Parameter(torch.randn(1000, generator=torch.Generator().manual_seed(1)).to(DEV))
    w = p.detach().double().cpu().numpy()
    opt = AdamWOptimizer([p], lr=1e-2, weight_decay=0.1, state_bits=bits)
    set_grads([p], 0)
    opt.step(grad_scale=torch.full((1,), float("nan"), device=DEV))
    assert (p.detach().double().cpu().numpy() == w).all() and opt.state[p]["step"] == 1
    assert not any(s.view(torch.uint8).any() for s in opt.state[p]["adamw"])
    set_grads([p], 1)
    opt.step()
    want, _, _ = T.adamw(w, p.grad.double().cpu().numpy(), 0 * w, 0 * w, 2, 1e-2, weight_decay=0.1)
    got = p.detach().double().cpu().numpy()
    assert (abs(got - want) <= 2.0 ** -18 * 1e-2 + 2.0 ** -22 * abs(w)).all()
    full, _, _ = T.adamw(w, p.grad.double().cpu().numpy(), 0 * w, 0 * w, 1, 1e-2, weight_decay=0.1)
    decayed = w * (1 - 1e-3)
    assert abs((want - decayed) / (full - decayed) - 0.744).max() < 1e-3   # the documented size


@pytest.mark.parametrize("bits", [32, 8])
def test_refused_states_leave_the_optimizer_as_it_was(bits):
    """States of the other kind, of another shape or type, and of another optimizer."""
    _need_gpu()
    a, b = params(5), params(5)
    x, y = AdamWOptimizer(a, lr=1e-2, state_bits=bits), AdamWOptimizer(b, lr=1e-2, state_bits=bits)
    other = AdamWOptimizer(params(5), lr=0.5, state_bits=40 - bits)
    torchs = torch.optim.AdamW(params(5), lr=0.5)
    short = AdamWOptimizer(params(5, [(7,), (300, 171), (1,), (64, 3, 3), (5000,)]), lr=0.5, state_bits=bits)
    for opt in (x, y, other, torchs, short):
        set_grads(opt.param_groups[0]["params"], 0)
        opt.step()
    cast = copy.deepcopy(x.state_dict())
    cast["state"][4]["adamw"] = tuple(s.double() for s in cast["state"][4]["adamw"])
    for sd in (other.state_dict(), torchs.state_dict(), short.state_dict(), cast):
        with pytest.raises(ValueError):
            x.load_state_dict(sd)
        same_states(x, a, y, b)
    assert x.param_groups[0]["lr"] == 1e-2
    for opt, ps in ((x, a), (y, b)):
        set_grads(ps, 1)
        opt.step()
    same_states(x, a, y, b)
