"""The operators on token distributions run together, as a post-training step has them (MI355X only): a policy draws tokens,
the policy loss takes them with their log probabilities, a teacher's top logits are distilled into the same
logits, and the gradients of both go through the model to GradNorm, HiMuon and AdamW."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
hm = pytest.importorskip("tiled_newton_schulz_tile_amd")
from tiled_newton_schulz_tile_amd.adamw import GradNorm  # noqa: E402
from tiled_newton_schulz_tile_amd.distill import distill_loss, top_logits  # noqa: E402
from tiled_newton_schulz_tile_amd.optim import AdamWOptimizer, HiMuonOptimizer  # noqa: E402
from tiled_newton_schulz_tile_amd.policy import policy_loss  # noqa: E402
from tiled_newton_schulz_tile_amd.sampling import sample  # noqa: E402

T = 1.5   # the distillation's temperature


def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def batch(N, V, width, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, width, generator=g)
    head, bias, teacher = (torch.randn(*s, generator=g) / width ** 0.5 for s in ((V, width), (V,), (V, width)))
    u, adv, weight = torch.rand(N, generator=g), torch.randn(N, generator=g), torch.rand(N, generator=g) / N
    weight[::5] = 0   # rows that are left out
    return [t.cuda() for t in (x, 2 * head, bias, 3 * teacher, u, adv, weight)]


def gradient_of(logits, teacher_logits, u, adv, weight, k):
    """What a step makes of its logits: the draw, and the gradient of both losses (the second over its own logits)."""
    drawn = sample(logits, u, temperature=1.0, top_p=0.9)
    first = policy_loss(logits, drawn.token, weight, adv, old_logp=drawn.logp)
    top = top_logits(teacher_logits, k, temperature=T)
    copy = logits.clone()
    second = distill_loss(copy, top.value, top.index, weight, top.rest, temperature=T, grad_scale=T * T, dlogits=copy)
    return drawn, first, second, first.dlogits + second.dlogits


@pytest.mark.parametrize("N,V,k", [(6, 509, 20), (150, 1031, 40), (70, 33003, 128)])
def test_step_matches_autograd(N, V, k):
    """The losses are torch's of the same formulas, in 64 bits on the CPU, and so is the model's gradient.  A logit's
    gradient is a probability times a weight of 1 / N and a factor of a few (advantages, T), each within about 2^-20 of
    itself in fp32 (exponents of 20 or less); an entry of head's gradient sums N of them times x in fp32, so 2^-18 of the
    sum of their sizes bounds it."""
    _need_gpu()
    x, head, bias, teacher, u, adv, weight = batch(N, V, 64, V)
    head.requires_grad_()
    logits = x @ head.t() + bias
    drawn, first, second, grad = gradient_of(logits.detach(), x @ teacher.t(), u, adv, weight, k)
    logits.backward(grad)

    z = logits.detach().double().cpu().requires_grad_()
    w, a, t = weight.double().cpu(), adv.double().cpu(), (x @ teacher.t()).double().cpu()
    logp = torch.log_softmax(z, 1)
    taken = logp.gather(1, drawn.token.cpu()[:, None])[:, 0]
    policy = -(w * a * (taken - taken.detach()).exp()).sum()
    q = torch.softmax(t / T, 1)
    p = torch.log_softmax(z / T, 1)
    value, index = t.topk(k)
    named = torch.zeros_like(q).scatter_(1, index, 1.0).bool()
    q_rest, p_rest = (q * ~named).sum(1), p.masked_fill(named, -math.inf).logsumexp(1)
    kl = torch.where(named, q * (q.log() - p), torch.zeros_like(q)).sum(1) + q_rest * (q_rest.log() - p_rest)
    (policy + T * T * (w * kl).sum()).backward()

    assert torch.allclose(drawn.logp.double().cpu(), taken.detach(), rtol=0, atol=2.0 ** -18)
    assert abs(float(first.loss) - policy.item()) <= 2.0 ** -18 * float((w * a.abs()).sum())
    assert abs(float(second.loss) - (w * kl).sum().item()) <= 2.0 ** -18 * (w * kl).sum().item() + 2.0 ** -20
    sizes = z.grad.abs().t() @ x.double().cpu().abs()
    error = (head.grad.double().cpu() - z.grad.t() @ x.double().cpu()).abs()
    assert (error <= 2.0 ** -18 * sizes + 2.0 ** -22 * float(sizes.max())).all()
    assert (grad[weight == 0] == 0).all()


def test_steps_run_and_repeat():
    """Steps run through HiMuon, AdamW and the clip factor, with finite weights, and repeat bit for bit."""
    _need_gpu()
    runs = []
    for _ in range(2):
        x, head, bias, teacher, u, adv, weight = batch(256, 509, 64, 3)
        head, bias = torch.nn.Parameter(head), torch.nn.Parameter(bias)
        opt = HiMuonOptimizer([{"params": [head]}, {"params": [bias], "use_himuon": False}], lr=0.01, tile=64,
                              fallback=lambda ps: AdamWOptimizer(ps, lr=1e-2, weight_decay=0.0))
        norm, kl = None, []
        for _ in range(8):
            logits = x @ head.t() + bias
            drawn, _, second, grad = gradient_of(logits.detach(), x @ teacher.t(), u, adv, weight, 32)
            opt.zero_grad()
            logits.backward(grad)
            if norm is None:
                norm = GradNorm([head.grad, bias.grad])
            else:
                norm.set_grads([head.grad, bias.grad])
            opt.step(grad_scale=norm.compute(max_norm=1.0)[1:])
            kl.append(second.kl)
        torch.cuda.synchronize()
        opt.close()
        runs.append((head.detach().clone(), bias.detach().clone(), drawn.token.clone(), torch.stack(kl)))
    for a, b in zip(*runs):
        assert torch.equal(a, b) and torch.isfinite(a.double()).all()


@pytest.mark.parametrize("N,V", [(6, 509), (150, 5003), (64, 33003), (9, 70001), (4200, 1031)])
def test_step_in_a_graph(N, V):
    """All of it captured, and replayed on new logits between eager calls: every replay is the eager result."""
    _need_gpu()
    x, head, bias, teacher, u, adv, weight = batch(N, V, 64, V + 1)
    logits, wanted = x @ head.t() + bias, x @ teacher.t()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gradient_of(logits, wanted, u, adv, weight, 16)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gradient_of(logits, wanted, u, adv, weight, 16)
    for seed in range(4):
        x, head, bias, teacher, u2, *_ = batch(N, V, 64, seed)
        logits.copy_(x @ head.t() + bias)
        wanted.copy_(x @ teacher.t())
        u.copy_(u2)
        graph.replay()
        torch.cuda.synchronize()
        eager = gradient_of(logits, wanted, u, adv, weight, 16)
        for a, b in zip(got, eager):
            for s, t in zip(a if isinstance(a, tuple) else (a,), b if isinstance(b, tuple) else (b,)):
                assert torch.equal(s, t)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,V", [(1, 131077), (31, 65601), (33, 70003), (64, 65601)])
def test_spans_and_rows_of_the_distillation_loss(N, V, dtype):
    """Few long rows are cut into spans, by other numbers of them with a gradient and without one: in place and not, the
    gradient is the same, and the divergences of both agree.  A divergence is an fp64 sum of terms q (log q - log p); the
    sum over the rest in them is fp32 in another order: V terms in trees and runs of 32 or fewer, so within 40 2^-24
    of itself, and its logarithm by that much, times the rest's probability of at most 1."""
    _need_gpu()
    g = torch.Generator().manual_seed(V)
    z = (4 * torch.randn(N, V, generator=g)).to(dtype).cuda()
    top = top_logits(z.flip(1).contiguous(), 50)
    weight = torch.rand(N, generator=g).cuda()
    got = distill_loss(z, top.value, top.index, weight, top.rest)
    forward = distill_loss(z, top.value, top.index, weight, top.rest, dlogits=False)
    copy = z.clone()
    again = distill_loss(copy, top.value, top.index, weight, top.rest, dlogits=copy)
    assert torch.equal(got.dlogits, copy) and torch.equal(got.kl, again.kl) and torch.equal(got.loss, again.loss)
    assert ((got.kl - forward.kl).abs() <= 40 * 2.0 ** -24 + 2.0 ** -23 * got.kl.abs()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_greedy_rows_of_equal_logits(dtype):
    """Temperature 0 without a filter takes the first of a row's equal largest logits, for every number of rows."""
    _need_gpu()
    for N, V in ((3, 20000), (300, 20000), (5000, 2500)):
        z = torch.zeros(N, V, dtype=dtype, device="cuda")
        z[:, :7] = -1
        z[::2, V // 2:] = 1
        want = torch.full((N,), 7, device="cuda")
        want[::2] = V // 2
        u = torch.rand(N, device="cuda")
        assert torch.equal(sample(z, u, temperature=0.0).token, want)
        assert torch.equal(sample(z, u, temperature=torch.zeros(N, device="cuda")).token, want)
