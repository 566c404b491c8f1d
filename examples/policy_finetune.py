"""Post-training a small token policy with every operator of the library's training step.

    python examples/policy_finetune.py [--steps 60] [--state-bits 8]

A two-layer network over a window of tokens learns by reward alone to continue sequences
by a fixed rule: it samples answers, scores them, and takes a few steps of the clipped
policy loss with a KL term to the starting policy on each batch (policy_loss gives the
gradient of the logits, torch the rest of the backward pass).  The gradient's norm and clip
factor stay on the device (GradNorm); the matrices are updated by HiMuon and everything else
(embedding, gains, biases) by the library's AdamW.  Synthetic data, random weights.
"""
import argparse
import copy
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import tiled_newton_schulz_tile_amd as hm  # noqa: E402
from tiled_newton_schulz_tile_amd.adamw import GradNorm  # noqa: E402
from tiled_newton_schulz_tile_amd.optim import AdamWOptimizer, HiMuonOptimizer  # noqa: E402
from tiled_newton_schulz_tile_amd.policy import policy_loss  # noqa: E402

VOCAB, WINDOW, WIDTH = 509, 3, 256


class Policy(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.embed = torch.nn.Parameter(0.5 * torch.randn(VOCAB, WIDTH))
        self.up = torch.nn.Parameter(torch.randn(2 * WIDTH, WINDOW * WIDTH) / (WINDOW * WIDTH) ** 0.5)
        self.gain = torch.nn.Parameter(torch.ones(2 * WIDTH))
        self.head = torch.nn.Parameter(torch.randn(VOCAB, 2 * WIDTH) / (2 * WIDTH) ** 0.5)
        self.bias = torch.nn.Parameter(torch.zeros(VOCAB))

    def forward(self, window):
        x = self.embed[window].flatten(1) @ self.up.t()
        x = torch.nn.functional.silu(x) * self.gain
        return x @ self.head.t() + self.bias


def rule(window):
    return window[:, 1] // 8 * 8   # the token that earns the reward: one of 64


def train(steps=60, state_bits=8, rows=2048, epochs=2, seed=0, log=print):
    """Mean rewards before and after, of sampled tokens."""
    torch.manual_seed(seed)
    model = Policy().cuda()
    reference = copy.deepcopy(model)   # the policy that the KL term holds on to
    matrices = [model.up, model.head]
    opt = HiMuonOptimizer([{"params": matrices}, {"params": [model.embed, model.gain, model.bias], "use_himuon": False}],
                          lr=0.02, tile=128, fallback=lambda ps: AdamWOptimizer(ps, lr=3e-3, weight_decay=0.0,
                                                                                state_bits=state_bits))
    norm, rewards = None, []
    for step in range(steps):
        window = torch.randint(0, VOCAB, (rows, WINDOW), device="cuda")
        with torch.no_grad():
            logits = model(window)
            token = torch.distributions.Categorical(logits=logits).sample()
            # a dense reward: how near the answer is to the rule's
            gap = (token - rule(window)).abs().float() / VOCAB
            reward = torch.exp(-8 * gap)
            rewards.append(reward.mean())
            advantage = (reward - reward.mean()) / (reward.std() + 1e-6)
            weight = torch.full((rows,), 1.0 / rows, device="cuda")
            old = policy_loss(logits, token, weight, advantage, dlogits=False).logp
            ref = policy_loss(reference(window), token, weight, advantage, dlogits=False).logp
        for _ in range(epochs):
            logits = model(window)
            got = policy_loss(logits.detach(), token, weight, advantage, old_logp=old, ref_logp=ref, clip=(0.2, 0.28),
                              kl_coef=0.002)
            opt.zero_grad()
            logits.backward(got.dlogits)
            grads = [p.grad for p in model.parameters()]
            if norm is None:
                norm = GradNorm(grads)
            else:
                norm.set_grads(grads)
            factor = norm.compute(max_norm=1.0)
            opt.step(grad_scale=factor[1:])
        if log and step % 10 == 9:
            log(f"step {step + 1}: reward {float(rewards[-1]):.3f} loss {float(got.loss):+.4f} "
                f"clipped {float(got.stats[3]):.3f} gradient norm {float(factor[0]):.3f}")
    opt.close()
    return float(rewards[0]), float(rewards[-1])


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    first, last = train(a.steps, a.state_bits)
    print(f"mean reward {first:.3f} -> {last:.3f} ({hm.library_path()})")
