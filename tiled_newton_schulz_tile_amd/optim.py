"""torch.optim integration of the HiMuon step.

"Hierarchical Muon: Tiled Newton-Schulz Updates for Efficient Muon Optimization"
(Abstract) applies the tiled Newton-Schulz map to the momentum-gradient matrices of
dense weights and names runtime tile-size schedules among what the tiling allows.
Which parameters count as such matrices, and what updates the rest, is not on the
pages; the convention here: every 2-D parameter goes through HiMuon, every other
parameter through a plain torch optimizer (AdamW unless one is given; AdamWOptimizer below
is this library's own, one launch over all of them, with 32-bit or 8-bit states).  A parameter
group can opt out with ``use_himuon=False``.  HiMuon parameters that share a learning
rate share one plan (one launch per kernel covers all of their layers); groups with
their own ``lr`` get a plan each, and the step reads every group's current ``lr``, so
learning-rate schedulers work as usual.

The HiMuon state lives on the device: fp32 weights are the parameters themselves, the
momentum is ``state[p]["momentum_buffer"]`` (the state dtype, saved and restored by
``state_dict`` / ``load_state_dict``), and the gradient is copied into a persistent
buffer of that dtype each step (torch may hand out a new .grad tensor every backward
pass, while the plan holds device pointers).
"""
from __future__ import annotations

import bisect
import random

import torch

from . import ADAMW_BLOCK, HiMuon, PREC_BF16X3, QUINTIC
from .adamw import AdamW, adamw_state


class TileSchedule:
    """Tile size as a function of the optimizer step: a list of (first_step, T) pairs in
    increasing first_step, the first at step 0; T = 0 is FULL.  A plain int is a constant
    schedule."""

    def __init__(self, spec):
        if isinstance(spec, int):
            spec = [(0, spec)]
        spec = [(int(s), int(t)) for s, t in spec]
        if not spec or spec[0][0] != 0:
            raise ValueError("the schedule must start at step 0")
        if any(b[0] <= a[0] for a, b in zip(spec, spec[1:])):
            raise ValueError("schedule steps must increase")
        if any(t < 0 for _, t in spec):
            raise ValueError("tile sizes must be >= 0 (0 = FULL)")
        self.starts = [s for s, _ in spec]
        self.tiles = [t for _, t in spec]

    def __call__(self, step: int) -> int:
        return self.tiles[bisect.bisect_right(self.starts, step) - 1]

    @classmethod
    def every(cls, tiles, period: int):
        """Each T of `tiles` for `period` steps, in order (the last one stays)."""
        return cls([(i * period, t) for i, t in enumerate(tiles)])


def split_params(params, lr: float):
    """(himuon_groups, other_params) under the convention above.  `params` is an iterable
    of tensors or of parameter-group dicts; himuon_groups is a list of (lr, [params]),
    one per distinct learning rate, in order of first appearance."""
    groups = list(params)
    if groups and not isinstance(groups[0], dict):
        groups = [{"params": groups}]
    by_lr, other = {}, []
    for g in groups:
        use = g.get("use_himuon", True)
        glr = float(g.get("lr", lr))
        for p in g["params"]:
            if not p.requires_grad:
                continue
            if use and p.dim() == 2:
                by_lr.setdefault(glr, []).append(p)
            else:
                other.append(p)
    return list(by_lr.items()), other


def _check_factor(grad_scale, params):
    """Refuses a factor for the gradients of `params` before anything changes, so that no step is half done."""
    if not isinstance(grad_scale, torch.Tensor) or grad_scale.dtype != torch.float32 or grad_scale.numel() < 1 or \
            any(p.device != grad_scale.device for p in params):
        raise ValueError("grad_scale must be a float32 tensor on the parameters' device")


class HiMuonOptimizer(torch.optim.Optimizer):
    """HiMuon on the 2-D parameters, a plain optimizer on the others.

    lr, beta (momentum), steps (K), coeffs, eps and tile (an int or a TileSchedule) set
    the HiMuon step; state_dtype (torch.bfloat16 or torch.float32) is the dtype of the
    momentum and of the gradient copy; precision defaults to bf16x3.  `fallback` is a
    factory taking the list of other parameters (default: AdamW with lr fallback_lr).
    The optimizer step count is saved with the state, so a restored optimizer resumes
    the tile schedule where it stopped."""

    def __init__(self, params, lr: float = 0.02, beta: float = 0.95, tile=128, steps: int = 5,
                 coeffs=QUINTIC, eps: float = 1e-7, state_dtype=torch.bfloat16, precision=PREC_BF16X3,
                 workspace_budget: int = 4 * 10 ** 9, fallback=None, fallback_lr: float = 3e-4):
        hm_groups, other = split_params(params, lr)
        if not hm_groups:
            raise ValueError("no 2-D parameters for HiMuon")
        for _, ps in hm_groups:
            for p in ps:
                if p.dtype != torch.float32 or not p.is_cuda:
                    raise ValueError("HiMuon parameters must be float32 CUDA tensors")
        super().__init__([{"params": ps, "lr": glr} for glr, ps in hm_groups], dict(lr=lr, step_count=0))
        self.schedule = tile if isinstance(tile, TileSchedule) else TileSchedule(tile)
        self.steps, self.coeffs, self.beta, self.eps = steps, coeffs, beta, eps
        self.state_dtype, self.precision, self.budget = state_dtype, precision, workspace_budget
        self.fallback = None
        if other:
            self.fallback = (fallback(other) if fallback is not None
                             else torch.optim.AdamW(other, lr=fallback_lr))
        self._engines = None
        self._grads = None
        self._tile = None

    @property
    def step_count(self) -> int:
        return int(self.param_groups[0]["step_count"])

    def _build(self):
        """One plan per parameter group over the group's weights, momentum buffers (made
        here on first use, or restored by load_state_dict) and gradient buffers."""
        self._tile = self.schedule(self.step_count)
        self._engines, self._grads = [], []
        for grp in self.param_groups:
            layers, grads = [], []
            for p in grp["params"]:
                st = self.state[p]
                if "momentum_buffer" not in st:
                    st["momentum_buffer"] = torch.zeros(p.shape, dtype=self.state_dtype, device=p.device)
                m = st["momentum_buffer"]
                if m.dtype != self.state_dtype or m.shape != p.shape or not m.is_contiguous():
                    raise ValueError("momentum_buffer must be a contiguous tensor of the state dtype")
                g = torch.zeros(p.shape, dtype=self.state_dtype, device=p.device)
                layers.append((p.data, m, g))
                grads.append(g)
            self._engines.append(HiMuon(layers, self._tile, self.steps, self.coeffs, self.beta, self.eps,
                                        self.budget, precision=self.precision))
            self._grads.append(grads)

    @torch.no_grad()
    def step(self, closure=None, grad_scale=None):
        """grad_scale: None, or a float32 CUDA tensor whose first element multiplies every gradient (the clip
        factor of adamw.GradNorm), read on the device.  Where it is NaN (a gradient that is not finite) the HiMuon
        gradients count as zero (the momentum decays and still moves the matrices) and an AdamWOptimizer fallback
        skips its step, which it counts.  Other fallbacks take unscaled
        gradients, so a grad_scale with them is refused."""
        if grad_scale is not None and self.fallback is not None and not isinstance(self.fallback, AdamWOptimizer):
            raise ValueError("grad_scale needs an AdamWOptimizer fallback")
        if grad_scale is not None:
            groups = self.param_groups + (self.fallback.param_groups if self.fallback is not None else [])
            _check_factor(grad_scale, [p for grp in groups for p in grp["params"]])
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        if self._engines is None:
            self._build()
        T = self.schedule(self.step_count)
        if T != self._tile:
            for eng in self._engines:
                eng.set_tile_schedule(T)
            self._tile = T
        for grp, eng, grads in zip(self.param_groups, self._engines, self._grads):
            for p, g in zip(grp["params"], grads):
                if p.grad is None:
                    g.zero_()
                elif grad_scale is None:
                    g.copy_(p.grad)
                else:
                    factor = grad_scale.flatten()[:1]
                    g.copy_(torch.where(factor.isnan(), 0.0, p.grad.flatten() * factor).view(p.grad.shape))
            eng.step(float(grp["lr"]))
        if self.fallback is not None:
            if grad_scale is None:
                self.fallback.step()
            else:
                self.fallback.step(grad_scale=grad_scale)
        for grp in self.param_groups:
            grp["step_count"] = self.step_count + 1
        return loss

    def zero_grad(self, set_to_none: bool = True):
        super().zero_grad(set_to_none)
        if self.fallback is not None:
            self.fallback.zero_grad(set_to_none)

    def state_dict(self):
        sd = super().state_dict()
        if self.fallback is not None:
            sd["fallback"] = self.fallback.state_dict()
        return sd

    def load_state_dict(self, state_dict):
        """Restores momentum, step count and the fallback's state; the plans are rebuilt
        on the next step over the restored momentum tensors."""
        state_dict = dict(state_dict)
        fb = state_dict.pop("fallback", None)
        self.close()
        super().load_state_dict(state_dict)
        for st in self.state.values():
            m = st.get("momentum_buffer")
            if m is not None and (m.dtype != self.state_dtype or not m.is_contiguous()):
                st["momentum_buffer"] = m.to(self.state_dtype).contiguous()
        if fb is not None and self.fallback is not None:
            self.fallback.load_state_dict(fb)

    def momentum(self, p):
        """The HiMuon momentum tensor of 2-D parameter p."""
        st = self.state.get(p)
        if not st or "momentum_buffer" not in st:
            raise KeyError("not a HiMuon parameter of this optimizer (or no step taken yet)")
        return st["momentum_buffer"]

    def close(self):
        if self._engines is not None:
            for eng in self._engines:
                eng.close()
            self._engines = None
            self._grads = None


class AdamWOptimizer(torch.optim.Optimizer):
    """AdamW on this library's kernels (adamw.AdamW): every parameter of a group in one launch.

    Parameters are contiguous float32 or bfloat16 CUDA tensors; lr, betas, eps and
    weight_decay are per group as in torch.  state_bits: 32 (float32 moments) or 8 (e4m3
    values with a scale per 256 elements; `seed` starts the random numbers of their
    rounding).  A parameter's state is ``state[p]["adamw"]``, the tensors that
    adamw.adamw_state makes; its step count starts with its first gradient."""

    ENGINES = 32   # sets of parameters whose descriptors are kept, a step's own always: they pile up where sets vary

    def __init__(self, params, lr: float = 3e-4, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 state_bits: int = 32, seed: int = 0):
        if state_bits not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay))
        self.state_bits = state_bits
        self._random = random.Random(seed)
        self._engines = {}

    def add_param_group(self, group):
        super().add_param_group(group)
        for p in self.param_groups[-1]["params"]:
            if p.dtype not in (torch.float32, torch.bfloat16) or not p.is_cuda or not p.is_contiguous():
                self.param_groups.pop()
                raise ValueError("parameters must be contiguous float32 or bfloat16 CUDA tensors")

    def _engine(self, key, params, grads, states, group):
        """The AdamW over these parameters, kept while they, their memory, their states and the group's constants
        stay the same."""
        grads = [g if g.is_contiguous() else g.contiguous() for g in grads]
        # (ids: what they stand for is held with them)
        kind = (group["betas"], group["eps"], group["weight_decay"], list(map(id, params)), list(map(id, states)))
        held = self._engines.pop(key, None)
        if held is None or held[1] != kind or held[0]._at[0] != [p.data_ptr() for p in params] or \
                held[0]._n != [p.numel() for p in params]:
            engine = AdamW([(p.data, g, *s) for p, g, s in zip(params, grads, states)], *kind[:3])
            held = (engine, kind, params, states)
        elif not held[0]._same_grads(grads):
            held[0].set_grads(grads)
        self._engines[key] = held   # the last one used stands last
        return held[0]

    @torch.no_grad()
    def step(self, closure=None, grad_scale=None):
        """grad_scale: None, or a float32 CUDA tensor whose first element multiplies the gradients; NaN leaves
        parameters and moments as they are.  Such a step still counts for the bias corrections, for only the device
        knows of it: after k skipped ones a step divides its moments by 1 - beta^t with t too large by k (which
        matters while beta^t does: skipping the very first step makes the second one 0.74 of its size)."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        calls = {}   # one launch each
        for k, group in enumerate(self.param_groups):
            for p in group["params"]:
                g = p.grad
                if g is None:
                    continue
                st = self.state[p]
                if "adamw" not in st:
                    st["step"], st["adamw"] = 0, adamw_state(p, self.state_bits)
                calls.setdefault((k, p.device, p.dtype, g.dtype, st["step"] + 1), []).append((p, g, st))
        if grad_scale is not None:
            _check_factor(grad_scale, [call[0][0] for call in calls.values()])
        of_group = [key[0] for key in calls]
        for (*key, t), call in calls.items():
            params, grads, states = zip(*call)
            group = self.param_groups[key[0]]
            # parameters that joined late have a step count, and an engine, of their own
            key = (*key, tuple(map(id, params)) if of_group.count(key[0]) > 1 else None)
            dither = [self._random.getrandbits(32) for _ in range(2)] if self.state_bits == 8 else None
            engine = self._engine(key, params, grads, [st["adamw"] for st in states], group)
            engine.step(float(group["lr"]), t, scale=grad_scale, dither=dither)
            engine.drop_grads()
            torch.autograd.graph.increment_version(params)   # a graph that saved them must not go on with the new ones
            for st in states:
                st["step"] = t
        while len(self._engines) > max(self.ENGINES, len(calls)):
            del self._engines[next(iter(self._engines))]
        return loss

    def __getstate__(self):
        """For copies and pickles, which make descriptors of their own."""
        return {**super().__getstate__(), "state_bits": self.state_bits, "_random": self._random, "_engines": {}}

    def state_dict(self):
        sd = super().state_dict()
        sd["random"] = self._random.getstate()
        return sd

    def load_state_dict(self, state_dict):
        """Restores states bit for bit (torch would cast them to the parameters' dtype) and the random numbers; a
        state_dict that does not fit leaves the optimizer as it was."""
        state_dict = dict(state_dict)
        rng, numbers = state_dict.pop("random", None), self._random
        if rng is not None:
            numbers = random.Random()
            numbers.setstate((rng[0], tuple(rng[1]), rng[2]))
        held, states = state_dict["state"], {}
        for saved, group in zip(state_dict["param_groups"], self.param_groups):
            for i, p in zip(saved["params"], group["params"]):
                if held.get(i):
                    states[p] = self._loaded(held[i], p)
        super().load_state_dict({**state_dict, "state": {}})
        self.state.update(states)
        self._random, self._engines = numbers, {}

    def _loaded(self, saved, p):
        """A copy of a saved state of parameter p on its device."""
        blocks = (-(-p.numel() // ADAMW_BLOCK),)
        kinds = ([(torch.float32, p.shape)] * 2 if self.state_bits == 32 else
                 [(torch.float8_e4m3fn, p.shape)] * 2 + [(torch.float32, blocks)] * 2)
        tensors = saved.get("adamw", ())
        if "step" not in saved or [(x.dtype, x.shape) for x in tensors] != kinds:
            raise ValueError("the saved states are of another kind or shape")
        return {"step": int(saved["step"]), "adamw": tuple(x.to(p.device, copy=True) for x in tensors)}
