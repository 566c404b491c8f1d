"""AdamW and the gradient norm over many torch tensors at once (himuon_adamw_step and
himuon_grad_norm of libhimuon): the update of the parameters that HiMuon leaves alone, and
the clip factor of the whole gradient, which stays on the device.

AdamW and GradNorm hold the descriptors of a list of tensors; formulas, the 8-bit state
format and conventions are in include/himuon.h.
"""
from __future__ import annotations

from . import (ADAMW_BLOCK, BF16, F32, himuon_adamw_config, himuon_adamw_step, himuon_adamw_tensor, himuon_grad,
               himuon_grad_norm, himuon_grad_norm_workspace)


def _dtype(t):
    import torch
    return F32 if t.dtype == torch.float32 else BF16


def _check_tensor(t, name, dtypes, device):
    if t.dtype not in dtypes or not t.is_cuda or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {' or '.join(str(d) for d in dtypes)} on {device}")


def adamw_state(W, bits: int = 32):
    """Zero states of parameter W as AdamW takes them: (m, v) in float32, or with bits=8
    (m, r, m_scale, r_scale) with e4m3 values and one float32 scale per 256 elements."""
    import torch
    if bits == 32:
        return tuple(torch.zeros(W.shape, dtype=torch.float32, device=W.device) for _ in range(2))
    if bits != 8:
        raise ValueError("bits must be 32 or 8")
    blocks = -(-W.numel() // ADAMW_BLOCK)
    return (*(torch.zeros(W.shape, dtype=torch.uint8, device=W.device).view(torch.float8_e4m3fn) for _ in range(2)),
            *(torch.zeros(blocks, dtype=torch.float32, device=W.device) for _ in range(2)))


def adamw_moments(state):
    """(m, v) in float32 that a tensor's states stand for."""
    import torch
    if len(state) == 2:
        return tuple(s.clone() for s in state)
    out = []
    for code, scale in zip(state[:2], state[2:]):
        unit = scale.repeat_interleave(ADAMW_BLOCK)[:code.numel()].view(code.shape)
        out.append(code.to(torch.float32) * unit)
    return out[0], out[1].square()


class AdamW:
    """AdamW over a list of contiguous CUDA tensors.

    tensors: list of (W, G, m, v) with float32 states, or of (W, G, m, r, m_scale, r_scale)
    with 8-bit states (adamw_state makes both).  All W share one dtype (float32 or
    bfloat16), all G share one, and all states are of one kind.  weight_decay is one number
    or one per tensor.  The tensors are referenced, not copied; set_grads replaces the
    gradients (a training program whose gradients are new tensors each step)."""

    def __init__(self, tensors, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.0):
        import torch
        self._torch = torch
        self.tensors = [tuple(t) for t in tensors]
        if not self.tensors:
            raise ValueError("no tensors")
        decay = [weight_decay] * len(self.tensors) if isinstance(weight_decay, (int, float)) else list(weight_decay)
        if len(decay) != len(self.tensors):
            raise ValueError("one weight_decay per tensor")
        first = self.tensors[0]
        if len(first) not in (4, 6):
            raise ValueError("a tensor is (W, G, m, v) or (W, G, m, r, m_scale, r_scale)")
        self.bits = 32 if len(first) == 4 else 8
        self.device = first[0].device
        floats = (torch.float32, torch.bfloat16)
        state = (torch.float32,) if self.bits == 32 else (torch.float8_e4m3fn,)
        self._c = (himuon_adamw_tensor * len(self.tensors))()
        for c, t, wd in zip(self._c, self.tensors, decay):
            if len(t) != len(first):
                raise ValueError("all states must be of one kind")
            n = t[0].numel()
            _check_tensor(t[0], "W", floats if t is first else (first[0].dtype,), self.device)
            _check_tensor(t[1], "G", floats if t is first else (first[1].dtype,), self.device)
            for x in t[2:4]:
                _check_tensor(x, "a state", state, self.device)
            for x in t[1:4]:
                if x.numel() != n:
                    raise ValueError("W, G and the states must have the same number of elements")
            for x in t[4:]:
                _check_tensor(x, "a scale", (torch.float32,), self.device)
                if x.numel() != -(-n // ADAMW_BLOCK):
                    raise ValueError(f"a scale holds one value per {ADAMW_BLOCK} elements")
            p = [x.data_ptr() for x in t]
            c.n, c.weight, c.grad, c.m, c.v = n, p[0], p[1], p[2], p[3]
            if self.bits == 8:
                c.m_scale, c.v_scale = p[4], p[5]
            c.weight_decay = wd
        self.cfg = himuon_adamw_config(_dtype(first[0]), _dtype(first[1]), self.bits, betas[0], betas[1], eps)

    def set_grads(self, grads) -> None:
        """Replaces the gradients from the next step on (same dtype and sizes)."""
        grads = list(grads)
        if len(grads) != len(self.tensors):
            raise ValueError("one gradient per tensor")
        for t, g in zip(self.tensors, grads):
            _check_tensor(g, "G", (t[1].dtype,), self.device)
            if g.numel() != t[0].numel():
                raise ValueError("a gradient must have its weight's number of elements")
        for k, (c, g) in enumerate(zip(self._c, grads)):
            c.grad = g.data_ptr()
            self.tensors[k] = (self.tensors[k][0], g, *self.tensors[k][2:])

    def step(self, lr: float, t: int, scale=None, dither=None, stream=None) -> None:
        """Step number t >= 1.  scale: None or a float32 CUDA tensor whose first element multiplies
        the gradients (GradNorm's factor; NaN leaves everything unchanged).  dither: two random
        numbers in [0, 2^32), new ones each step, for 8-bit states."""
        torch = self._torch
        if scale is not None:
            if scale.dtype != torch.float32 or scale.device != self.device or scale.numel() < 1:
                raise ValueError(f"scale must be a float32 tensor on {self.device}")
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        with torch.cuda.device(self.device):
            himuon_adamw_step(self._c, self.cfg, t, lr, scale.data_ptr() if scale is not None else 0, dither,
                              s.cuda_stream)


class GradNorm:
    """Norm and clip factor of a list of contiguous CUDA tensors of one dtype (float32 or bfloat16)."""

    def __init__(self, grads):
        import torch
        self._torch = torch
        grads = list(grads)
        if not grads:
            raise ValueError("no tensors")
        self.device = grads[0].device
        self._dt = grads[0].dtype
        self._c = (himuon_grad * len(grads))()
        self.set_grads(grads)
        self._ws = torch.empty(himuon_grad_norm_workspace(len(grads)), dtype=torch.uint8, device=self.device)

    def set_grads(self, grads) -> None:
        """Replaces the tensors (as many as before, of the same dtype)."""
        torch = self._torch
        grads = list(grads)
        if len(grads) != len(self._c):
            raise ValueError("as many gradients as before")
        for g in grads:
            _check_tensor(g, "a gradient", (self._dt,) if self._dt in (torch.float32, torch.bfloat16) else
                          (torch.float32, torch.bfloat16), self.device)
        self.grads = grads
        for c, g in zip(self._c, grads):
            c.n, c.grad = g.numel(), g.data_ptr()

    def compute(self, max_norm: float, out=None, stream=None):
        """A float32 CUDA tensor (norm, factor): the 2-norm over all tensors and min(1, max_norm / (norm + 1e-6)),
        NaN where the gradient is not finite.  out: a tensor of two elements to write to instead of a new one.
        Calls of one GradNorm share its workspace: they go on one stream, or the caller orders them."""
        torch = self._torch
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        with torch.cuda.device(self.device), torch.cuda.stream(s):
            if out is None:
                out = torch.empty(2, dtype=torch.float32, device=self.device)
            elif out.dtype != torch.float32 or out.shape != (2,) or out.device != self.device or not out.is_contiguous():
                raise ValueError(f"out must be a contiguous float32 tensor of two elements on {self.device}")
            himuon_grad_norm(self._c, _dtype(self.grads[0]), max_norm, out.data_ptr(), self._ws.data_ptr(),
                             self._ws.numel(), s.cuda_stream)
        return out
