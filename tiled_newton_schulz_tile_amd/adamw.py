"""AdamW and the gradient norm over many torch tensors at once (himuon_adamw_step and
himuon_grad_norm of libhimuon): the update of the parameters that HiMuon leaves alone, and
the clip factor of a gradient, which stays on the device.

AdamW and GradNorm hold the descriptors of a list of tensors; formulas, the 8-bit state
format and conventions are in include/himuon.h.
"""
from __future__ import annotations

import struct
from array import array

from . import (ADAMW_BLOCK, BF16, F32, himuon_adamw_config, himuon_adamw_step, himuon_adamw_table,
               himuon_adamw_table_size, himuon_adamw_tensor, himuon_grad, himuon_grad_norm, himuon_grad_norm_workspace)


def _column(tensors, name, dtypes, device):
    """(element counts, addresses) of tensors that share one dtype out of `dtypes`."""
    dtype = tensors[0].dtype
    if dtype not in dtypes or device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor of {' or '.join(str(d) for d in dtypes)}")
    for t in tensors:
        if t.dtype is not dtype or t.device != device or not t.is_contiguous():
            raise ValueError(f"every {name} must be a contiguous {dtype} tensor on {device}")
    return [t.numel() for t in tensors], [t.data_ptr() for t in tensors]


def _launch(torch, device, stream, call, *args):
    """call(*args, stream) with `device` the current one, as the library needs it; returns the stream's handle.  The
    current stream is asked for by its raw handle where torch gives it: a call of a few microseconds should not spend
    two on a Stream object."""
    if stream is not None:
        s = stream.cuda_stream
    else:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        s = raw(device.index) if raw is not None else torch.cuda.current_stream(device).cuda_stream
    if torch.cuda.current_device() == device.index:
        call(*args, s)
    else:
        with torch.cuda.device(device):
            call(*args, s)
    return s


class _Streams:
    """The streams, besides the one that an object was made on, that its calls went to: memory that the object lets
    go of has to wait for them."""

    def _made(self, memory):
        """memory: the object's own tensor on the device, or None."""
        self._own, self._abroad = memory, []
        self._home = self._torch.cuda.current_stream(self.device).cuda_stream

    def _went_abroad(self, stream, of_call=None):
        """A call went to `stream` (None: the current one), whose handle is not self._home; of_call: a tensor that it
        was given and that is not held."""
        if stream is None:
            stream = self._torch.cuda.current_stream(self.device)
        for t in (self._own, of_call):
            if t is not None:
                t.record_stream(stream)
        if stream not in self._abroad:
            self._abroad.append(stream)

    def _let_go(self, tensors):
        for stream in self._abroad:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)

    def __del__(self):
        try:
            self._let_go(self._held())
        except Exception:   # not made, or the interpreter ends
            pass


def _empty(torch, stream, size, dtype):
    """A new tensor that work on `stream` may write at once.  One of the current stream's pool may be memory that
    kernels still pending there use; this one is of `stream`'s own, recorded on the current one, whose work will
    read it."""
    with torch.cuda.stream(stream):
        t = torch.empty(size, dtype=dtype, device=stream.device)
    t.record_stream(torch.cuda.current_stream(stream.device))
    return t


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


class AdamW(_Streams):
    """AdamW over a list of contiguous CUDA tensors.

    tensors: list of (W, G, m, v) with float32 states, or of (W, G, m, r, m_scale, r_scale)
    with 8-bit states (adamw_state makes both).  All W share one dtype (float32 or
    bfloat16), all G share one, and all states are of one kind.  weight_decay is one number
    or one per tensor.  The tensors are referenced, not copied; set_grads replaces the
    gradients (a training program whose gradients are new tensors each step).  For more
    tensors than a small argument table takes (8) the descriptors are kept on the device;
    set_grads and the steps after it then go on one stream.  A graph that captured its calls
    needs the object, and its tensors, for as long as it is replayed."""

    def __init__(self, tensors, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.0):
        import torch
        self._torch = torch
        tensors = [tuple(t) for t in tensors]
        if not tensors:
            raise ValueError("no tensors")
        if len({len(t) for t in tensors}) != 1 or len(tensors[0]) not in (4, 6):
            raise ValueError("every tensor is (W, G, m, v), or every one (W, G, m, r, m_scale, r_scale)")
        decay = [weight_decay] * len(tensors) if isinstance(weight_decay, (int, float)) else list(weight_decay)
        if len(decay) != len(tensors):
            raise ValueError("one weight_decay per tensor")
        cols = list(zip(*tensors))
        self.bits = 32 if len(cols) == 4 else 8
        self.device = cols[0][0].device
        floats = (torch.float32, torch.bfloat16)
        state = (torch.float32,) if self.bits == 32 else (torch.float8_e4m3fn,)
        n, w = _column(cols[0], "W", floats, self.device)
        ptrs = [w]
        for col, name, dtypes in zip(cols[1:4], ("G", "m", "v"), (floats, state, state)):
            size, at = _column(col, name, dtypes, self.device)
            if size != n:
                raise ValueError("W, G and the states must have the same number of elements")
            ptrs.append(at)
        self._at = ptrs[:2]   # addresses of W and G
        for col in cols[4:]:
            size, at = _column(col, "scale", (torch.float32,), self.device)
            if size != [-(-k // ADAMW_BLOCK) for k in n]:
                raise ValueError(f"a scale holds one value per {ADAMW_BLOCK} elements")
            ptrs.append(at)
        if self.bits == 32:
            ptrs += [[0] * len(n)] * 2
        bits = [struct.unpack("q", struct.pack("d", d))[0] for d in decay]
        self._words = array("Q")   # the C structures: n, six addresses, weight_decay
        for row in zip(n, *ptrs, bits):
            self._words.extend([x & (2 ** 64 - 1) for x in row])
        self._c = (himuon_adamw_tensor * len(n)).from_buffer(self._words)
        self._n, self._tensors, self._grad_dtype = n, cols, cols[1][0].dtype
        dt = lambda t: F32 if t.dtype == torch.float32 else BF16  # noqa: E731
        self.cfg = himuon_adamw_config(dt(cols[0][0]), dt(cols[1][0]), self.bits, betas[0], betas[1], eps)
        size = himuon_adamw_table_size(self._c, self.cfg)
        self._table = torch.empty(size, dtype=torch.uint8, device=self.device) if size else None
        self._made(self._table)
        if size:
            host = array("Q", bytes(-(-size // 8) * 8))
            himuon_adamw_table(self._c, self.cfg, host.buffer_info()[0], size)
            self._table.copy_(torch.frombuffer(host, dtype=torch.uint8)[:size])   # done when it returns

    @property
    def tensors(self):
        return list(zip(*self._tensors))

    def _held(self):
        return [t for col in self._tensors for t in col]

    def set_grads(self, grads, stream=None) -> None:
        """Replaces the gradients from the next step on (same dtype and sizes)."""
        torch = self._torch
        grads = tuple(grads)
        if self._table is not None and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("set the gradients before the graph is captured: their table is copied from host memory")
        if len(grads) != len(self._n):
            raise ValueError("one gradient per tensor")
        size, at = _column(grads, "G", (self._grad_dtype,), self.device)
        if size != self._n:
            raise ValueError("a gradient must have its weight's number of elements")
        self._let_go(self._tensors[1])
        self._tensors[1], self._at[1] = grads, at
        self._words[2::8] = array("Q", at)
        if self._table is not None:
            host = torch.empty(self._table.numel(), dtype=torch.uint8, pin_memory=True)
            himuon_adamw_table(self._c, self.cfg, host.data_ptr(), host.numel())
            with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(self.device)):
                self._table.copy_(host[:self._table.numel()], non_blocking=True)
            if (stream if stream is not None else torch.cuda.current_stream(self.device)).cuda_stream != self._home:
                self._went_abroad(stream)

    def drop_grads(self) -> None:
        """Forgets the gradients, so that their memory may go; a step needs new ones first (set_grads)."""
        self._let_go(self._tensors[1])
        self._tensors[1] = (None,) * len(self._n)

    def _same_grads(self, grads) -> bool:
        """Holds `grads` again, after drop_grads, if they are where the descriptors say."""
        if [g.data_ptr() for g in grads] != self._at[1] or [g.numel() for g in grads] != self._n:
            return False
        self._tensors[1] = tuple(grads)
        return True

    def step(self, lr: float, t: int, scale=None, dither=None, stream=None) -> None:
        """Step number t >= 1.  scale: None or a float32 CUDA tensor whose first element multiplies
        the gradients (GradNorm's factor; NaN leaves everything unchanged).  dither: two random
        numbers in [0, 2^32), new ones each step, for 8-bit states."""
        torch = self._torch
        if self._tensors[1][0] is None:
            raise RuntimeError("the gradients were dropped: set_grads gives the step's")
        at = 0
        if scale is not None:
            if scale.dtype != torch.float32 or scale.device != self.device or scale.numel() < 1:
                raise ValueError(f"scale must be a float32 tensor on {self.device}")
            at = scale.data_ptr()
        if _launch(torch, self.device, stream, himuon_adamw_step, self._c, self.cfg, t, lr, at, dither,
                   self._table.data_ptr() if self._table is not None else 0) != self._home:
            self._went_abroad(stream, scale)


class GradNorm(_Streams):
    """Norm and clip factor of a list of contiguous CUDA tensors of one dtype (float32 or bfloat16)."""

    def __init__(self, grads):
        import torch
        self._torch = torch
        grads = tuple(grads)
        if not grads:
            raise ValueError("no tensors")
        self.device = grads[0].device
        self._dtypes = (torch.float32, torch.bfloat16)
        self._c = None
        self._n = len(grads)
        self.set_grads(grads)
        self._dtypes = (grads[0].dtype,)
        self._dt = F32 if grads[0].dtype == torch.float32 else BF16
        self._ws = torch.zeros(himuon_grad_norm_workspace(len(grads)), dtype=torch.uint8, device=self.device)
        self._made(self._ws)
        torch.cuda.current_stream(self.device).synchronize()   # the zeros are there for a call on any stream

    def _held(self):
        return self.grads

    def set_grads(self, grads) -> None:
        """Replaces the tensors (as many as before, of the same dtype)."""
        grads = tuple(grads)
        if len(grads) != self._n:
            raise ValueError("as many gradients as before")
        n, at = _column(grads, "gradient", self._dtypes, self.device)
        words = array("Q")
        for row in zip(n, at):
            words.extend(row)
        if self._c is not None:
            self._let_go(self.grads)
        self._words, self.grads = words, grads
        self._c = (himuon_grad * len(n)).from_buffer(words)

    def compute(self, max_norm: float, out=None, stream=None):
        """A float32 CUDA tensor (norm, factor): the 2-norm over all tensors and min(1, max_norm / (norm + 1e-6)),
        NaN where the gradient is not finite.  out: a tensor of two elements to write to instead of a new one
        (allocated on the stream of the call).  Calls of one GradNorm share its workspace: they go on one stream, or
        the caller orders them."""
        torch = self._torch
        if out is None:
            if stream is None:
                out = torch.empty(2, dtype=torch.float32, device=self.device)
            else:
                out = _empty(torch, stream, (2,), torch.float32)
        elif out.dtype != torch.float32 or out.shape != (2,) or out.device != self.device or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous float32 tensor of two elements on {self.device}")
        if _launch(torch, self.device, stream, himuon_grad_norm, self._c, self._dt, max_norm, out.data_ptr(),
                   self._ws.data_ptr(), self._ws.numel()) != self._home:
            self._went_abroad(stream, out)
        return out
