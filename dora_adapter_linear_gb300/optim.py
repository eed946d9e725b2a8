"""AdamW over a set of tensors at once, such as the A and B of every adapted projection."""
from __future__ import annotations

import math
from ctypes import c_float

import torch

from . import _lib as L

BLOCK = 256     # elements of a state block


def _each(name, value, count):
    values = list(value) if isinstance(value, (list, tuple)) else [value] * count
    if len(values) != count:
        raise ValueError(f"{name}: {len(values)} values for {count} tensors")
    if not all(math.isfinite(v) for v in values):
        raise ValueError(f"{name} must be finite")
    return values


class AdamW:
    """The optimiser of `params`: contiguous fp32 or bf16 CUDA tensors, updated in place in the storage
    they have now.  lr_mul (a factor on lr, such as a larger step for B) and weight_decay are numbers
    or lists with one for each tensor.  state_bits 32 keeps m and v in fp32, 8 as e4m3 codes of m and
    sqrt(v) with a scale for every 256 elements.  master: bf16 tensors keep their exact values in fp32.

    State, on the device: m, v (and m_scale, v_scale, master) with 256 elements a row, each tensor from
    a row of its own, and the number of steps done.  The steps are the set's: a tensor that had no gradient
    for some of them comes back with the bias correction of all."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, lr_mul=1.0, state_bits=32,
                 master=True):
        params = [p.detach() for p in params]
        for i, p in enumerate(params):
            if p.dtype not in (torch.float32, torch.bfloat16) or not p.is_cuda or not p.is_contiguous():
                raise ValueError(f"tensor {i} must be a contiguous fp32 or bf16 CUDA tensor, got {p.dtype} on "
                                 f"{p.device} with strides {p.stride()}")
            if p.device != params[0].device:
                raise ValueError(f"tensor {i} is on {p.device}, the first on {params[0].device}")
        if not params:
            raise ValueError("no tensors to optimise")
        self._device = params[0].device
        L.need_current("the tensors", self._device)
        spans = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size()) for p in params if p.numel())
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("two of the tensors share memory: each would be updated under the other's hands")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        b1, b2 = betas
        if not (0.0 <= b1 < 1.0 and 0.0 <= b2 < 1.0 and 2.0 ** -126 <= eps < 2.0 ** 128):
            raise ValueError(f"betas must be in [0, 1) and eps a normal fp32 number, got {betas}, {eps}")
        self.params, self.lr, self.betas, self.eps, self.state_bits = params, lr, (b1, b2), eps, state_bits
        n = len(params)
        self._tensors = L.adamw_tensors(params, _each("lr_mul", lr_mul, n), _each("weight_decay", weight_decay, n))
        dev, blocks = params[0].device, L.adamw_state_blocks(self._tensors, n)
        code = torch.float8_e4m3fn if state_bits == 8 else torch.float32
        new = lambda dtype, width: torch.zeros(blocks, width, dtype=dtype, device=dev)  # noqa: E731
        self.m, self.v = new(code, BLOCK), new(code, BLOCK)
        self.m_scale, self.v_scale = (new(torch.float32, 1), new(torch.float32, 1)) if state_bits == 8 else (None, None)
        self.master = None
        if master and any(p.dtype == torch.bfloat16 for p in params):
            self.master = new(torch.float32, BLOCK)
            L.adamw_fill_master(self._tensors, n, self.master)
        self._ctl = torch.zeros(2, dtype=torch.int32, device=dev)
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self._state = L.LoraAdamwState(ptr(self.m), ptr(self.v), ptr(self.m_scale), ptr(self.v_scale),
                                       ptr(self.master), ptr(self._ctl), state_bits)
        # of its own, so that a captured step keeps what it was captured with
        self._ws = torch.zeros(L.adamw_norm_workspace_bytes(n), dtype=torch.uint8, device=dev)

    @property
    def steps(self) -> int:
        """Steps done (waits for the device)."""
        return int(self._ctl[0])

    def _pointers(self, grads):
        """The gradients' addresses, 0 for a None, of other sequences than lists and tuples; what does not fit is
        named."""
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} tensors")
        grads = list(grads)
        for i, (g, p) in enumerate(zip(grads, self.params)):
            if g is not None and (g.shape != p.shape or g.dtype != p.dtype or g.device != p.device
                                  or not g.is_contiguous()):
                raise ValueError(f"gradient {i} must be a contiguous {tuple(p.shape)} {p.dtype} tensor on {p.device}, "
                                 f"got {tuple(g.shape)} {g.dtype} on {g.device}")
        return L.host().pointers(grads, self.params)

    def step(self, grads, lr=None, max_norm=None, grad_scale=1.0):
        """One step from `grads`, a tensor (or None: its tensor stays) for each parameter, on the current
        stream.  lr: a number or a 0-d fp32 CUDA tensor (read when the step runs: a captured graph
        follows it); by default the one given at first.  grad_scale multiplies every gradient;
        max_norm then clips their global norm.  With max_norm the norm before the clip is returned (a
        0-d tensor, nothing waits), and a step whose norm is not finite changes nothing and is not
        counted; max_norm=inf only guards."""
        L.need_current("the tensors", self._device)
        host, n, norm = L.host(), len(self.params), None
        at = host.pointers(grads, self.params)
        if at is None:
            at = self._pointers(grads)
        lr = self.lr if lr is None else lr
        lr_dev = None
        if isinstance(lr, torch.Tensor):
            if lr.dtype != torch.float32 or lr.numel() != 1 or lr.device != self.params[0].device:
                raise ValueError(f"lr must be a number or one fp32 value on {self.params[0].device}")
            lr, lr_dev = 0.0, lr.data_ptr()
        hyper = L.LoraAdamwHyper(lr, *self.betas, self.eps, grad_scale, lr_dev)
        if max_norm is not None:
            if not c_float(max_norm).value > 0:     # as the kernels have it; 0 there is no clip at all
                raise ValueError(f"max_norm must be above 0 in fp32, got {max_norm}")
            norm = host.pair(self.params[0])   # shows the norm, the factor lies behind it
            L.adamw_grad_norm(self._tensors, at, n, grad_scale, max_norm, norm, self._ws)
        L.adamw_step(self._tensors, at, n, self._state, hyper, norm)
        host.written(self.params, at)
        return norm

    def state_dict(self):
        """The state as tensors (the optimiser's own, not copies) and the step count."""
        return {"step": self.steps, "m": self.m, "v": self.v, "m_scale": self.m_scale, "v_scale": self.v_scale,
                "master": self.master, "sizes": [p.numel() for p in self.params]}

    def load_state_dict(self, state):
        """Copies a state_dict() of an optimiser of the same tensors and state_bits into this one.  The
        tensors themselves are the caller's to restore; with masters the next step sets them from those."""
        if state.get("sizes", [p.numel() for p in self.params]) != [p.numel() for p in self.params]:
            raise ValueError("the state is of tensors of other sizes")
        for k in ("m", "v", "m_scale", "v_scale", "master"):
            mine, other = getattr(self, k), state[k]
            if (mine is None) != (other is None) or (mine is not None and (mine.shape != other.shape
                                                                          or mine.dtype != other.dtype)):
                raise ValueError(f"{k} of the state does not fit this optimiser")
        for k in ("m", "v", "m_scale", "v_scale", "master"):
            if state[k] is not None:
                getattr(self, k).copy_(state[k])
        self._ctl.copy_(torch.tensor([state["step"], 0], dtype=torch.int32))


def clip_grads(grads, max_norm, groups=None):
    """Scales gradients in place by min(1, max_norm / (norm + 1e-6)) of their group's norm, and returns the
    norms before that, fp32 [groups] on the device; nothing waits.  grads: contiguous fp32 or bf16 CUDA
    tensors (or None); groups: None, one group of all; a list with the number of each tensor's group, 0 to
    the largest; or a number G: every tensor is a stack of G groups along its first dimension, as the
    gradients of ops.lora_multi_bwd are.  A group whose norm is not finite (from 2^64 on) becomes
    zeros, the others go on.  max_norm None: the norms alone; infinity: only such groups change.  A list without
    any tensor is refused: it has no device."""
    grads = grads if isinstance(grads, (list, tuple)) else list(grads)
    each = None
    if groups is None:
        count, each = 1, [0] * len(grads)
    elif isinstance(groups, int):
        count = groups
    else:
        each = list(groups)
        if len(each) != len(grads):
            raise ValueError(f"{len(each)} groups for {len(grads)} gradients")
        count = max(each, default=0) + 1
    if max_norm is None:
        limit = 0.0
    elif c_float(max_norm).value > 0:       # as the kernels have it
        limit = max_norm
    else:
        raise ValueError(f"max_norm must be above 0 in fp32, got {max_norm}")
    norms = L.host().clip_grads(grads, each, count, limit)
    if norms is None:
        _check_grads(grads, each, count)
        raise ValueError("no gradients to clip")
    if isinstance(norms, int):
        if norms == 1:
            raise ValueError("two of the gradients share memory: each would be scaled under the other's hands")
        raise L.LoraError(norms, "grad_clip")
    return norms


def _check_grads(grads, each, count):
    """Names what clip_grads cannot take."""
    if not 1 <= count <= 65535:
        raise ValueError(f"there must be 1 to 65535 groups, got {count}")
    for i, g in enumerate(grads):
        if g is None:
            continue
        if not isinstance(g, torch.Tensor):
            raise ValueError(f"gradient {i} must be a tensor or None, got {type(g).__name__}")
        if g.dtype not in (torch.float32, torch.bfloat16) or not g.is_cuda or g.layout != torch.strided \
                or not g.is_contiguous():
            raise ValueError(f"gradient {i} must be a contiguous fp32 or bf16 CUDA tensor, got {g.dtype} on {g.device}")
        L.need_current(f"gradient {i}", g.device)
        if each is None and (g.dim() < 1 or g.shape[0] != count):
            raise ValueError(f"gradient {i} must be a stack of {count} groups, got {tuple(g.shape)}")
        if each is not None and not 0 <= each[i] < count:
            raise ValueError(f"group {each[i]} of gradient {i} is not in 0 to {count - 1}")
