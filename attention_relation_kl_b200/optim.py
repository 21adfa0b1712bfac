"""The update of the trained weights: AdamW over many tensors in one launch, with
float32 or 8-bit states, and the norm of all their gradients.

LinearARD trains the student's Q/K/V projections; ``relkl_weight_grad`` gives their
gradients, and this step applies them.
"""
from __future__ import annotations

import math
import struct
from typing import NamedTuple, Optional, Sequence, Union

import torch

from . import _abi
from ._abi import check
from .ops import _on

__all__ = ["AdamWState", "adamw_state", "relkl_adamw", "relkl_grad_norm", "AdamW"]

BLOCK = 256     # elements that share one scale of an 8-bit state
_E4M3 = torch.float8_e4m3fn
_PLAN = struct.Struct("@iiddddqPPP")     # relkl_adamw_plan (include/relkl.h)


class AdamWState(NamedTuple):
    """Moments of one parameter.  32 bits: ``m`` and ``v`` are float32 of the parameter's
    shape.  8 bits: ``m`` and ``v`` are e4m3 codes of its shape (``v`` holds those of the
    root of the second moment), with a float32 scale for each block of 256 consecutive
    elements in ``m_scale`` and ``v_scale``."""
    m: torch.Tensor
    v: torch.Tensor
    m_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None


def adamw_state(param: torch.Tensor, bits: int = 32) -> AdamWState:
    """A fresh state: zeros."""
    if bits == 32:
        return AdamWState(*(torch.zeros(param.shape, dtype=torch.float32, device=param.device)
                            for _ in range(2)))
    if bits != 8:
        raise ValueError("states have 32 or 8 bits")
    blocks = -(-param.numel() // BLOCK)
    return AdamWState(*(torch.zeros(param.shape, dtype=torch.uint8, device=param.device).view(_E4M3)
                        for _ in range(2)),
                      *(torch.zeros(blocks, dtype=torch.float32, device=param.device)
                        for _ in range(2)))


def _scalar(x: torch.Tensor, dtype: torch.dtype, index: int, what: str) -> int:
    if x.dtype != dtype or x.numel() != 1 or x.get_device() != index:
        raise ValueError(f"{what} must be one {dtype} number on the parameters' device")
    return x.data_ptr()


def relkl_adamw(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                states: Sequence[AdamWState], *, lr: Union[float, torch.Tensor],
                step: Union[int, Sequence[int], torch.Tensor], betas=(0.9, 0.999), eps: float = 1e-8,
                weight_decay: Union[float, Sequence[float]] = 0.01,
                copies: Optional[Sequence[torch.Tensor]] = None,
                grad_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """One AdamW step, in place, over tensors of bf16 or float32 (parameters and
    gradients each), contiguous and on one device.

    ``step`` is the number of this step, from 1.  ``lr`` (float32) and ``step`` (int64)
    may be CUDA tensors of one number, read when the work runs, for captured graphs.
    ``weight_decay`` and ``step`` may give a number for each tensor (a launch for each
    number of steps among them).  ``copies`` are bf16 tensors
    that receive the new parameters rounded.  ``grad_scale``, one float32 number on the
    device, multiplies the gradients; where it is not finite nothing is written at all.
    """
    if len(params) == 0 and len(grads) == 0 and len(states) == 0:
        return
    lr_ptr = step_ptr = scale_ptr = 0
    step_dev = None
    if isinstance(step, torch.Tensor):
        step, step_dev = 1, step
    index, groups = _abi.marshal().adamw(params, grads, states, copies, weight_decay, step)
    if isinstance(lr, torch.Tensor):
        lr, lr_ptr = 0.0, _scalar(lr, torch.float32, index, "lr")
    if step_dev is not None:
        step_ptr = _scalar(step_dev, torch.int64, index, "step")
    if grad_scale is not None:
        scale_ptr = _scalar(grad_scale, torch.float32, index, "grad_scale")
    lib, launched = _abi.lib(), 0
    with _on(params[0].device, stream) as handle:
        for bits, number, n, table in groups if len(groups) > 1 else ():    # all are refused, or none
            plan = _PLAN.pack(bits, 0, lr, betas[0], betas[1], eps, number, lr_ptr, step_ptr, scale_ptr)
            check(lib.relkl_adamw_check(n, table, plan), "relkl_adamw")
        for bits, number, n, table in groups:
            plan = _PLAN.pack(bits, 0, lr, betas[0], betas[1], eps, number, lr_ptr, step_ptr, scale_ptr)
            status = lib.relkl_adamw(n, table, plan, handle)
            if status != _abi.RELKL_OK:
                break
            launched += 1
    if launched or status == _abi.RELKL_ERR_CUDA:     # something may have been written
        _abi.marshal().written(params)
        if copies is not None:
            _abi.marshal().written(copies)
    check(status, "relkl_adamw")


def relkl_grad_norm(grads: Sequence[torch.Tensor], max_norm: float = math.inf, *,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Two float32 numbers on the device: the norm of all gradients (bf16 or float32) taken
    together, and the factor min(1, max_norm / (norm + 1e-6)) that clips them to
    ``max_norm`` (NaN where the norm is not finite, as with an element from 2^64 on), for
    relkl_adamw's ``grad_scale``."""
    marshal = _abi.marshal()
    index, table = marshal.norm(grads)
    first = grads[0]
    if out is not None and (out.dtype != torch.float32 or tuple(out.shape) != (2,) or
                            not out.is_contiguous() or out.get_device() != index):
        raise ValueError("out must be a contiguous float32 tensor of two numbers on the "
                         "gradients' device")
    with _on(first.device, stream) as handle:
        status, got = marshal.grad_norm(first, table, max_norm, out, handle)
    check(status, "relkl_grad_norm")
    if out is not None:
        marshal.written([out])
    return got


class AdamW:
    """AdamW over a fixed list of parameters, with their states and step count.

    ``step(grads)`` takes the gradients in the parameters' order (None leaves a parameter as
    it is), or the parameters' ``.grad`` without them; with ``max_norm`` the gradients are
    clipped by the norm of all of them, and a step whose norm is not finite changes nothing
    but the counts.  ``counts`` holds the steps of each parameter, by which its moments are
    corrected: those that had a gradient for it; ``steps`` those of any, and setting it sets
    them all.  The counts are host numbers: for a captured graph call relkl_adamw with
    ``step`` and ``lr`` on the device.
    """

    def __init__(self, params: Sequence[torch.Tensor], lr: float = 1e-3, betas=(0.9, 0.999),
                 eps: float = 1e-8, weight_decay: Union[float, Sequence[float]] = 0.01, *,
                 state_bits: int = 32, max_norm: Optional[float] = None,
                 copies: Optional[Sequence[torch.Tensor]] = None):
        self.params = list(params)
        self.lr, self.betas, self.eps, self.max_norm = lr, tuple(betas), eps, max_norm
        n = len(self.params)
        self.weight_decay = ([float(weight_decay)] * n if isinstance(weight_decay, (int, float))
                             else list(weight_decay))
        self.copies = None if copies is None else list(copies)
        if len(self.weight_decay) != n or (self.copies is not None and len(self.copies) != n):
            raise ValueError("weight_decay and copies need one entry for each parameter")
        self.state = [adamw_state(p, state_bits) for p in self.params]
        self.steps = 0

    @property
    def steps(self) -> int:
        return self._steps

    @steps.setter
    def steps(self, number: int) -> None:
        self._steps, self.counts = number, [number] * len(self.params)

    def step(self, grads: Optional[Sequence[Optional[torch.Tensor]]] = None) -> Optional[torch.Tensor]:
        """Updates the parameters; returns the gradients' norm (on the device) with max_norm."""
        if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("AdamW.step counts on the host: capture relkl_adamw with step and lr "
                               "on the device")
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        if len(grads) != len(self.params):
            raise ValueError("grads need one entry for each parameter")
        at = [k for k, g in enumerate(grads) if g is not None]
        if not at:
            return None
        pick = lambda xs: [xs[k] for k in at]  # noqa: E731
        grads = pick(grads)
        clip = None if self.max_norm is None else relkl_grad_norm(grads, self.max_norm)
        counts, n = self.counts, len(self.params)
        even = counts.count(counts[0]) == n
        step = counts[0] + 1 if even else [counts[k] + 1 for k in at]
        relkl_adamw(pick(self.params), grads, pick(self.state), lr=self.lr, step=step,
                    betas=self.betas, eps=self.eps, weight_decay=pick(self.weight_decay),
                    copies=None if self.copies is None else pick(self.copies),
                    grad_scale=None if clip is None else clip[1:])
        self._steps += 1
        if even and len(at) == n:
            self.counts = [step] * n
        else:
            for k in at:
                counts[k] += 1
        return None if clip is None else clip[0]

    def state_dict(self) -> dict:
        return {"steps": self.steps, "counts": list(self.counts), "state": [tuple(s) for s in self.state]}

    def load_state_dict(self, saved: dict) -> None:
        """Copies a state_dict's values into this optimizer's states (which keep their place).
        One without ``counts`` has the same count for all parameters."""
        states, steps = saved["state"], int(saved["steps"])
        counts = [int(c) for c in saved.get("counts", [steps] * len(states))]
        if len(states) != len(self.state) or len(counts) != len(states):
            raise ValueError("the saved state is of another number of parameters")
        for mine, theirs in zip(self.state, states):
            for a, b in zip(mine, theirs):
                if (a is None) != (b is None) or (a is not None and (a.dtype != b.dtype or a.shape != b.shape)):
                    raise ValueError("the saved state is of other parameters or another state_bits")
        for mine, theirs in zip(self.state, states):
            for a, b in zip(mine, theirs):
                if a is not None:
                    a.copy_(b)
        self._steps, self.counts = steps, counts
