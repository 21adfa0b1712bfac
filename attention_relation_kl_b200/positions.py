"""Rotary positions of the relation inputs, and of their gradients.

The teacher's Q and K are rotated at its own positions, the student's at scaled
ones; V is only brought into the same layout.  All tensors are logically
[B, H, N, d], with any strides: a projection's output is passed as
``proj.view(B, N, H, d).transpose(1, 2)``, and a view of that kind as ``out``
gives the token-major layout that ``relkl_weight_grad`` reads.
"""
from __future__ import annotations

import math
from typing import List, NamedTuple, Optional, Sequence

import torch

from . import _abi
from ._abi import check
from .ops import _DTYPES, _on

__all__ = ["RotaryFreqs", "rotary_freqs", "relkl_rotary_qkv", "relkl_rotary", "Rotary", "rotary"]


class RotaryFreqs(NamedTuple):
    """Pair frequencies (float64 [rot / 2]) and the factor on the rotated entries."""
    inv_freq: torch.Tensor
    mscale: float


def rotary_freqs(rot: int, base: float = 1e4, scaling: str = "none", factor: float = 1.0, *,
                 original_length: int = 4096, low_turns: float = 1.0,
                 high_turns: Optional[float] = None, device="cuda") -> RotaryFreqs:
    """Frequencies f_i = base^(-2i/rot) of ``rot / 2`` pairs, scaled for contexts
    ``factor`` times as long as the ``original_length``:

    * ``"none"``: as they are;
    * ``"linear"``: f_i / factor (positional interpolation);
    * ``"ntk"``: those of the base ``base * factor^(rot / (rot - 2))``;
    * ``"yarn"``: pairs that turn at least ``high_turns`` times within the original
      length keep f_i, those below ``low_turns`` take f_i / factor, with a ramp over
      the pairs between; the factor on the rotated entries is 0.1 ln(factor) + 1;
    * ``"bands"``: as yarn, with the ramp over the number of turns, and no factor.

    Without ``high_turns`` it is 32 with yarn and 4 with bands, as is usual for them.
    """
    if rot < 0 or rot % 2:
        raise ValueError("rot must be even and not negative")
    if not (math.isfinite(base) and base > 1.0 and math.isfinite(factor) and factor > 0.0):
        raise ValueError("base must be above 1 and factor positive")
    if high_turns is None:
        high_turns = 4.0 if scaling == "bands" else 32.0
    if original_length < 1 or not 0.0 < low_turns < high_turns:
        raise ValueError("original_length must be positive and 0 < low_turns < high_turns")
    i = torch.arange(rot // 2, dtype=torch.float64)
    exponent = -2.0 * i / max(rot, 1)
    f, m = base ** exponent, 1.0
    if scaling == "none":
        pass
    elif scaling == "linear":
        f = f / factor
    elif scaling == "ntk":
        if rot == 2:
            raise ValueError("ntk scaling needs at least two pairs")
        f = (base * factor ** (rot / (rot - 2.0))) ** exponent
    elif scaling == "yarn":
        def pair_of(turns):   # the pair that turns this often within the original length
            return rot * math.log(original_length / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        first = max(math.floor(pair_of(high_turns)), 0)
        last = min(math.ceil(pair_of(low_turns)), rot - 1)
        ramp = ((i - first) / max(last - first, 1e-3)).clamp(0.0, 1.0)
        f = f / factor * ramp + f * (1.0 - ramp)
        m = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
    elif scaling == "bands":
        turns = original_length * f / (2.0 * math.pi)
        keep = ((turns - low_turns) / (high_turns - low_turns)).clamp(0.0, 1.0)
        f = (1.0 - keep) * f / factor + keep * f
    else:
        raise ValueError(f"unknown scaling {scaling!r}")
    return RotaryFreqs(f.to(device), m)


def relkl_rotary_qkv(xs: Sequence[torch.Tensor], inv_freq: torch.Tensor, *,
                     apply: Optional[Sequence[bool]] = None, pos_scale: float = 1.0,
                     pos_offset: float = 0.0, positions: Optional[torch.Tensor] = None,
                     mscale: float = 1.0, interleaved: bool = False, inverse: bool = False,
                     out: Optional[Sequence[torch.Tensor]] = None,
                     out_dtype: Optional[torch.dtype] = None, stream=None) -> List[torch.Tensor]:
    """Rotates 1..3 [B, H, N, d] tensors (bf16 or float32; H may differ) in one launch.

    Entry pair i of the first ``2 * inv_freq.numel()`` entries turns by
    ``(pos_offset + pos_scale * p) * inv_freq[i]``, p = ``positions[b, n]`` (int32 or
    int64, [B, N] or [N]) or n without them, and is multiplied by ``mscale``; pairs are
    (i, i + rot/2), or (2i, 2i + 1) with ``interleaved``.  ``inverse`` turns back: the
    gradient of the input from that of the output.  ``apply[r] = False`` only moves
    tensor r to its output's layout and type.  ``out`` may have any non-overlapping
    strides and may be the inputs themselves, but no element of it is written twice: a
    tensor given twice is refused as ``out``, in place too; without it the outputs are
    contiguous tensors of ``out_dtype`` (default: the inputs' type)."""
    marshal = _abi.marshal()
    marshal.rotary_inputs(xs, inv_freq)
    if apply is not None and len(apply) != len(xs) or out is not None and len(out) != len(xs):
        raise ValueError("apply and out need one entry for each tensor")
    x0 = xs[0]
    if out is None:
        out_dtype = x0.dtype if out_dtype is None else out_dtype
        if out_dtype not in _DTYPES:
            raise TypeError(f"unsupported output dtype {out_dtype}")
    elif out_dtype is not None and any(y.dtype != out_dtype for y in out):
        raise ValueError(f"out must be {out_dtype} tensors")
    with _on(x0.device, stream) as handle:
        status, got = marshal.rotary(xs, out, out_dtype, apply, inv_freq, positions, interleaved, inverse,
                                     mscale, pos_scale, pos_offset, handle)
    check(status, "relkl_rotary")
    if out is not None:
        marshal.written(got)
    return got


def relkl_rotary(x: torch.Tensor, inv_freq: torch.Tensor, *, pos_scale: float = 1.0,
                 pos_offset: float = 0.0, positions: Optional[torch.Tensor] = None,
                 mscale: float = 1.0, interleaved: bool = False, inverse: bool = False,
                 out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                 stream=None) -> torch.Tensor:
    """relkl_rotary_qkv for one tensor."""
    return relkl_rotary_qkv([x], inv_freq, pos_scale=pos_scale, pos_offset=pos_offset,
                            positions=positions, mscale=mscale, interleaved=interleaved,
                            inverse=inverse, out=None if out is None else [out],
                            out_dtype=out_dtype, stream=stream)[0]


class Rotary(torch.autograd.Function):
    """Rotation whose backward turns the gradient back by the same angles."""

    @staticmethod
    def forward(ctx, x, inv_freq, positions, args, out_dtype):
        ctx.save_for_backward(inv_freq, positions)
        ctx.args, ctx.dtype = args, x.dtype
        ctx.elsewhere = (x.requires_grad and x.is_cuda and torch.cuda.is_current_stream_capturing()
                         and _abi.marshal().graph_elsewhere(x))
        return relkl_rotary(x.detach(), inv_freq, positions=positions, out_dtype=out_dtype, **args)

    @staticmethod
    def backward(ctx, dy):
        # autograd would make that stream wait for the captured one, which ends the process
        if ctx.elsewhere and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a leaf of this graph belongs to an eager graph on another stream: drop "
                               "that graph before capturing a backward pass")
        inv_freq, positions = ctx.saved_tensors
        if dy.dim() and dy.stride(-1) != 1:
            dy = dy.contiguous()
        # the rotation is linear: its gradient is the same operator, turned round
        args = dict(ctx.args, inverse=not ctx.args["inverse"])
        return Rotary.apply(dy, inv_freq, positions, args, ctx.dtype), None, None, None, None


def rotary(x: torch.Tensor, inv_freq: torch.Tensor, *, positions: Optional[torch.Tensor] = None,
           pos_scale: float = 1.0, pos_offset: float = 0.0, mscale: float = 1.0,
           interleaved: bool = False, inverse: bool = False,
           out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Differentiable relkl_rotary (the frequencies and positions get no gradient).

    It has a backward pass, itself differentiable, and no forward-mode derivative or rule for
    torch.func's transforms, which refuse it.  The backward pass may be captured into a graph
    once no eager graph of the same leaves, made on another stream, is alive; until then it
    is refused."""
    args = dict(pos_scale=pos_scale, pos_offset=pos_offset, mscale=mscale, interleaved=interleaved,
                inverse=bool(inverse))
    return Rotary.apply(x, inv_freq, positions, args, out_dtype)
