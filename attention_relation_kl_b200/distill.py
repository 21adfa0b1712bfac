"""One layer's distillation step around the relation loss: the frozen teacher's relation
inputs from its 8-bit projections, and the student's update from its weight gradients."""
from __future__ import annotations

from typing import Dict, Optional, Sequence, Tuple

import torch

from . import _abi
from .int8 import relkl_linear_i8, relkl_matmul_i8, relkl_quantize_rows
from .ops import student_weight_grads
from .optim import AdamW
from .positions import RotaryFreqs, relkl_rotary_qkv

__all__ = ["teacher_relations_i8", "student_step"]


def teacher_relations_i8(h_t: torch.Tensor, weights: Dict[str, Sequence[torch.Tensor]], d: int,
                         freqs: RotaryFreqs, *, pos_scale: float = 1.0,
                         positions: Optional[torch.Tensor] = None,
                         interleaved: bool = False) -> Dict[str, torch.Tensor]:
    """Teacher inputs {rel: [B, heads, N, d]} (bf16) of the relations in ``weights``, from its
    hidden states h_t [B, N, D]: ``weights[rel]`` holds the codes and scales of the projection
    [heads * d, D] (relkl_quantize_rows), and a bias if it has one.  q and k are rotated at the
    teacher's positions; v is brought into the same layout by the same launch."""
    if h_t.dim() != 3:
        raise ValueError("expected [B, N, D] hidden states")
    if not 1 <= len(weights) <= 3:
        raise ValueError("1 to 3 relations per call")
    B, N, D = h_t.shape
    # Few tokens are coded by the kernel that multiplies them; more are coded once for all
    # relations: 32768 x 4096 tokens through 32, 8 and 8 heads of 128 and the rotation take
    # 700 us on the GPU, coded for each relation 825.
    codes = None
    if len(weights) > 1 and _abi.lib().relkl_linear_i8_bytes(B * N, D) > 0:
        codes = relkl_quantize_rows(h_t)
    rels, xs = list(weights), []
    for r in rels:
        w, scale, *bias = weights[r]
        if w.shape[0] % d:
            raise ValueError(f"{r} has {w.shape[0]} channels, no multiple of the head size {d}")
        args = dict(bias=bias[0] if bias else None, out_dtype=torch.bfloat16)
        y = relkl_linear_i8(h_t, w, scale, **args) if codes is None else relkl_matmul_i8(*codes, w, scale, **args)
        xs.append(y.view(B, N, w.shape[0] // d, d).transpose(1, 2))
    out = relkl_rotary_qkv(xs, freqs.inv_freq, apply=[r != "v" for r in rels], pos_scale=pos_scale,
                           positions=positions, mscale=freqs.mscale, interleaved=interleaved)
    return dict(zip(rels, out))


def student_step(pairs: Dict[str, Tuple[torch.Tensor, torch.Tensor]], h_s: torch.Tensor,
                 optimizer: AdamW, rope_base: float = 1e4, pos_scale: float = 1.0,
                 causal: bool = True, dkl: Optional[Dict[str, torch.Tensor]] = None, *,
                 freqs: Optional[RotaryFreqs] = None, positions: Optional[torch.Tensor] = None,
                 interleaved: bool = False
                 ) -> Tuple[Dict[str, torch.Tensor], Optional[torch.Tensor]]:
    """student_weight_grads and one step of ``optimizer``, whose parameters are the student's
    projections [D, heads * d] in the order of ``pairs``.  Returns the gradients and, where the
    optimizer clips, their norm."""
    if len(optimizer.params) != len(pairs):
        raise ValueError("the optimizer needs one parameter for each relation, in their order")
    grads = student_weight_grads(pairs, h_s, rope_base, pos_scale, causal, dkl, freqs=freqs,
                                 positions=positions, interleaved=interleaved)
    return grads, optimizer.step([grads[r] for r in pairs])
