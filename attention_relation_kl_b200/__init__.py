"""B200-native (sm_100a) linear-memory relation-KL distillation loss.

The hot path of LinearARD's relation distillation: per-row KL between the
row-softmaxed Q/Q, K/K and V/V self-relations of a frozen teacher and a
RoPE-scaled student, and its gradient dL/dX_s, without an N x N matrix.
Compute runs in librelkl.so (tcgen05/TMA kernels); this package only marshals
PyTorch tensors into its C ABI (include/relkl.h).
"""
from .ops import (RelationKL, make_desc, relation_kl, relkl_bwd, relkl_bwd_qkv, relkl_fwd,
                  relkl_fwd_noalloc, relkl_fwd_qkv, relkl_get_device_error, relkl_path_for, relkl_set_wait_timeout_ns,
                  relkl_workspace_bytes, relkl_workspace_init, workspace, relkl_rope_bwd,
                  relkl_weight_grad, student_weight_grads, relkl_cast_bf16)
from .positions import (Rotary, RotaryFreqs, relkl_rotary, relkl_rotary_qkv, rotary, rotary_freqs)
from .optim import AdamW, AdamWState, adamw_state, relkl_adamw, relkl_grad_norm
from .int8 import relkl_linear_i8, relkl_matmul_i8, relkl_quantize_rows
from .distill import student_step, teacher_relations_i8

__all__ = ["RelationKL", "make_desc", "relation_kl", "relkl_bwd", "relkl_bwd_qkv", "relkl_fwd",
           "relkl_fwd_noalloc", "relkl_fwd_qkv", "relkl_get_device_error", "relkl_path_for",
           "relkl_set_wait_timeout_ns", "relkl_workspace_bytes", "relkl_workspace_init",
           "workspace", "relkl_rope_bwd", "relkl_weight_grad", "student_weight_grads",
           "relkl_cast_bf16", "Rotary", "RotaryFreqs", "relkl_rotary", "relkl_rotary_qkv", "rotary",
           "rotary_freqs", "AdamW", "AdamWState", "adamw_state", "relkl_adamw", "relkl_grad_norm",
           "relkl_linear_i8", "relkl_matmul_i8", "relkl_quantize_rows",
           "student_step", "teacher_relations_i8"]
