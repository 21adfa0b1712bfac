"""Products in 8-bit integers with a scale for each token and each channel.

The teacher is frozen, so its projections are coded once (``relkl_quantize_rows`` of the
[out, in] weight) and kept in 8 bits; every call codes its tokens by their largest
magnitude and multiplies the codes exactly.  There is no gradient: nothing behind the
teacher is trained.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _abi
from ._abi import check
from .ops import _DTYPES, _WS, _on, workspace

__all__ = ["relkl_quantize_rows", "relkl_matmul_i8", "relkl_linear_i8"]


def _record(device: torch.device, ws: Optional[torch.Tensor]) -> torch.Tensor:
    if ws is not None:
        if ws.device != device:
            raise ValueError("ws must be on the inputs' device")
        return ws
    ws = _WS.get(device.index)
    if ws is None:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("call workspace(device) before capturing the first call of a device")
        ws = workspace(device)
    return ws


def _output(out: Optional[torch.Tensor], shape, dtype: torch.dtype, device: torch.device):
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported output dtype {dtype}")
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype or out.device != device:
        raise ValueError(f"out must be a {dtype} tensor of shape {tuple(shape)} on {device}")
    return out


def _extent(t: torch.Tensor) -> Tuple[int, int]:
    begin = t.data_ptr()
    return begin, begin + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


def _apart(out: torch.Tensor, *inputs: Optional[torch.Tensor]) -> None:
    """Refuses an output whose addresses meet an input's."""
    if out.numel() == 0:
        return
    a0, a1 = _extent(out)
    for t in inputs:
        if t is not None and t.numel():
            b0, b1 = _extent(t)
            if a0 < b1 and b0 < a1:
                raise ValueError("out must not overlap an input")


def relkl_quantize_rows(x: torch.Tensor, *, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Codes and scales of the rows of x [..., K] (bf16 or float32): int8 [rows, K], a view
    of rows that start at 16-byte boundaries, rint(127 x / max|row|) with ties to even, and
    float32 [rows], max|row| / 127.  A row of zeros gets scale 0, one that holds an infinity
    or a NaN a NaN scale.  For a weight [out, in] the rows are its channels."""
    rows, K, stride, ptr, dtype, _ = _abi.marshal().matrix(x, "x")
    line = 128 if K >= 128 else 16
    pitch = (K + line - 1) // line * line
    with _on(x.device, stream) as handle:
        q = torch.empty(rows, pitch, dtype=torch.int8, device=x.device)
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
        if rows:
            check(_abi.lib().relkl_quantize_rows(rows, K, ptr, dtype, stride, q.data_ptr(), pitch,
                                                 scale.data_ptr(), handle), "relkl_quantize_rows")
    return q[:, :K], scale


def relkl_matmul_i8(q: torch.Tensor, q_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                    *, bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                    out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """[rows, cols] product of codes q [rows, K] and w [cols, K] (relkl_quantize_rows), times
    their scales, plus ``bias`` (float32 [cols]).  The sums are exact (0 < K < 131072)."""
    m, device, index = _abi.marshal(), q.device, q.get_device()
    rows, K, q_stride, q_ptr = m.codes(q, "q", -1)
    cols, Kw, w_stride, w_ptr = m.codes(w, "w", index)
    if Kw != K:
        raise ValueError(f"q has rows of {K} codes, w of {Kw}")
    qs, s = m.vector(q_scale, rows, "q_scale", index), m.vector(w_scale, cols, "w_scale", index)
    b = m.vector(bias, cols, "bias", index)
    with _on(device, stream) as handle:
        y = _output(out, (rows, cols), out_dtype, device)
        if out is not None:
            _apart(out, q, w, q_scale, w_scale, bias)
        _, _, y_stride, y_ptr, y_type, _ = m.matrix(y, "out")
        ws = _record(device, ws)
        check(_abi.lib().relkl_matmul_i8(rows, cols, K, q_ptr, q_stride, qs, w_ptr, w_stride, s, b,
                                         y_ptr, y_type, y_stride, ws.data_ptr(), ws.numel(), handle),
              "relkl_matmul_i8")
    if out is not None:
        m.written([out])
    return y


def relkl_linear_i8(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, *,
                    bias: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                    out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """x [..., K] (bf16 or float32) through a projection in 8 bits: its rows are coded as by
    relkl_quantize_rows and multiplied with the codes w [cols, K] as by relkl_matmul_i8.
    Returns [..., cols] of ``out_dtype`` (x's type without it); one kernel for up to 4 rows.
    ``out`` may have rows at any one stride; its addresses may not meet an input's."""
    m = _abi.marshal()
    index = m.matrix(x, "x")[5]
    device = x.device
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if out is not None:
        cols = m.codes(w, "w", index)[0]
        _output(out, (*x.shape[:-1], cols), out_dtype, device)
        _apart(out, x, w, w_scale, bias)
    with _on(device, stream) as handle:
        status, y = m.linear_i8(x, w, w_scale, bias, out_dtype, out, _record(device, ws), handle)
    check(status, "relkl_linear_i8")
    if out is not None:
        m.written([out])
    return y
