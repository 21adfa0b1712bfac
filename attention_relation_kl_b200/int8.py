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
from .ops import _DTYPES, _WS, _cuda, _on, workspace

__all__ = ["relkl_quantize_rows", "relkl_matmul_i8", "relkl_linear_i8"]


def _matrix(x: torch.Tensor, what: str) -> Tuple[int, int, int]:
    """(rows, K, row stride) of x [..., K], whose rows must follow one another evenly."""
    dims = x.dim()
    if dims < 1:
        raise ValueError(f"{what} must have at least one dimension")
    K = x.shape[-1]
    if K > 1 and x.stride(-1) != 1:
        raise ValueError(f"{what}'s last dimension must be contiguous")
    if dims == 2:
        rows, stride = x.shape[0], x.stride(0)
    elif x.is_contiguous():
        rows, stride = x.numel() // K if K else 0, K
    else:
        try:
            flat = x.view(-1, K)
        except RuntimeError:
            raise ValueError(f"{what}'s rows must follow one another at one stride") from None
        rows, stride = flat.shape[0], flat.stride(0)
    return rows, K, stride if rows > 1 else max(stride, K)


def _codes(q: torch.Tensor, what: str) -> int:
    """Row stride of a [rows, K] int8 matrix laid out as relkl_quantize_rows lays it out."""
    if q.dtype != torch.int8 or q.dim() != 2:
        raise ValueError(f"{what} must be an int8 matrix")
    K = q.shape[1]
    stride = q.stride(0) if q.shape[0] > 1 else max(q.stride(0), (K + 15) // 16 * 16)
    if (K > 1 and q.stride(1) != 1) or stride % 16 or stride < K or q.data_ptr() % 16:
        raise ValueError(f"{what}'s rows must be contiguous and start at 16-byte boundaries, as "
                         "relkl_quantize_rows lays them out")
    return stride


def _vector(v: Optional[torch.Tensor], n: int, what: str, index: int) -> int:
    if v is None:
        return 0
    if v.dtype != torch.float32 or v.dim() != 1 or v.numel() != n or not v.is_contiguous() or \
            v.get_device() != index:
        raise ValueError(f"{what} must be a contiguous float32 vector of {n} on the inputs' device")
    return v.data_ptr()


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
    _cuda(x, "x")
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    rows, K, stride = _matrix(x, "x")
    line = 128 if K >= 128 else 16
    pitch = (K + line - 1) // line * line
    with _on(x.device, stream) as handle:
        q = torch.empty(rows, pitch, dtype=torch.int8, device=x.device)
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
        if rows:
            check(_abi.lib().relkl_quantize_rows(rows, K, x.data_ptr(), _DTYPES[x.dtype], stride,
                                                 q.data_ptr(), pitch, scale.data_ptr(), handle),
                  "relkl_quantize_rows")
    return q[:, :K], scale


def relkl_matmul_i8(q: torch.Tensor, q_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                    *, bias: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                    out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """[rows, cols] product of codes q [rows, K] and w [cols, K] (relkl_quantize_rows), times
    their scales, plus ``bias`` (float32 [cols]).  The sums are exact (0 < K < 131072)."""
    _cuda(q, "q")
    device, index = q.device, q.get_device()
    if w.device != device:
        raise ValueError("q and w must live on the same device")
    q_stride, w_stride = _codes(q, "q"), _codes(w, "w")
    (rows, K), cols = q.shape, w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"q has rows of {K} codes, w of {w.shape[1]}")
    qs, s = _vector(q_scale, rows, "q_scale", index), _vector(w_scale, cols, "w_scale", index)
    b = _vector(bias, cols, "bias", index)
    with _on(device, stream) as handle:
        y = _output(out, (rows, cols), out_dtype, device)
        if out is not None:
            _apart(out, q, w, q_scale, w_scale, bias)
        _, _, y_stride = _matrix(y, "out")
        ws = _record(device, ws)
        check(_abi.lib().relkl_matmul_i8(rows, cols, K, q.data_ptr(), q_stride, qs, w.data_ptr(),
                                         w_stride, s, b, y.data_ptr(), _DTYPES[out_dtype], y_stride,
                                         ws.data_ptr(), ws.numel(), handle), "relkl_matmul_i8")
    return y


def relkl_linear_i8(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, *,
                    bias: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                    out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """x [..., K] (bf16 or float32) through a projection in 8 bits: its rows are coded as by
    relkl_quantize_rows and multiplied with the codes w [cols, K] as by relkl_matmul_i8.
    Returns [..., cols] of ``out_dtype`` (x's type without it); one kernel for up to 8 rows."""
    _cuda(x, "x")
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    device, index = x.device, x.get_device()
    if w.device != device:
        raise ValueError("x and w must live on the same device")
    rows, K, stride = _matrix(x, "x")
    w_stride, cols = _codes(w, "w"), w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"x has rows of {K} elements, w of {w.shape[1]}")
    s, b = _vector(w_scale, cols, "w_scale", index), _vector(bias, cols, "bias", index)
    out_dtype = x.dtype if out_dtype is None else out_dtype
    lib = _abi.lib()
    with _on(device, stream) as handle:
        y = _output(out, (*x.shape[:-1], cols), out_dtype, device)
        y_stride = cols
        if out is not None:
            _apart(out, x, w, w_scale, bias)
            _, _, y_stride = _matrix(y, "out")
        nbytes = lib.relkl_linear_i8_bytes(rows, K)
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
        ws = _record(device, ws)
        check(lib.relkl_linear_i8(rows, cols, K, x.data_ptr(), _DTYPES[x.dtype], stride, w.data_ptr(),
                                  w_stride, s, b, y.data_ptr(), _DTYPES[out_dtype], y_stride,
                                  None if scratch is None else scratch.data_ptr(), nbytes, ws.data_ptr(), ws.numel(), handle), "relkl_linear_i8")
    return y
