"""Microscaled 8-bit floating point (MXFP8) matrices, the form of activations
beside 4-bit weights: quantisation and the values back (sffn_mx8_* of
include/sffn.h). :func:`mx_matmul` multiplies them with MXTensors, and
:func:`rms_norm` writes them.
"""
from __future__ import annotations

from typing import Optional

import torch

from .binding import load_library
from .mxfp4 import _MX, _launch, _matrix, _result


class MX8Tensor(_MX):
    """A matrix of ``rows`` x ``cols`` elements in MXFP8 (e4m3), one scale for
    32 elements along a row. ``codes`` [rows, Kp] and ``scales`` [Kp / 128,
    rows, 4] are uint8 tensors, Kp = cols rounded up to 128. Made by
    :func:`mx8_quantize`, :func:`rms_norm` or :func:`mx8_empty`, or from codes
    and scales kept elsewhere, as an MXTensor."""

    __slots__ = ()
    BITS = 8


def mx8_empty(rows: int, cols: int, device) -> MX8Tensor:
    """An MX8Tensor with uninitialised memory: one buffer, the codes and then
    the scales."""
    return MX8Tensor._empty(rows, cols, device)


def _mx8_result(out: Optional[MX8Tensor], rows: int, cols: int, device) -> MX8Tensor:
    if out is None:
        return MX8Tensor._empty(rows, cols, device)
    if (not isinstance(out, MX8Tensor) or out.rows != rows or out.cols != cols
            or out.device != device):
        raise ValueError(f"out must be an MX8Tensor of {rows} x {cols} on {device}")
    return out


def mx8_quantize(x: torch.Tensor, out: Optional[MX8Tensor] = None) -> MX8Tensor:
    """``x`` [rows, cols] (float32 or bfloat16, contiguous rows, any row
    stride) in MXFP8. ``out`` may pass an MX8Tensor of its size to reuse."""
    rows, cols, ld, dt = _matrix(x, "x")
    out = _mx8_result(out, rows, cols, x.device)
    _launch(x.device, "sffn_mx8_quantize", load_library().sffn_mx8_quantize, x.data_ptr(), dt,
            rows, cols, ld, out._pc, out._ps)
    return out


def mx8_dequantize(q: MX8Tensor, dtype: torch.dtype = torch.float32,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of ``q`` [rows, cols] as float32 or bfloat16, exact (bfloat16
    down to its subnormals), in ``out`` when given (contiguous rows, any row
    stride)."""
    if not isinstance(q, MX8Tensor):
        raise ValueError("q must be an MX8Tensor")
    out, ld, dt = _result(out, q.rows, q.cols, dtype, q.device)
    _launch(q.device, "sffn_mx8_dequantize", load_library().sffn_mx8_dequantize, q._pc, q._ps,
            q.rows, q.cols, out.data_ptr(), dt, ld)
    return out
