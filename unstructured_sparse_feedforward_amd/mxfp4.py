"""Microscaled 4-bit floating point (MXFP4) matrices: quantisation, the
values back, and the product of two of them (sffn_mx_* of include/sffn.h).

As everywhere in this package, the calls only marshal torch tensors: they
run on the tensors' device, on that device's current stream, synchronise
nothing and may be captured into a graph.
"""
from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional

import torch

from .binding import SFFN_BF16, SFFN_F32, SFFN_OK, SffnError, load_library

_DTYPES = {torch.float32: SFFN_F32, torch.bfloat16: SFFN_BF16}
_SAME_DEVICE = contextlib.nullcontext()


class MXTensor(NamedTuple):
    """A matrix of ``rows`` x ``cols`` elements in MXFP4, one scale for 32
    elements along a row. ``codes`` [rows, Kp / 2] and ``scales`` [Kp / 128,
    rows, 4] are uint8 tensors, Kp = cols rounded up to 128; include/sffn.h
    gives the layout."""

    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int


def _on(device: torch.device):
    """The library launches on the current device."""
    if device.index == torch.cuda.current_device():
        return _SAME_DEVICE
    return torch.cuda.device(device)


def _check(st: int, what: str) -> None:
    if st != SFFN_OK:
        raise SffnError(st, f"{what}: {load_library().sffn_status_string(st).decode()}")


def _matrix(t: torch.Tensor, what: str) -> int:
    """The row stride of a 2-D float matrix with contiguous rows."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be on the GPU")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{what} must be float32 or bfloat16, not {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{what} must have 2 dimensions, not {t.dim()}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must have contiguous rows")
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{what}'s rows overlap")
    return ld


def check_mx(q: MXTensor, what: str) -> None:
    """Raise ValueError unless ``q`` is whole: uint8, contiguous, on one GPU,
    of the shapes its rows and columns ask for."""
    Kp = (q.cols + 127) // 128 * 128
    if q.codes.shape != (q.rows, Kp // 2) or q.scales.shape != (Kp // 128, q.rows, 4):
        raise ValueError(f"{what}: codes {tuple(q.codes.shape)} and scales "
                         f"{tuple(q.scales.shape)} do not hold {q.rows} x {q.cols} elements")
    for t in (q.codes, q.scales):
        if t.dtype != torch.uint8 or not t.is_contiguous():
            raise ValueError(f"{what}: codes and scales must be contiguous uint8 tensors")
    if not q.codes.is_cuda or q.codes.device != q.scales.device:
        raise ValueError(f"{what}: codes and scales must be on one GPU")


def mx_empty(rows: int, cols: int, device) -> MXTensor:
    """An MXTensor with uninitialised memory."""
    g = (cols + 127) // 128
    return MXTensor(torch.empty((rows, g * 64), dtype=torch.uint8, device=device),
                    torch.empty((g, rows, 4), dtype=torch.uint8, device=device), rows, cols)


def mx_quantize(x: torch.Tensor, transposed: bool = False,
                out: Optional[MXTensor] = None) -> MXTensor:
    """``x`` [rows, cols] (float32 or bfloat16, contiguous rows, any row
    stride) in MXFP4. With ``transposed`` the result is x^T's, its blocks
    down the columns of x: the form of a weight stored [F, d] for a product
    over F. ``out`` may pass an MXTensor of the result's size to reuse."""
    ld = _matrix(x, "x")
    rows, cols = x.shape
    R, K = (cols, rows) if transposed else (rows, cols)
    if out is None:
        out = mx_empty(R, K, x.device)
    else:
        check_mx(out, "out")
        if (out.rows, out.cols) != (R, K) or out.codes.device != x.device:
            raise ValueError(f"out must be {R} x {K} on {x.device}")
    with _on(x.device):
        _check(load_library().sffn_mx_quantize(
            x.data_ptr(), _DTYPES[x.dtype], rows, cols, ld, int(transposed), out.codes.data_ptr(),
            out.scales.data_ptr(), torch.cuda.current_stream().cuda_stream), "sffn_mx_quantize")
    return out


def mx_dequantize(q: MXTensor, dtype: torch.dtype = torch.float32,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of ``q`` [rows, cols], exact, as float32 or bfloat16 (in
    ``out`` when given: contiguous rows, any row stride)."""
    check_mx(q, "q")
    if out is None:
        if dtype not in _DTYPES:
            raise ValueError(f"dtype must be float32 or bfloat16, not {dtype}")
        out = torch.empty((q.rows, q.cols), dtype=dtype, device=q.codes.device)
    ld = _matrix(out, "out")
    if out.shape != (q.rows, q.cols) or out.device != q.codes.device:
        raise ValueError(f"out must be {q.rows} x {q.cols} on {q.codes.device}")
    with _on(out.device):
        _check(load_library().sffn_mx_dequantize(
            q.codes.data_ptr(), q.scales.data_ptr(), q.rows, q.cols, out.data_ptr(),
            _DTYPES[out.dtype], ld, torch.cuda.current_stream().cuda_stream),
            "sffn_mx_dequantize")
    return out


def mx_matmul(a: MXTensor, b: MXTensor, dtype: torch.dtype = torch.float32,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a b^T for ``a`` [M, K] and ``b`` [N, K]: [M, N] float32 or bfloat16
    (in ``out`` when given: contiguous rows, any row stride). Sums are
    float32, rounded once when stored as bfloat16."""
    check_mx(a, "a")
    check_mx(b, "b")
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b {b.cols}")
    if a.codes.device != b.codes.device:
        raise ValueError("a and b must be on one GPU")
    if out is None:
        if dtype not in _DTYPES:
            raise ValueError(f"dtype must be float32 or bfloat16, not {dtype}")
        out = torch.empty((a.rows, b.rows), dtype=dtype, device=a.codes.device)
    ld = _matrix(out, "out")
    if out.shape != (a.rows, b.rows) or out.device != a.codes.device:
        raise ValueError(f"out must be {a.rows} x {b.rows} on {a.codes.device}")
    with _on(out.device):
        _check(load_library().sffn_mx_matmul(
            a.codes.data_ptr(), a.scales.data_ptr(), a.rows, b.codes.data_ptr(),
            b.scales.data_ptr(), b.rows, a.cols, out.data_ptr(), _DTYPES[out.dtype], ld,
            torch.cuda.current_stream().cuda_stream), "sffn_mx_matmul")
    return out
