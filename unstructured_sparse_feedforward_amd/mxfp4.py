"""Microscaled 4-bit floating point (MXFP4) matrices: quantisation, the
values back, and the product of two of them (sffn_mx_* of include/sffn.h).

As everywhere in this package, the calls only marshal torch tensors: they
run on the tensors' device, on that device's current stream, synchronise
nothing and may be captured into a graph.
"""
from __future__ import annotations

from typing import Optional

import torch

from .binding import SFFN_BF16, SFFN_F32, SFFN_OK, SffnError, load_library

_DTYPES = {torch.float32: SFFN_F32, torch.bfloat16: SFFN_BF16}

# The current stream's handle. A small call's time is the host's, and the
# public call, which builds a Stream object, takes 3 us of it (this one 0.1).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    def _raw_stream(index: int) -> int:
        return torch.cuda.current_stream(index).cuda_stream


class MXTensor:
    """A matrix of ``rows`` x ``cols`` elements in MXFP4, one scale for 32
    elements along a row. ``codes`` [rows, Kp / 2] and ``scales`` [Kp / 128,
    rows, 4] are uint8 tensors, Kp = cols rounded up to 128; include/sffn.h
    gives the layout. Made by :func:`mx_quantize` or :func:`mx_empty`, or
    from codes and scales kept elsewhere (contiguous, on one GPU; the codes
    of elements from cols on are 0). The scale bytes of blocks that lie from
    cols on have to be 0 for a product: here those of ``scales`` are cleared,
    on its device's current stream."""

    __slots__ = ("rows", "cols", "device", "_codes", "_scales", "_buf", "_pc", "_ps")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int):
        G = (cols + 127) // 128
        if rows < 0 or cols < 0 or codes.shape != (rows, G * 64) or scales.shape != (G, rows, 4):
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not "
                             f"hold {rows} x {cols} elements")
        for t in (codes, scales):
            if t.dtype != torch.uint8 or not t.is_contiguous():
                raise ValueError("codes and scales must be contiguous uint8 tensors")
        if not codes.is_cuda or codes.device != scales.device:
            raise ValueError("codes and scales must be on one GPU")
        live = -(-cols // 32) % 4
        if live:
            with torch.inference_mode():   # scales may have been made in it
                scales[-1, :, live:].zero_()
        self.rows, self.cols, self.device = rows, cols, codes.device
        self._codes, self._scales, self._buf = codes, scales, None
        self._pc, self._ps = codes.data_ptr(), scales.data_ptr()

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            row = (self.cols + 127) // 128 * 64
            self._codes = self._buf[:self.rows * row].view(self.rows, row)
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            G = (self.cols + 127) // 128
            self._scales = self._buf[self.rows * G * 64:].view(G, self.rows, 4)
        return self._scales


def mx_empty(rows: int, cols: int, device) -> MXTensor:
    """An MXTensor with uninitialised memory: one buffer, the codes and then
    the scales."""
    g = (cols + 127) // 128
    q = MXTensor.__new__(MXTensor)
    q._buf = buf = torch.empty(rows * g * 68, dtype=torch.uint8, device=device)
    if not buf.is_cuda:
        raise ValueError("device must be a GPU")
    q.rows, q.cols, q.device, q._codes, q._scales = rows, cols, buf.device, None, None
    q._pc = buf.data_ptr()
    q._ps = q._pc + rows * g * 64
    return q


def _launch(device: torch.device, what: str, f, *args) -> None:
    """f(*args, stream) on ``device`` (the library launches on the current
    device) and its current stream."""
    i = device.index
    if i == torch.cuda.current_device():
        st = f(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            st = f(*args, _raw_stream(i))
    if st != SFFN_OK:
        raise SffnError(st, f"{what}: {load_library().sffn_status_string(st).decode()}")


def _matrix(t: torch.Tensor, what: str):
    """(rows, columns, row stride, type's number) of a 2-D float matrix with
    contiguous rows."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be on the GPU")
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{what} must be float32 or bfloat16, not {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{what} must have 2 dimensions, not {t.dim()}")
    rows, cols = t.shape
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{what} must have contiguous rows")
    if rows <= 1:
        return rows, cols, cols, dt
    if ld < cols:
        raise ValueError(f"{what}'s rows overlap")
    return rows, cols, ld, dt


def _result(out: Optional[torch.Tensor], rows: int, cols: int, dtype: torch.dtype,
            device: torch.device):
    """(out, its row stride, its type's number), made when not given."""
    if out is None:
        dt = _DTYPES.get(dtype)
        if dt is None:
            raise ValueError(f"dtype must be float32 or bfloat16, not {dtype}")
        # (0.3 us less of the host's time than torch.empty of a shape)
        out = torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)
        return out, cols, dt
    r, c, ld, dt = _matrix(out, "out")
    if r != rows or c != cols or out.device != device:
        raise ValueError(f"out must be {rows} x {cols} on {device}")
    return out, ld, dt


def mx_quantize(x: torch.Tensor, transposed: bool = False,
                out: Optional[MXTensor] = None) -> MXTensor:
    """``x`` [rows, cols] (float32 or bfloat16, contiguous rows, any row
    stride) in MXFP4. With ``transposed`` the result is x^T's, its blocks
    down the columns of x: the form of a weight stored [F, d] for a product
    over F. ``out`` may pass an MXTensor of the result's size to reuse."""
    rows, cols, ld, dt = _matrix(x, "x")
    R, K = (cols, rows) if transposed else (rows, cols)
    device = x.device
    if out is None:
        out = mx_empty(R, K, device)
    elif out.rows != R or out.cols != K or out.device != device:
        raise ValueError(f"out must be {R} x {K} on {device}")
    _launch(device, "sffn_mx_quantize", load_library().sffn_mx_quantize, x.data_ptr(), dt,
            rows, cols, ld, 1 if transposed else 0, out._pc, out._ps)
    return out


def mx_dequantize(q: MXTensor, dtype: torch.dtype = torch.float32,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values of ``q`` [rows, cols], exact, as float32 or bfloat16 (in
    ``out`` when given: contiguous rows, any row stride)."""
    out, ld, dt = _result(out, q.rows, q.cols, dtype, q.device)
    _launch(q.device, "sffn_mx_dequantize", load_library().sffn_mx_dequantize, q._pc, q._ps,
            q.rows, q.cols, out.data_ptr(), dt, ld)
    return out


def mx_matmul(a: MXTensor, b: MXTensor, dtype: torch.dtype = torch.float32,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """a b^T for ``a`` [M, K] and ``b`` [N, K]: [M, N] float32 or bfloat16
    (in ``out`` when given: contiguous rows, any row stride). Sums are
    float32, rounded once when stored as bfloat16."""
    if a.cols != b.cols:
        raise ValueError(f"a has {a.cols} columns, b {b.cols}")
    if a.device != b.device:
        raise ValueError("a and b must be on one GPU")
    out, ld, dt = _result(out, a.rows, b.rows, dtype, a.device)
    _launch(a.device, "sffn_mx_matmul", load_library().sffn_mx_matmul, a._pc, a._ps, a.rows, b._pc,
            b._ps, b.rows, a.cols, out.data_ptr(), dt, ld)
    return out
