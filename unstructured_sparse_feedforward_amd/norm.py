"""What stands between two layers: the residual's addition and the
root-mean-square norm of the sum, and its gradient (sffn_rms_norm* of
include/sffn.h)."""
from __future__ import annotations

import ctypes
from typing import Dict, Optional, Tuple, Union

import torch

from .binding import (SFFN_F32, SFFN_MXFP8, SFFN_OK, SffnError, SffnNorm, SffnNormGrad,
                      load_library)
from .mxfp4 import _DTYPES, _launch, _matrix, _result
from .mxfp8 import MX8Tensor, _mx8_result


def _like(t: torch.Tensor, rows: int, cols: int, device, what: str) -> Tuple[int, int]:
    """(row stride, type's number) of a matrix that has to be rows x cols."""
    r, c, ld, dt = _matrix(t, what)
    if r != rows or c != cols or t.device != device:
        raise ValueError(f"{what} must be {rows} x {cols} on {device}")
    return ld, dt


def _vector(t: torch.Tensor, n: int, device, what: str, f32: bool = False) -> Tuple[int, int]:
    """(pointer, type's number) of a contiguous vector of n elements."""
    dt = _DTYPES.get(t.dtype)
    if dt is None or (f32 and dt != SFFN_F32):
        raise ValueError(f"{what} must be float32{'' if f32 else ' or bfloat16'}, not {t.dtype}")
    if t.shape != (n,) or t.device != device or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous vector of {n} elements on {device}")
    return t.data_ptr(), dt


def _count(n: Optional[torch.Tensor], device, what: str) -> Optional[int]:
    if n is None:
        return None
    if n.dtype != torch.int32 or n.numel() != 1 or n.device != device:
        raise ValueError(f"{what} must be an int32 tensor of one element on {device}")
    return n.data_ptr()


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
             residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             dtype: Union[torch.dtype, str] = torch.bfloat16,
             out: Union[torch.Tensor, MX8Tensor, None] = None,
             residual_out: Optional[torch.Tensor] = None,
             rstd: Optional[torch.Tensor] = None, n_rows: Optional[torch.Tensor] = None):
    """The root-mean-square norm of the rows of s = ``x`` + ``residual``:
    s / sqrt(mean(s^2) + eps) * weight.

    ``x`` and ``residual`` are [rows, cols] matrices, float32 or bfloat16 each
    (contiguous rows, any row stride, up to 16384 columns), ``weight`` [cols] is
    float32 or bfloat16. The result is of ``dtype`` float32, bfloat16 or
    "mxfp8" (an MX8Tensor, for :func:`mx_matmul`), or ``out``, which sets the
    type. With a residual (result, s) is returned, s rounded to the residual's
    type, the norm being that of the rounded sum; it is made here or is
    ``residual_out``, which may be the residual itself (``out`` and
    ``residual_out`` are either an operand, rows in the same places, or share no
    memory with any). ``rstd`` [rows] float32
    receives 1 / sqrt(mean(s^2) + eps) for :func:`rms_norm_backward`.
    ``n_rows``, an int32 tensor of one element on the GPU, says how many of the
    rows count: the results of the others are left as they were."""
    rows, cols, ldx, xd = _matrix(x, "x")
    dev = x.device
    pr = po = None
    ldr = ldro = rd = 0
    if residual is not None:
        ldr, rd = _like(residual, rows, cols, dev, "residual")
        if residual_out is None:
            residual_out, ldro = torch.empty_strided((rows, cols), (cols, 1), dtype=residual.dtype,
                                                     device=dev), cols
        else:
            ldro, od = _like(residual_out, rows, cols, dev, "residual_out")
            if od != rd:
                raise ValueError("residual_out must have the residual's type")
        pr, po = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out is given without a residual")
    pw, wd = (None, 0) if weight is None else _vector(weight, cols, dev, "weight")
    ps = None if rstd is None else _vector(rstd, rows, dev, "rstd", f32=True)[0]
    pn = _count(n_rows, dev, "n_rows")
    if isinstance(out, MX8Tensor) or (out is None and dtype == "mxfp8"):
        out = _mx8_result(out, rows, cols, dev)
        py, sc, ldo, yd = out._pc, out._ps, 0, SFFN_MXFP8
    else:
        out, ldo, yd = _result(out, rows, cols, dtype, dev)
        py, sc = out.data_ptr(), None
    _launch(dev, "sffn_rms_norm", load_library().sffn_rms_norm,
            SffnNorm(x.data_ptr(), pr, po, pw, py, sc, ps, ldx, ldr, ldro, ldo, xd, rd, wd, yd),
            rows, cols, eps, pn)
    return out if residual is None else (out, residual_out)


_ws_bytes: Dict[Tuple[int, int], int] = {}


def _workspace_bytes(rows: int, cols: int) -> int:
    n = _ws_bytes.get((rows, cols))
    if n is None:
        lib, c = load_library(), ctypes.c_size_t()
        st = lib.sffn_rms_norm_backward_workspace_bytes(rows, cols, ctypes.byref(c))
        if st != SFFN_OK:
            raise SffnError(st, "sffn_rms_norm_backward_workspace_bytes: "
                                + lib.sffn_status_string(st).decode())
        if len(_ws_bytes) > 1024:
            _ws_bytes.clear()
        n = _ws_bytes[(rows, cols)] = c.value
    return n


def rms_norm_backward(dy: torch.Tensor, s: torch.Tensor, rstd: torch.Tensor,
                      weight: Optional[torch.Tensor] = None,
                      dstream: Optional[torch.Tensor] = None,
                      dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                      dweight: Optional[torch.Tensor] = None):
    """The gradient of :func:`rms_norm` from that of its result, ``dy``:
    (ds, dweight). ``s`` is the normalised sum (x where there was no residual)
    and ``rstd`` what the forward call wrote. ds, the gradient of x and of the
    residual alike, has ``dstream`` added, the gradient that reaches s from
    elsewhere; it is of ``dtype``, or ``out`` (which may be dy, s or dstream, and
    shares no memory with them otherwise). Every row counts: after a forward call
    with ``n_rows`` pass the valid ones alone. dweight [cols] float32 (``dweight`` when given) is None without a
    weight."""
    rows, cols, lddy, yd = _matrix(dy, "dy")
    dev = dy.device
    lds, sd = _like(s, rows, cols, dev, "s")
    pr, _ = _vector(rstd, rows, dev, "rstd", f32=True)
    pi, ldi, di = None, 0, 0
    if dstream is not None:
        ldi, di = _like(dstream, rows, cols, dev, "dstream")
        pi = dstream.data_ptr()
    pw = pdw = pws = None
    wd = nb = 0
    if weight is not None:
        pw, wd = _vector(weight, cols, dev, "weight")
        if dweight is None:
            dweight = torch.empty(cols, dtype=torch.float32, device=dev)
            pdw = dweight.data_ptr()
        else:
            pdw, _ = _vector(dweight, cols, dev, "dweight", f32=True)
        nb = _workspace_bytes(rows, cols)
        if nb > 0:
            # torch's allocations are 512-byte aligned
            ws = torch.empty(nb, dtype=torch.uint8, device=dev)
            pws = ws.data_ptr()
    elif dweight is not None:
        raise ValueError("dweight is given without a weight")
    out, ldo, od = _result(out, rows, cols, dtype, dev)
    _launch(dev, "sffn_rms_norm_backward", load_library().sffn_rms_norm_backward,
            SffnNormGrad(dy.data_ptr(), s.data_ptr(), pi, pw, pr, out.data_ptr(), pdw, lddy, lds,
                         ldi, ldo, yd, sd, di, wd, od), rows, cols, pws, nb)
    return out, dweight
