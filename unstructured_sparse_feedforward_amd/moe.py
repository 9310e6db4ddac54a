"""A mixture-of-experts layer of activation-sparse ReLU experts for few
tokens (sffn_moe_* of include/sffn.h)."""
from __future__ import annotations

import ctypes
from typing import Dict, Optional, Tuple, Union

import torch

from .binding import (SFFN_BF16, SFFN_MOE_MAX_TOKENS, SFFN_MXFP4, SFFN_OK, SffnError,
                      SffnMoeDesc, SffnMoeWeights, load_library)
from .mxfp4 import MXTensor, _launch

Weight = Union[torch.Tensor, MXTensor]


class SparseMoE:
    """Router, top-k selection, the selected ReLU experts and their weighted
    sum, for calls of up to SFFN_MOE_MAX_TOKENS tokens.

    Weights are passed to each call: ``w_router`` [E, d] bfloat16, and
    ``w_gate``, ``w_up`` (None when non-gated) and ``w_down`` [E, F, d]
    bfloat16, neuron-major as in :class:`SparseFFN`; with
    ``weights="mxfp4"`` the experts' matrices are MXTensors of E F rows and d
    columns, ``mx_quantize(w.view(E * F, d))``.

    ``normalize``: a token's weights are the softmax over its top_k experts
    (default), or over all experts.

    The object holds no device state: each call takes its workspace from
    torch's allocator on the current stream, so calls on different streams
    may overlap and several graphs may be captured.
    """

    def __init__(self, d: int, d_ff: int, n_experts: int, top_k: int, gated: bool = True,
                 normalize: bool = True, weights: str = "bf16"):
        if weights not in ("bf16", "mxfp4"):
            raise ValueError(f"weights must be 'bf16' or 'mxfp4', not {weights!r}")
        self.lib = load_library()
        self.d, self.d_ff, self.n_experts, self.top_k = d, d_ff, n_experts, top_k
        self.gated, self.normalize, self.weights = gated, normalize, weights
        self.desc = SffnMoeDesc(d, d_ff, n_experts, top_k, int(gated), int(normalize),
                                SFFN_MXFP4 if weights == "mxfp4" else SFFN_BF16)
        self._desc = ctypes.byref(self.desc)
        self._bytes: Dict[int, int] = {}
        self.workspace_bytes(1)      # the descriptor's validation

    def workspace_bytes(self, T: int) -> int:
        n = self._bytes.get(T)
        if n is None:
            c = ctypes.c_size_t()
            st = self.lib.sffn_moe_workspace_bytes(ctypes.byref(self.desc), T, ctypes.byref(c))
            if st != SFFN_OK:
                raise SffnError(st, "sffn_moe_workspace_bytes: "
                                    + self.lib.sffn_status_string(st).decode())
            n = self._bytes[T] = c.value
        return n

    def _plain(self, t: torch.Tensor, shape: Tuple[int, ...], dtype: torch.dtype, device,
               what: str) -> int:
        if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous {dtype} tensor {shape} on {device}, not "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    @staticmethod
    def _new(rows: int, cols: int, dtype: torch.dtype, device) -> Tuple[torch.Tensor, int]:
        # (0.3 us less of the host's time than torch.empty of a shape)
        t = torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)
        return t, t.data_ptr()

    def _weight(self, w: Weight, device, what: str) -> Tuple[int, Optional[int]]:
        E, F, d = self.n_experts, self.d_ff, self.d
        if self.weights == "bf16":
            if isinstance(w, MXTensor):
                raise ValueError(f"{what} is an MXTensor: the layer's weights are bf16")
            return self._plain(w, (E, F, d), torch.bfloat16, device, what), None
        if not isinstance(w, MXTensor):
            raise ValueError(f"{what} must be an MXTensor of {E * F} x {d}")
        if w.rows != E * F or w.cols != d or w.device != device:
            raise ValueError(f"{what} must be an MXTensor of {E * F} x {d} on {device}")
        return w._pc, w._ps

    def forward(self, x: torch.Tensor, w_router: torch.Tensor, w_gate: Weight,
                w_up: Optional[Weight], w_down: Weight, y: Optional[torch.Tensor] = None,
                n_tokens: Optional[torch.Tensor] = None, return_routing: bool = False,
                routing: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
        """y [T, d] float32 for ``x`` [T, d] bfloat16; with
        ``return_routing`` (y, ids [T, k] int32, probs [T, k] float32), the
        chosen experts in descending order of their logits and their
        weights. ``n_tokens``, an int32 tensor of one element on the GPU,
        says how many of the rows are tokens: the others are neither read
        nor written (in results made here they are uninitialised). ``y`` and
        ``routing`` (ids, probs) may pass result tensors to reuse."""
        if x.dim() != 2 or not x.is_cuda:
            raise ValueError("x must be a [T, d] tensor on the GPU")
        T, dev = x.shape[0], x.device
        if T > SFFN_MOE_MAX_TOKENS:
            raise ValueError(f"{T} tokens: at most {SFFN_MOE_MAX_TOKENS} a call")
        px = self._plain(x, (T, self.d), torch.bfloat16, dev, "x")
        pr = self._plain(w_router, (self.n_experts, self.d), torch.bfloat16, dev, "w_router")
        g, gs = self._weight(w_gate, dev, "w_gate")
        if self.gated:
            if w_up is None:
                raise ValueError("w_up is missing: the layer is gated")
            u, us = self._weight(w_up, dev, "w_up")
        elif w_up is not None:
            raise ValueError("w_up must be None: the layer is not gated")
        else:
            u = us = None
        dn, ds = self._weight(w_down, dev, "w_down")
        w = SffnMoeWeights(pr, g, u, dn, gs, us, ds)
        pn = None
        if n_tokens is not None:
            pn = self._plain(n_tokens, tuple(n_tokens.shape), torch.int32, dev, "n_tokens")
            if n_tokens.numel() != 1:
                raise ValueError("n_tokens must have one element")
        k = self.top_k
        if y is None:
            y, py = self._new(T, self.d, torch.float32, dev)
        else:
            py = self._plain(y, (T, self.d), torch.float32, dev, "y")
        ids = probs = pi = pp = None
        if routing is not None:
            ids, probs = routing
            pi = self._plain(ids, (T, k), torch.int32, dev, "ids")
            pp = self._plain(probs, (T, k), torch.float32, dev, "probs")
        elif return_routing:
            ids, pi = self._new(T, k, torch.int32, dev)
            probs, pp = self._new(T, k, torch.float32, dev)
        if T > 0:
            nb = self.workspace_bytes(T)
            # torch's allocations are 512-byte aligned
            ws = torch.empty(nb, dtype=torch.uint8, device=dev)
            _launch(dev, "sffn_moe_forward", self.lib.sffn_moe_forward, self._desc, px,
                    ctypes.byref(w), T, pn, py, pi, pp, ws.data_ptr(), nb)
        return (y, ids, probs) if return_routing else y
