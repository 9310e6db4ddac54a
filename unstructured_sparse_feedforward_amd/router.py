"""The choice of a token's experts from a router's logits, and the logits'
gradient (sffn_route* of include/sffn.h)."""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .binding import SFFN_OK, SffnError, SffnRouteDesc, load_library
from .mxfp4 import _launch, _result
from .norm import _count, _like, _vector


class MoERouter:
    """Chooses ``top_k`` of ``n_experts`` experts for every token by the scores
    s, the softmax of the token's logits or (``scores="sigmoid"``) 1 / (1 +
    exp(-logit)), plus a bias for balance. With ``groups`` the experts, in
    groups of n_experts / groups consecutive ones, are chosen from the
    ``top_groups`` groups whose ``group_best`` (1 or 2) largest sums of score
    and bias are largest. A chosen expert's weight is ``scale`` s, or
    (``normalize``, the default) scale s over the sum of the chosen experts'
    s. Ties go to the lower index.

    The object holds no device state."""

    def __init__(self, n_experts: int, top_k: int, scores: str = "softmax", groups: int = 1,
                 top_groups: Optional[int] = None, group_best: int = 1, normalize: bool = True,
                 scale: float = 1.0):
        if scores not in ("softmax", "sigmoid"):
            raise ValueError(f"scores must be 'softmax' or 'sigmoid', not {scores!r}")
        self.lib = load_library()
        self.n_experts, self.top_k, self.scores = n_experts, top_k, scores
        self.groups, self.group_best = groups, group_best
        self.top_groups = groups if top_groups is None else top_groups
        self.normalize, self.scale = normalize, scale
        self.desc = SffnRouteDesc(n_experts, top_k, groups, self.top_groups, group_best,
                                  int(scores == "sigmoid"), int(normalize), scale)
        self._desc = ctypes.byref(self.desc)
        # the descriptor's validation
        st = self.lib.sffn_route(self._desc, None, 0, 0, 0, None, None, None, None, None)
        if st != SFFN_OK:
            raise SffnError(st, "sffn_route: " + self.lib.sffn_status_string(st).decode())

    def _logits(self, logits: torch.Tensor) -> Tuple[int, int, int]:
        if logits.dim() != 2 or not logits.is_cuda:
            raise ValueError("logits must be a [T, n_experts] tensor on the GPU")
        T = logits.shape[0]
        return (T, *_like(logits, T, self.n_experts, logits.device, "logits"))

    def _chosen(self, t: torch.Tensor, T: int, dtype: torch.dtype, device, what: str) -> int:
        if (t.shape != (T, self.top_k) or t.dtype != dtype or t.device != device
                or not t.is_contiguous()):
            raise ValueError(f"{what} must be a contiguous {dtype} tensor {(T, self.top_k)} on "
                             f"{device}, not {t.dtype} {tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def forward(self, logits: torch.Tensor, bias: Optional[torch.Tensor] = None,
                n_tokens: Optional[torch.Tensor] = None,
                out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None
                ) -> Tuple[torch.Tensor, torch.Tensor]:
        """(ids [T, k] int32, probs [T, k] float32) of ``logits`` [T, n_experts]
        (float32 or bfloat16, contiguous rows, any row stride), the chosen
        experts in descending order of score plus ``bias`` [n_experts] float32.
        ``SparseMoE.forward`` takes them as ``chosen``. ``n_tokens`` as there;
        ``out`` may pass (ids, probs) to reuse."""
        T, ld, dt = self._logits(logits)
        dev, k = logits.device, self.top_k
        pb = None if bias is None else _vector(bias, self.n_experts, dev, "bias", f32=True)[0]
        pn = _count(n_tokens, dev, "n_tokens")
        if out is None:
            ids = torch.empty_strided((T, k), (k, 1), dtype=torch.int32, device=dev)
            probs = torch.empty_strided((T, k), (k, 1), dtype=torch.float32, device=dev)
            pi, pp = ids.data_ptr(), probs.data_ptr()
        else:
            ids, probs = out
            pi = self._chosen(ids, T, torch.int32, dev, "ids")
            pp = self._chosen(probs, T, torch.float32, dev, "probs")
        _launch(dev, "sffn_route", self.lib.sffn_route, self._desc, logits.data_ptr(), dt, T, ld,
                pb, pn, pi, pp)
        return ids, probs

    def backward(self, dprobs: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor,
                 dtype: torch.dtype = torch.float32, n_tokens: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The gradient of the logits [T, n_experts], of ``dtype`` (or in
        ``out``, which may be ``logits``), from ``dprobs`` [T, k] float32, that of
        the weights.
        ``logits`` and ``ids`` are the forward call's. (The bias takes part in
        the choice alone and has no gradient.)"""
        T, ld, dt = self._logits(logits)
        dev = logits.device
        pd = self._chosen(dprobs, T, torch.float32, dev, "dprobs")
        pi = self._chosen(ids, T, torch.int32, dev, "ids")
        pn = _count(n_tokens, dev, "n_tokens")
        out, ldo, od = _result(out, T, self.n_experts, dtype, dev)
        _launch(dev, "sffn_route_backward", self.lib.sffn_route_backward, self._desc, pd,
                logits.data_ptr(), dt, T, ld, pi, pn, out.data_ptr(), od, ldo)
        return out
