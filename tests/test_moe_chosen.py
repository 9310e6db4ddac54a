"""Refusals of the expert layer's call with given experts (no GPU needed)."""
import ctypes

import pytest

from unstructured_sparse_feedforward_amd import binding as B

P = 1 << 20          # stands for a device pointer: no valid call is made with it
BASE = dict(d=256, d_ff=96, n_experts=8, top_k=2, gated=1, normalize=1, weights=B.SFFN_BF16)


def _call(kw, **desc):
    D = B.SffnMoeDesc(**{**BASE, **desc})
    a = dict(x=P, router=None, gate=P, up=P, down=P, T=4, n=None, ids=P, probs=P, y=P, ws=P,
             ws_bytes=1 << 40)
    a.update(kw)
    w = B.SffnMoeWeights(a["router"], a["gate"], a["up"], a["down"], None, None, None)
    return B.load_library().sffn_moe_forward_chosen(
        ctypes.byref(D), a["x"], ctypes.byref(w), a["T"], a["n"], a["ids"], a["probs"], a["y"],
        a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw", [
    dict(router=P), dict(ids=None), dict(ids=P + 2), dict(probs=None), dict(probs=P + 1),
    dict(x=None), dict(x=P + 8), dict(gate=None), dict(up=None), dict(down=P + 4), dict(T=-1),
    dict(n=P + 2), dict(y=None), dict(ws=None), dict(ws=P + 16), dict(ws_bytes=100)])
def test_refusals(kw):
    assert _call(kw) == B.SFFN_E_ARG


def test_limits():
    assert _call(dict(T=0, ids=None)) == B.SFFN_OK
    assert _call(dict(T=257)) == B.SFFN_E_UNSUPPORTED
    assert _call({}, top_k=9) == B.SFFN_E_ARG

