"""The expert layer on the CPU: its oracle against hand-worked and torch
results, and the refusals of the C entries and the Python class."""
import ctypes

import numpy as np
import pytest
import torch

import moe_pins as mp
import unstructured_sparse_feedforward_amd as sffn
from oracle import moe_oracle as mo
from unstructured_sparse_feedforward_amd import binding as B


def test_oracle_by_hand():
    # logits 0, ln 3, 0 over three experts: top 2 are expert 1, then expert
    # 0 (the tie with 2 goes to the lower); weights 3/4, 1/4, or 3/5, 1/5
    x = np.array([[1.0, 2.0]])
    wr = np.array([[0.0, 0.0], [np.log(3.0), 0.0], [2.0, -1.0]])
    wg = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[9.0, 9.0]]])        # z = 1, 2
    wu = np.array([[[3.0, 0.0]], [[0.0, 0.5]], [[9.0, 9.0]]])        # u = 3, 1
    wd = np.array([[[1.0, 0.0]], [[0.0, 4.0]], [[9.0, 9.0]]])        # h = 3, 2
    y, ids, p, bound = mo.forward(x, wr, wg, wu, wd, 2, True)
    assert ids.tolist() == [[1, 0]] and np.allclose(p, [[0.75, 0.25]])
    assert np.allclose(y, [[0.75, 6.0]]) and (bound > 0).all()
    y, _, p, _ = mo.forward(x, wr, wg, None, wd, 2, False)           # h = 1, 2
    assert np.allclose(p, [[0.6, 0.2]]) and np.allclose(y, [[0.2, 4.8]])
    y, *_ = mo.forward(x, wr, -wg, wu, wd, 2, True)                  # nothing active
    assert (y == 0).all()


@pytest.mark.parametrize("gated", [True, False])
def test_oracle_against_torch(gated):
    g = torch.Generator().manual_seed(0)
    T, d, F, E, k = 5, 24, 12, 6, 3
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, wr, wg, wu, wd = r(T, d), r(E, d), r(E, F, d), r(E, F, d), r(E, F, d)
    p, ids = torch.softmax(x @ wr.t(), 1).topk(k)
    h = torch.relu(torch.einsum("td,efd->tef", x, wg))
    if gated:
        h = h * torch.einsum("td,efd->tef", x, wu)
    ye = torch.einsum("tef,efd->ted", h, wd)
    full = torch.zeros(T, E, dtype=torch.float64).scatter_(1, ids, p)
    args = [v.numpy() for v in (x, wr, wg)] + [wu.numpy() if gated else None, wd.numpy()]
    y, oi, op, _ = mo.forward(*args, k, False)
    assert np.array_equal(oi, ids.numpy()) and np.allclose(op, p.numpy())
    assert np.allclose(y, torch.einsum("te,ted->td", full, ye).numpy())
    y, _, op, _ = mo.forward(*args, k, True)
    assert np.allclose(op.sum(1), 1.0)
    assert np.allclose(y, (torch.einsum("te,ted->td", full, ye) / p.sum(1, keepdim=True)).numpy())


BASE = dict(d=256, d_ff=96, n_experts=8, top_k=2, gated=1, normalize=1, weights=B.SFFN_BF16)
BAD = [(dict(d=0), B.SFFN_E_ARG), (dict(d_ff=0), B.SFFN_E_ARG), (dict(n_experts=0), B.SFFN_E_ARG),
       (dict(top_k=0), B.SFFN_E_ARG), (dict(top_k=9), B.SFFN_E_ARG), (dict(gated=2), B.SFFN_E_ARG),
       (dict(normalize=-1), B.SFFN_E_ARG), (dict(weights=B.SFFN_F32), B.SFFN_E_ARG),
       (dict(d=200), B.SFFN_E_UNSUPPORTED), (dict(d=8320), B.SFFN_E_UNSUPPORTED),
       (dict(d_ff=48), B.SFFN_E_UNSUPPORTED), (dict(d_ff=65568), B.SFFN_E_UNSUPPORTED),
       (dict(n_experts=1025), B.SFFN_E_UNSUPPORTED),
       (dict(n_experts=64, top_k=33), B.SFFN_E_UNSUPPORTED),
       (dict(n_experts=1024, d_ff=65536 * 2), B.SFFN_E_UNSUPPORTED)]
P = 1 << 20     # stands for a device pointer: no valid call is made with it


@pytest.mark.parametrize("kw,expect", BAD)
def test_descriptor(kw, expect):
    lib = B.load_library()
    D = B.SffnMoeDesc(**{**BASE, **kw})
    n = ctypes.c_size_t()
    assert lib.sffn_moe_workspace_bytes(ctypes.byref(D), 4, ctypes.byref(n)) == expect
    w = B.SffnMoeWeights(P, P, P, P, None, None, None)
    assert lib.sffn_moe_forward(ctypes.byref(D), P, ctypes.byref(w), 4, None, P, None, None, P,
                                1 << 40, None) == expect


def test_workspace_bytes():
    lib = B.load_library()
    D = B.SffnMoeDesc(**BASE)
    n = ctypes.c_size_t()
    ref = ctypes.byref
    assert lib.sffn_moe_workspace_bytes(ref(D), 0, ref(n)) == B.SFFN_OK and n.value == 0
    last = 0
    for T in (1, 2, 16, 256):
        assert lib.sffn_moe_workspace_bytes(ref(D), T, ref(n)) == B.SFFN_OK
        assert n.value > last and n.value % 256 == 0
        last = n.value
    assert lib.sffn_moe_workspace_bytes(ref(D), -1, ref(n)) == B.SFFN_E_ARG
    assert lib.sffn_moe_workspace_bytes(ref(D), 4, None) == B.SFFN_E_ARG
    assert lib.sffn_moe_workspace_bytes(None, 4, ref(n)) == B.SFFN_E_ARG
    assert lib.sffn_moe_workspace_bytes(ref(D), 257, ref(n)) == B.SFFN_E_UNSUPPORTED


@pytest.mark.parametrize("mx,gated,kw", [
    (0, 1, dict(x=None)), (0, 1, dict(x=P + 8)), (0, 1, dict(w=None)), (0, 1, dict(T=-1)),
    (0, 1, dict(y=None)), (0, 1, dict(y=P + 4)), (0, 1, dict(ws=None)), (0, 1, dict(ws=P + 16)),
    (0, 1, dict(ws_bytes=16)), (0, 1, dict(n=P + 1)), (0, 1, dict(ids=P + 2)),
    (0, 1, dict(probs=P + 2)), (0, 1, dict(router=None)), (0, 1, dict(gate=None)),
    (0, 1, dict(up=None)), (0, 0, dict(up=P)), (0, 1, dict(down=P + 2)), (0, 1, dict(gs=P)),
    (1, 1, dict(gs=None)), (1, 1, dict(us=None)), (1, 0, dict(up=None)), (1, 1, dict(ds=P + 2)),
    (1, 0, dict(up=None, us=P))])
def test_forward_refusals(mx, gated, kw):
    lib = B.load_library()
    D = B.SffnMoeDesc(**{**BASE, "gated": gated, "weights": B.SFFN_MXFP4 if mx else B.SFFN_BF16})
    s = P if mx else None
    a = dict(x=P, router=P, gate=P, up=P if gated else None, down=P, gs=s, us=s if gated else None,
             ds=s, T=4, n=None, y=P, ids=None, probs=None, ws=P, ws_bytes=1 << 40, w=1)
    if mx and not gated:
        a.update(gs=None)       # the fault; the parameters say which layer
    a.update(kw)
    w = B.SffnMoeWeights(a["router"], a["gate"], a["up"], a["down"], a["gs"], a["us"], a["ds"])
    assert lib.sffn_moe_forward(ctypes.byref(D), a["x"], ctypes.byref(w) if a["w"] else None,
                                a["T"], a["n"], a["y"], a["ids"], a["probs"], a["ws"],
                                a["ws_bytes"], None) == B.SFFN_E_ARG


def test_no_tokens_is_a_no_op():
    lib = B.load_library()
    D = B.SffnMoeDesc(**BASE)
    w = B.SffnMoeWeights()
    assert lib.sffn_moe_forward(ctypes.byref(D), None, ctypes.byref(w), 0, None, None, None, None,
                                None, 0, None) == B.SFFN_OK
    assert lib.sffn_moe_forward(ctypes.byref(D), P, ctypes.byref(w), 257, None, P, None, None,
                                P, 1 << 40, None) == B.SFFN_E_UNSUPPORTED


def test_python_refusals():
    with pytest.raises(ValueError, match="weights"):
        sffn.SparseMoE(256, 96, 8, 2, weights="int4")
    with pytest.raises(sffn.SffnError):
        sffn.SparseMoE(200, 96, 8, 2)
    with pytest.raises(sffn.SffnError):
        sffn.SparseMoE(256, 96, 2, 3)
    m = sffn.SparseMoE(256, 96, 8, 2)
    with pytest.raises(ValueError, match="GPU"):
        m.forward(torch.zeros(1, 256, dtype=torch.bfloat16), None, None, None, None)


@pytest.mark.parametrize("gated", [True, False])
def test_pins_tell_the_parts_of_h_apart(gated):
    """The exact inputs of the GPU tests: three bfloat16 parts of h give
    their y, two or one do not, for any neuron."""
    x, gate, up, down, y = mp.hidden_24_bits(7, 128, 96, gated)
    for w in (x, gate, down) + ((up,) if gated else ()):
        assert np.array_equal(mp.bf16(w), w)
    h = x @ gate.T if up is None else (x @ gate.T) * (x @ up.T)
    assert np.array_equal(h.astype(np.float32), h)      # 24 bits, no rounding
    oy, *_ = mo.forward(x, np.zeros((1, 128)), gate[None], None if up is None else up[None],
                        down[None], 1)
    assert np.array_equal(oy, y)
    rest, parts = h, []
    for _ in range(3):
        parts.append(mp.bf16(rest))
        rest = rest - parts[-1]
    assert (rest == 0).all()
    cols = (down != 0).any(0)
    for n in (1, 2):
        assert (sum(parts[:n]) @ down != y)[:, cols].all()
    assert np.array_equal(sum(parts) @ down, y)


@pytest.mark.parametrize("E", [2, 16, 64])
def test_near_tie_needs_64_bits(E):
    w, ids = mp.near_tie(E, 128)
    x = np.zeros((1, 128))
    x[0, [0, 127]] = 1.0
    assert np.array_equal(mp.bf16(w), w)
    assert mo.route(x, w, 2, True)[0].tolist() == [ids]
    low = (w.astype(np.float32) @ x[0].astype(np.float32)).astype(np.float64)
    assert sorted(range(E), key=lambda e: (-low[e], e))[:2] == ids[::-1]
