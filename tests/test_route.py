"""The choice of experts without a GPU: pins of the oracle, refusals of the C
ABI."""
import ctypes

import numpy as np
import pytest
import torch

import unstructured_sparse_feedforward_amd as sffn
from oracle import route_oracle as ro
from unstructured_sparse_feedforward_amd import binding as B

P = 1 << 20          # stands for a device pointer: no valid call is made with it


def test_hand_worked():
    l = [[0.0, np.log(3.0), 0.0, np.log(4.0)]]           # softmax 1/9 3/9 1/9 4/9
    ids, p = ro.forward(l, 2)
    assert ids.tolist() == [[3, 1]] and np.allclose(p, [[4 / 7, 3 / 7]])
    ids, p = ro.forward(l, 3, normalize=False, scale=9.0)
    assert ids.tolist() == [[3, 1, 0]] and np.allclose(p, [[4, 3, 1]])
    # a bias chooses, the weights are without it
    ids, p = ro.forward(l, 2, bias=[1.0, 0.0, 0.0, 0.0], normalize=False)
    assert ids.tolist() == [[0, 3]] and np.allclose(p, [[1 / 9, 4 / 9]])
    # groups {0, 1} and {2, 3}: by the best one, 4/9; by the two best, 4/9 and 5/9
    l = [[np.log(2.0), np.log(2.0), 0.0, np.log(3.0)]]   # 2/8 2/8 1/8 3/8
    assert ro.forward(l, 2, groups=2, top_groups=1)[0].tolist() == [[3, 2]]
    assert ro.forward(l, 2, groups=2, top_groups=1, group_best=2)[0].tolist() == [[0, 1]]
    s = ro.forward([[0.0, -np.log(3.0)]], 2, sigmoid=True, normalize=False)[1]
    assert np.allclose(s, [[0.5, 0.25]])
    assert ro.forward([[-np.inf] * 3], 2)[1].tolist() == [[0.0, 0.0]]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
def test_gradient_is_autograds(sigmoid, normalize):
    g = torch.Generator().manual_seed(0)
    l = torch.randn(6, 20, generator=g, dtype=torch.float64, requires_grad=True)
    dp = torch.randn(6, 4, generator=g, dtype=torch.float64)
    ids = ro.forward(l.detach().numpy(), 4, sigmoid=sigmoid)[0]
    s = torch.sigmoid(l) if sigmoid else torch.softmax(l, 1)
    c = s.gather(1, torch.from_numpy(ids.astype(np.int64)))
    p = 1.5 * (c / c.sum(1, keepdim=True) if normalize else c)
    (p * dp).sum().backward()
    w = [ro.weights(a, i, sigmoid, normalize, 1.5) for a, i in zip(l.detach().numpy(), ids)]
    assert np.allclose(w, p.detach().numpy(), rtol=1e-13)
    d = ro.backward(dp.numpy(), l.detach().numpy(), ids, sigmoid, normalize, 1.5)
    assert np.allclose(d, l.grad.numpy(), rtol=1e-10, atol=1e-14)


BASE = dict(n_experts=64, top_k=6, groups=8, top_groups=4, group_best=2, sigmoid=1, normalize=1,
            scale=1.0)


@pytest.mark.parametrize("kw,expect", [
    (dict(n_experts=0), -1), (dict(top_k=0), -1), (dict(groups=0), -1), (dict(top_groups=0), -1),
    (dict(group_best=0), -1), (dict(group_best=3), -1), (dict(sigmoid=2), -1),
    (dict(normalize=-1), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(groups=7), -1), (dict(top_groups=9), -1), (dict(top_k=33), -1),
    (dict(groups=64, top_groups=5), -1), (dict(groups=64, group_best=1, top_k=5), -1),
    (dict(n_experts=1025, groups=1, top_groups=1), -2),
    (dict(top_k=33, groups=1, top_groups=1), -2),
    (dict(n_experts=256, groups=128, top_groups=64), -2),
    (dict(), 0), (dict(n_experts=1024, top_k=32, groups=64, top_groups=2), 0)])
def test_descriptor(kw, expect):
    D = B.SffnRouteDesc(**{**BASE, **kw})
    lib = B.load_library()
    assert lib.sffn_route(ctypes.byref(D), None, 0, 0, 0, None, None, None, None, None) == expect
    assert lib.sffn_route_backward(ctypes.byref(D), None, None, 0, 0, 0, None, None, None, 0, 0,
                                   None) == expect


def test_refusals():
    lib = B.load_library()
    D = B.SffnRouteDesc(**BASE)
    f = dict(logits=P, dtype=0, T=3, ldl=64, bias=P, n=P, ids=P, probs=P)
    for kw in (dict(logits=None), dict(logits=P + 2), dict(dtype=2), dict(T=-1), dict(ldl=63),
               dict(bias=P + 2), dict(n=P + 1), dict(ids=None), dict(ids=P + 2), dict(probs=None),
               dict(probs=P + 1)):
        assert lib.sffn_route(ctypes.byref(D), *{**f, **kw}.values(), None) == B.SFFN_E_ARG
    g = dict(dprobs=P, logits=P, dtype=1, T=3, ldl=64, ids=P, n=P, dl=P, dl_dtype=0, lddl=64)
    for kw in (dict(dprobs=None), dict(dprobs=P + 2), dict(logits=None), dict(logits=P + 1),
               dict(dtype=3), dict(T=-1), dict(ldl=63), dict(ids=None), dict(ids=P + 2),
               dict(n=P + 1), dict(dl=None), dict(dl=P + 2), dict(dl_dtype=2), dict(lddl=63)):
        assert lib.sffn_route_backward(ctypes.byref(D), *{**g, **kw}.values(), None) == B.SFFN_E_ARG
    assert lib.sffn_route(None, *f.values(), None) == B.SFFN_E_ARG
    for T, st in (((1 << 25) + 1, B.SFFN_E_UNSUPPORTED), (1 << 25, B.SFFN_E_ARG)):
        assert lib.sffn_route(ctypes.byref(D), *{**f, "T": T, "logits": None}.values(), None) == st
        assert lib.sffn_route_backward(ctypes.byref(D), *{**g, "T": T, "dl": None}.values(),
                                       None) == st


def test_python_refusals():
    with pytest.raises(ValueError, match="scores"):
        sffn.MoERouter(8, 2, scores="relu")
    for kw in (dict(top_k=9), dict(groups=3), dict(scale=float("nan")), dict(group_best=3)):
        with pytest.raises(sffn.SffnError):
            sffn.MoERouter(**{**dict(n_experts=8, top_k=2), **kw})
    with pytest.raises(ValueError, match="GPU"):
        sffn.MoERouter(8, 2).forward(torch.zeros(3, 8))
