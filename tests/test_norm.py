"""The residual norm without a GPU: pins of the oracle, refusals of the C
ABI."""
import ctypes

import numpy as np
import pytest
import torch

import unstructured_sparse_feedforward_amd as sffn
from oracle import mx8_oracle as m8
from oracle import norm_oracle as no
from unstructured_sparse_feedforward_amd import binding as B

P = 1 << 20          # stands for a device pointer: no valid call is made with it


def test_hand_worked():
    y, r = no.forward([[3.0, 4.0]], [2.0, 10.0], 0.0)
    assert np.allclose(r, [1 / np.sqrt(12.5)], rtol=1e-15)
    assert np.allclose(y, [[6 / np.sqrt(12.5), 40 / np.sqrt(12.5)]], rtol=1e-15)


def test_gradient_is_autograds():
    g = torch.Generator().manual_seed(0)
    s = torch.randn(7, 33, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(33, generator=g, dtype=torch.float64, requires_grad=True)
    dy, d = (torch.randn(7, 33, generator=g, dtype=torch.float64) for _ in range(2))
    y = s * torch.rsqrt(s.square().mean(1, keepdim=True) + 1e-6) * w
    ((y * dy).sum() + (s * d).sum()).backward()
    oy, r = no.forward(s.detach().numpy(), w.detach().numpy(), 1e-6)
    assert np.allclose(oy, y.detach().numpy(), rtol=1e-13)
    ds, dw = no.backward(dy.numpy(), s.detach().numpy(), w.detach().numpy(), r, d.numpy())
    assert np.allclose(ds, s.grad.numpy(), rtol=1e-11, atol=1e-13)
    assert np.allclose(dw, w.grad.numpy(), rtol=1e-11, atol=1e-13)


def test_e4m3_pins():
    assert m8.e4m3(0x7E) == 448 and m8.e4m3(0x38) == 1 and m8.e4m3(0xB8) == -1
    assert m8.e4m3(1) == 2.0 ** -9 and np.isnan(m8.e4m3(0x7F)) and np.isnan(m8.e4m3(0xFF))
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, m8.GRID)
    # (no tie: torch's conversion rounds to even as well)
    x = np.random.default_rng(0).uniform(0, 448, 500).astype(np.float32)
    c = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert [m8.nearest_code(float(v)) for v in x] == c.tolist()
    assert [m8.nearest_code(v) for v in (17.0, 19.0, 464.0, 500.0)] == [0x58, 0x5A, 0x7E, 0x7E]
    codes, e = m8.quantize([[256.0, -1.0] + [0.0] * 31 + [1.0]])
    assert e.tolist() == [[0, -8]] and codes[0, 0] == 0x78 and codes[0, 1] == 0xB8
    c, s = m8.pack(codes, e)
    assert c.shape == (1, 128) and s.tolist() == [[[127, 119, 0, 0]]]
    assert np.array_equal(m8.unpack(c, s, 34)[0], codes)
    assert np.isnan(m8.values(*m8.quantize([[np.inf]]))).all()


def _norm(kw, **base):
    a = dict(x=P, residual=P, residual_out=P, weight=P, out=P, out_scales=None, rstd=P, ldx=64,
             ldr=64, ldro=64, ldo=64, x_dtype=0, residual_dtype=1, weight_dtype=0, out_dtype=1)
    b = dict(rows=2, cols=64, eps=1e-6, n=None)
    for k, v in {**base, **kw}.items():
        (a if k in a else b)[k] = v
    return B.load_library().sffn_rms_norm(ctypes.byref(B.SffnNorm(**a)), b["rows"], b["cols"],
                                          b["eps"], b["n"], None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=P + 2), dict(x_dtype=3), dict(ldx=63), dict(residual=None),
    dict(residual_out=None), dict(residual=P + 1), dict(residual_out=P + 1), dict(ldr=63),
    dict(ldro=1), dict(residual_dtype=2), dict(weight=P + 2), dict(weight_dtype=9), dict(out=None),
    dict(out=P + 1), dict(ldo=63), dict(out_scales=P), dict(out_dtype=2), dict(rstd=P + 2),
    dict(rows=-1), dict(cols=-1), dict(eps=-1e-9), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(n=P + 2),
    dict(out_dtype=3), dict(out_dtype=3, out_scales=P + 1), dict(out_dtype=3, out_scales=P, out=P + 8)])
def test_refusals(kw):
    assert _norm(kw) == B.SFFN_E_ARG


def test_limits_and_empty():
    assert _norm(dict(cols=16385, ldx=20000, ldr=20000, ldro=20000, ldo=20000)) == B.SFFN_E_UNSUPPORTED
    assert _norm(dict(rows=(1 << 27) + 1)) == B.SFFN_E_UNSUPPORTED
    for cols, rows in ((64, 25), (512, 25), (513, 24), (2048, 23), (2049, 22), (4097, 21),
                       (16384, 21)):
        ld = dict(cols=cols, ldx=cols, ldr=cols, ldro=cols, ldo=cols)
        assert _norm(dict(rows=(1 << rows) + 1, **ld)) == B.SFFN_E_UNSUPPORTED
        assert _norm(dict(rows=1 << rows, x=None, **ld)) == B.SFFN_E_ARG
    assert _norm(dict(rows=0, x=None, out=None)) == B.SFFN_OK
    assert _norm(dict(cols=0, x=None, out=None)) == B.SFFN_OK
    lib = B.load_library()
    assert lib.sffn_rms_norm(None, 1, 1, 0.0, None, None) == B.SFFN_E_ARG
    assert lib.sffn_rms_norm_backward(None, 1, 1, None, 0, None) == B.SFFN_E_ARG
    n = ctypes.c_size_t()
    f = lib.sffn_rms_norm_backward_workspace_bytes
    assert f(-1, 1, ctypes.byref(n)) == f(1, -1, ctypes.byref(n)) == f(1, 1, None) == B.SFFN_E_ARG
    assert f(1, 16385, ctypes.byref(n)) == B.SFFN_E_UNSUPPORTED
    assert f(1 << 27, 16384, ctypes.byref(n)) == B.SFFN_OK and 0 < n.value < 1 << 28


@pytest.mark.parametrize("kw", [
    dict(dy=None), dict(dy=P + 2), dict(s=None), dict(s=P + 1), dict(rstd=None), dict(rstd=P + 2),
    dict(ds=None), dict(ds=P + 2), dict(dstream=P + 1), dict(weight=None), dict(weight=P + 2),
    dict(dweight=P + 2), dict(lddy=63), dict(lds=63), dict(lddstream=63), dict(ldds=63),
    dict(dy_dtype=2), dict(s_dtype=-1), dict(dstream_dtype=3), dict(weight_dtype=2),
    dict(ds_dtype=3), dict(rows=-1), dict(cols=-1), dict(rows=1 << 20, ws=None),
    dict(rows=1 << 20, ws=P + 16), dict(rows=1 << 20, ws_bytes=512 * 64 * 4 - 1),
    dict(rows=0, weight=None), dict(rows=0, weight=P + 2)])
def test_backward_refusals(kw):
    a = dict(dy=P, s=P, dstream=P, weight=P, rstd=P, ds=P, dweight=P, lddy=64, lds=64,
             lddstream=64, ldds=64, dy_dtype=0, s_dtype=1, dstream_dtype=1, weight_dtype=0,
             ds_dtype=0)
    b = dict(rows=1, cols=64, ws=P, ws_bytes=1 << 30)
    for k, v in kw.items():
        (a if k in a else b)[k] = v
    assert B.load_library().sffn_rms_norm_backward(
        ctypes.byref(B.SffnNormGrad(**a)), b["rows"], b["cols"], b["ws"], b["ws_bytes"],
        None) == B.SFFN_E_ARG


def test_mx8_refusals():
    lib = B.load_library()
    q = dict(x=P, dtype=0, rows=2, cols=64, ldx=64, codes=P, scales=P)
    for kw in (dict(x=None), dict(x=P + 2), dict(codes=P + 8), dict(scales=P + 2), dict(dtype=3),
               dict(rows=-1), dict(cols=-1), dict(ldx=63), dict(rows=(1 << 27) + 1)):
        assert lib.sffn_mx8_quantize(*{**q, **kw}.values(), None) == B.SFFN_E_ARG
    d = dict(codes=P, scales=P, rows=2, cols=64, out=P, dtype=0, ldo=64)
    for kw in (dict(codes=None), dict(scales=P + 1), dict(out=P + 2), dict(dtype=2), dict(ldo=63)):
        assert lib.sffn_mx8_dequantize(*{**d, **kw}.values(), None) == B.SFFN_E_ARG
    m = dict(a=P, asc=P, M=4, b=P, bsc=P, N=6, K=64, out=P, dtype=1, ldo=6)
    for kw in (dict(a=None), dict(a=P + 4), dict(asc=P + 1), dict(b=None), dict(b=P + 4),
               dict(bsc=None), dict(out=P + 1), dict(dtype=-1), dict(M=-1), dict(ldo=5),
               dict(M=(1 << 21) + 1), dict(K=(1 << 22) + 1)):
        assert lib.sffn_mx8_matmul(*{**m, **kw}.values(), None) == B.SFFN_E_ARG
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.sffn_mx8_bytes(3, 129, ctypes.byref(c), ctypes.byref(s)) == B.SFFN_OK
    assert (c.value, s.value) == (3 * 256, 3 * 8)
    assert lib.sffn_mx8_quantize(None, 0, 0, 64, 64, None, None, None) == B.SFFN_OK
    assert lib.sffn_mx8_matmul(None, None, 0, None, None, 5, 64, None, 0, 5, None) == B.SFFN_OK


def test_python_refusals():
    x = torch.zeros(4, 64)
    for f in (sffn.rms_norm, sffn.mx8_quantize,
              lambda t: sffn.rms_norm_backward(t, t, torch.zeros(4))):
        with pytest.raises(ValueError, match="GPU"):
            f(x)
    with pytest.raises(ValueError, match="GPU"):
        sffn.mx8_empty(4, 128, "cpu")
    codes, scales = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="do not hold"):
        sffn.MX8Tensor(codes[:, :64].contiguous(), scales, 4, 100)
    with pytest.raises(ValueError, match="GPU"):
        sffn.MX8Tensor(codes, scales, 4, 100)
