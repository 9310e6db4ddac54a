"""MXFP4 on the CPU: the oracle against hand-worked blocks, and the
refusals of the C entries and of the Python calls."""
import ctypes

import numpy as np
import pytest
import torch

import unstructured_sparse_feedforward_amd as sffn
from oracle import mx_oracle as mo
from unstructured_sparse_feedforward_amd import binding as B


# (value / scale, element): the ties go to the even code
@pytest.mark.parametrize("v,want", [
    (0.0, 0.0), (0.25, 0.0), (0.250001, 0.5), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0),
    (2.51, 3.0), (3.5, 4.0), (5.0, 4.0), (5.01, 6.0), (6.0, 6.0), (7.0, 6.0), (7.99, 6.0)])
def test_oracle_nearest(v, want):
    assert mo.GRID[mo.nearest_code(v)] == want


def test_oracle_block_by_hand():
    # largest magnitude 5: exponent 2, the scale 2^(2 - 2) = 1; the second
    # block holds 0.3 = 1.2 * 2^-2: scale 2^-4, 0.3 / 2^-4 = 4.8 -> 4
    x = np.zeros((1, 34))
    x[0, :4] = [5.0, -1.25, 0.3, -0.2]
    x[0, 33] = 0.3
    codes, exps = mo.quantize(x)
    assert exps.tolist() == [[0, -4]]
    assert mo.values(codes, exps)[0, [0, 1, 2, 3, 33]].tolist() == [4.0, -1.0, 0.5, 0.0, 0.25]
    assert codes[0, :4].tolist() == [6, 10, 1, 8]
    c, s = mo.pack(codes, exps)
    assert c.shape == (1, 64) and s.shape == (1, 1, 4)
    assert c[0, :2].tolist() == [6 | 10 << 4, 1 | 8 << 4]
    assert s[0, 0].tolist() == [127, 123, 0, 0]
    back = mo.unpack(c, s, 34)
    assert np.array_equal(back[0], codes) and np.array_equal(back[1], exps)


@pytest.mark.parametrize("block,e", [
    ([0.0, -0.0], -127), ([1.0], -2), ([1.9999999], -2), ([2.0], -1), ([2.0 ** -126], -127),
    ([1e-45], -127), ([3.4e38], 125), ([float("nan"), 1.0], None), ([float("inf")], None)])
def test_oracle_exponent(block, e):
    assert mo.block_exponent(block) == e


def test_bytes():
    lib = B.load_library()
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.sffn_mx_bytes(3, 130, ctypes.byref(c), ctypes.byref(s)) == B.SFFN_OK
    assert (c.value, s.value) == (3 * 128, 3 * 8)
    assert lib.sffn_mx_bytes(0, 5, ctypes.byref(c), ctypes.byref(s)) == B.SFFN_OK
    assert (c.value, s.value) == (0, 0)
    for r, k in ((-1, 5), (5, -1), (1 << 28, 5), (5, 1 << 23)):
        assert lib.sffn_mx_bytes(r, k, ctypes.byref(c), ctypes.byref(s)) == B.SFFN_E_ARG
    assert lib.sffn_mx_bytes(1, 1, None, ctypes.byref(s)) == B.SFFN_E_ARG
    assert lib.sffn_mx_bytes(1, 1, ctypes.byref(c), None) == B.SFFN_E_ARG


# host addresses stand for device pointers: no valid call is made with them
P = 1 << 20


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=P + 2), dict(codes=None), dict(codes=P + 8), dict(scales=None),
    dict(scales=P + 2), dict(dtype=7), dict(rows=-1), dict(cols=-1), dict(ldx=63),
    dict(transposed=2), dict(rows=(1 << 27) + 1), dict(cols=(1 << 22) + 1, ldx=1 << 23),
    dict(rows=(1 << 22) + 1, transposed=1)])
def test_quantize_refusals(kw):
    a = dict(x=P, dtype=B.SFFN_F32, rows=2, cols=64, ldx=64, transposed=0, codes=P, scales=P)
    a.update(kw)
    assert B.load_library().sffn_mx_quantize(*a.values(), None) == B.SFFN_E_ARG


@pytest.mark.parametrize("kw", [
    dict(codes=None), dict(codes=P + 8), dict(scales=None), dict(scales=P + 1), dict(out=None),
    dict(out=P + 2), dict(dtype=2), dict(rows=-1), dict(cols=-1), dict(ldo=63)])
def test_dequantize_refusals(kw):
    a = dict(codes=P, scales=P, rows=2, cols=64, out=P, dtype=B.SFFN_F32, ldo=64)
    a.update(kw)
    assert B.load_library().sffn_mx_dequantize(*a.values(), None) == B.SFFN_E_ARG


@pytest.mark.parametrize("kw", [
    dict(a=None), dict(a=P + 4), dict(asc=None), dict(asc=P + 1), dict(b=None), dict(b=P + 4),
    dict(bsc=None), dict(bsc=P + 1), dict(out=None), dict(out=P + 1), dict(dtype=-1), dict(M=-1),
    dict(N=-1), dict(K=-1), dict(ldo=5), dict(M=(1 << 21) + 1), dict(N=(1 << 21) + 1, ldo=1 << 22),
    dict(K=(1 << 22) + 1)])
def test_matmul_refusals(kw):
    a = dict(a=P, asc=P, M=4, b=P, bsc=P, N=6, K=64, out=P, dtype=B.SFFN_BF16, ldo=6)
    a.update(kw)
    assert B.load_library().sffn_mx_matmul(*a.values(), None) == B.SFFN_E_ARG


def test_empty_calls_touch_nothing():
    lib = B.load_library()
    assert lib.sffn_mx_quantize(None, 0, 0, 64, 64, 0, None, None, None) == B.SFFN_OK
    assert lib.sffn_mx_quantize(None, 0, 4, 0, 0, 1, None, None, None) == B.SFFN_OK
    assert lib.sffn_mx_dequantize(None, None, 0, 64, None, 0, 64, None) == B.SFFN_OK
    assert lib.sffn_mx_matmul(None, None, 0, None, None, 5, 64, None, 0, 5, None) == B.SFFN_OK
    assert lib.sffn_mx_matmul(None, None, 5, None, None, 0, 64, None, 0, 0, None) == B.SFFN_OK


def test_python_refusals():
    with pytest.raises(ValueError, match="GPU"):
        sffn.mx_quantize(torch.zeros(4, 64))
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8)
    for c, s, r, k, why in ((codes, scales, 4, 129, "do not hold"), (codes, scales, 5, 100, "do not hold"),
                            (codes, scales[0], 4, 100, "do not hold"),
                            (codes.int(), scales, 4, 100, "uint8"), (codes, scales, 4, 100, "GPU"),
                            (codes.expand(4, 64)[:, ::1].t().contiguous().t(), scales, 4, 100,
                             "contiguous")):
        with pytest.raises(ValueError, match=why):
            sffn.MXTensor(c, s, r, k)


def test_empty_on_the_cpu_is_refused():
    """Its pointers would reach a kernel through mx_dequantize."""
    with pytest.raises(ValueError, match="GPU"):
        sffn.mx_empty(4, 128, "cpu")
