"""MXFP8 on the GPU: quantisation and values bit for bit against the oracle,
the product with MXFP4 weights against a float64 product of the same values.

The product's bound: products of two elements are exact, so only the sum
rounds. A float32 sum of K terms in any order errs by at most K half steps
of its running magnitude, which sum |a b| bounds; a truncating adder errs by
whole steps; the two parts of a make it two sums of K. So |got - ref| <= 2 K
2^-23 sum |a b|, and a bfloat16 result by half a step of itself (2^-8
relative) more. Sums that float32 holds exactly in any order are equal."""
import numpy as np
import pytest
import torch

import unstructured_sparse_feedforward_amd as sffn
from oracle import mx8_oracle as m8
from oracle import mx_oracle as m4

pytestmark = pytest.mark.gpu


def _values(q):
    o = m8 if isinstance(q, sffn.MX8Tensor) else m4
    return o.values(*o.unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.cols))


def _rand(shape, seed, dtype=torch.float32, spread=12):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp2(
        torch.randint(-spread, spread + 1, shape, generator=g).float())
    return x.to(dtype).cuda()


def _check_quantized(q, x):
    codes, exps = m8.quantize(x)
    c, s = m8.pack(codes, exps)
    assert np.array_equal(q.codes.cpu().numpy(), c)
    assert np.array_equal(m8.unpack(c, q.scales.cpu().numpy(), q.cols)[1], exps)
    live = -(-q.cols // 32) % 4
    if live:
        assert (q.scales[-1, :, live:] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 33), (16, 128), (17, 129), (5, 512),
                                       (33, 520), (2, 1003)])
def test_quantize(rows, cols, dtype):
    x = _rand((rows, cols), rows * 1000 + cols, dtype)
    q = sffn.mx8_quantize(x)
    _check_quantized(q, x.double().cpu().numpy())
    v = sffn.mx8_dequantize(q)
    assert np.array_equal(v.cpu().numpy().astype(np.float64), _values(q))
    assert torch.equal(sffn.mx8_dequantize(q, dtype=torch.bfloat16).float(), v)


def test_quantize_borders():
    """Ties of every pair of neighbouring values and what lies beside them,
    saturation, subnormals, zeros of both signs, the largest values."""
    rows = []
    mid = [(m8.e4m3(c) + m8.e4m3(c + 1)) / 2 for c in range(126)]
    for s in (1.0, 2.0 ** -100, 2.0 ** 100):
        for c in range(0, 126, 10):
            r = [256.0]
            for t in mid[c:c + 10]:
                r += [float(np.nextafter(np.float32(t), np.float32(0))), -t,
                      float(np.nextafter(np.float32(t), np.float32(999)))]
            rows.append([v * s for v in (r + [0.0] * 32)[:32]])
    rows.append([448.0, 449.0, 463.9, 464.0, 464.1, 480.0, 500.0, -511.9, -464.0, 0.0, -0.0] +
                [256.0] * 21)
    rows.append([float(np.float32(2.0 ** -149)) * k for k in range(32)])
    rows.append([0.0] * 16 + [-0.0] * 16)
    rows.append([float(np.float32(3.4028235e38))] * 31 + [-1e38])
    rows.append([float(np.float32(2.0) ** (k - 20)) for k in range(32)])
    rows.append([2.0 ** -126, 2.0 ** -127, 2.0 ** -128, -2.0 ** -129] + [0.0] * 28)
    x = torch.tensor(np.array(rows, np.float32)).cuda()
    q = sffn.mx8_quantize(x)
    _check_quantized(q, x.double().cpu().numpy())
    assert np.array_equal(sffn.mx8_dequantize(q).cpu().numpy().astype(np.float64), _values(q))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nonfinite_block(bad):
    x = _rand((5, 100), 3)
    x[2, 40] = bad
    q = sffn.mx8_quantize(x)
    _check_quantized(q, x.double().cpu().numpy())
    want = torch.zeros(5, 100, dtype=torch.bool, device="cuda")
    want[2, 32:64] = True
    for dt in (torch.float32, torch.bfloat16):
        assert torch.equal(torch.isnan(sffn.mx8_dequantize(q, dtype=dt)), want)
    out = sffn.mx_matmul(q, sffn.mx_quantize(_rand((7, 100), 4)))
    assert torch.isnan(out[2]).all() and torch.isfinite(out[[0, 1, 3, 4]]).all()
    w = _rand((7, 100), 5)
    w[3, 99] = bad
    out = sffn.mx_matmul(sffn.mx8_quantize(_rand((40, 100), 6)), sffn.mx_quantize(w))
    assert torch.isnan(out[:, 3]).all() and torch.isfinite(out[:, [0, 1, 2, 4, 5, 6]]).all()


SHAPES = [(1, 1, 1), (1, 5, 32), (1, 300, 2048), (3, 33, 129), (15, 64, 96), (16, 16, 128),
          (16, 1000, 4224), (17, 65, 257), (32, 64, 640), (33, 130, 1003), (64, 64, 64),
          (65, 257, 300), (100, 1000, 2000), (129, 513, 1999), (256, 256, 256), (300, 900, 1152),
          (512, 2048, 640), (1000, 2100, 512), (1024, 4096, 256), (2100, 4100, 131),
          (4096, 2304, 1280), (9, 14400, 4100), (16, 16384, 4200), (7, 14400, 4100),
          (2600, 4200, 1500), (4000, 3300, 1100), (5000, 5000, 1030)]


def _product(a, b):
    """Values and magnitudes of a b^T in float64, on the GPU."""
    va, vb = (torch.from_numpy(_values(q)).cuda() for q in (a, b))
    return va @ vb.t(), va.abs() @ vb.abs().t()


def _bound(mag, K, dtype, ref):
    t = 2 * K * 2.0 ** -23 * mag
    return t if dtype == torch.float32 else t + 2.0 ** -8 * (ref.abs() + t)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, dtype):
    a = sffn.mx8_quantize(_rand((M, K), M + N, spread=3))
    b = sffn.mx_quantize(_rand((N, K), M + N + 1, spread=2))
    out = sffn.mx_matmul(a, b, dtype=dtype)
    ref, mag = _product(a, b)
    assert out.shape == (M, N) and out.dtype == dtype
    assert ((out.double() - ref).abs() <= _bound(mag, K, dtype, ref)).all()
    assert torch.equal(out, sffn.mx_matmul(a, b, dtype=dtype))


def _wide(M, K, seed, every):
    """Codes of a whose products with +-0.5 or 1.5 and their sums are all
    multiples of 2^-10 below 2^13: exact in float32 in any order. In every
    (of long rows, every eighth) run of 8 one element is 256, the others are at
    most 2^-4 and go down to the smallest, 2^-9."""
    g = np.random.default_rng(seed)
    c = g.integers(0, 24, (M, K)).astype(np.uint8)       # 0 .. 15 / 8 2^-5
    big = g.integers(0, 8, (M, -(-K // 8)))
    sign = g.integers(0, 2, (M, K)).astype(np.uint8) << 7
    for i in range(0, big.shape[1], every):
        k = np.minimum(i * 8 + big[:, i], K - 1)
        c[np.arange(M), k] = (8 + 7) << 3
    return c | sign


@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (5, 100, 128), (16, 33, 250), (33, 64, 128),
                                   (100, 300, 96), (300, 1100, 128), (700, 2100, 160),
                                   (2304, 4352, 128), (4100, 4100, 100), (3, 200, 4200),
                                   (10, 16300, 4200), (4000, 3300, 1100)])
def test_wide_exponents_lose_nothing(M, N, K):
    """Large and small elements side by side: exact sums come out exactly."""
    c = _wide(M, K, M + N + K, 1 if K < 300 else 32 if K > 4000 else 8)
    q = m8.pack(c, np.zeros((M, -(-K // 32)), np.int64))
    a = sffn.MX8Tensor(torch.from_numpy(q[0]).cuda(), torch.from_numpy(q[1]).cuda(), M, K)
    g = np.random.default_rng(N)
    w = np.where(g.integers(0, 2, (N, K)) == 1, 0.5, 1.5) * g.choice([-1.0, 1.0], (N, K))
    # blocks of largest magnitude 1.5 (or 0.5) have the exponent -2 (-3)
    b = sffn.mx_quantize(torch.from_numpy(w).float().cuda())
    ref = torch.from_numpy(m8.values(c, np.zeros((M, -(-K // 32)), np.int64))).cuda() @ \
        torch.from_numpy(w).cuda().t()
    assert np.array_equal(_values(b), w)
    assert torch.equal(ref.float().double(), ref)        # the pin's own claim
    out = sffn.mx_matmul(a, b)
    assert torch.equal(out.double(), ref)


def test_every_code():
    """Every e4m3 value against every e2m1 value, and a NaN code."""
    c = np.zeros((256, 32), np.uint8)
    c[:, 7] = np.arange(256)
    q = m8.pack(c, np.zeros((256, 1), np.int64))
    a = sffn.MX8Tensor(torch.from_numpy(q[0]).cuda(), torch.from_numpy(q[1]).cuda(), 256, 32)
    w = np.zeros((16, 32), np.uint8)
    w[:, 7] = np.arange(16)
    p = m4.pack(w, np.zeros((16, 1), np.int64))
    b = sffn.MXTensor(torch.from_numpy(p[0]).cuda(), torch.from_numpy(p[1]).cuda(), 16, 32)
    ref = np.array([m8.e4m3(i) for i in range(256)])[:, None] * m4.values(
        np.arange(16, dtype=np.uint8)[:, None], np.zeros((16, 1), np.int64))[:, 0]
    got = sffn.mx_matmul(a, b).double().cpu().numpy()
    assert np.array_equal(got, ref, equal_nan=True)


def test_scales_of_every_block():
    """Each block of k has its own scale in either operand."""
    M, N, K = 70, 90, 640
    g = np.random.default_rng(1)
    ea, eb = g.integers(-20, 20, (M, 20)), g.integers(-20, 20, (N, 20))
    for k in range(0, K, 32):
        ca, cb = np.zeros((M, K), np.uint8), np.zeros((N, K), np.uint8)
        ca[:, k + k // 32 % 32] = 56          # 1
        cb[:, k + k // 32 % 32] = 2           # 1
        qa, qb = m8.pack(ca, ea), m4.pack(cb, eb)
        a = sffn.MX8Tensor(*(torch.from_numpy(v).cuda() for v in qa), M, K)
        b = sffn.MXTensor(*(torch.from_numpy(v).cuda() for v in qb), N, K)
        ref = 2.0 ** (ea[:, k // 32][:, None] + eb[:, k // 32][None])
        assert np.array_equal(sffn.mx_matmul(a, b).double().cpu().numpy(), ref), k


def test_zero_k_and_empty():
    a, b = sffn.mx8_empty(5, 0, "cuda"), sffn.mx_empty(9, 0, "cuda")
    assert torch.equal(sffn.mx_matmul(a, b), torch.zeros(5, 9, device="cuda"))
    big = sffn.mx_matmul(sffn.mx8_empty(3000, 0, "cuda"), sffn.mx_empty(3000, 0, "cuda"))
    assert (big == 0).all()
    assert sffn.mx_matmul(sffn.mx8_empty(0, 64, "cuda"), sffn.mx_empty(9, 64, "cuda")).shape == (0, 9)
    q = sffn.mx8_quantize(torch.empty(0, 50, device="cuda"))
    assert sffn.mx8_dequantize(q).shape == (0, 50)


def test_views_and_out():
    big = _rand((9, 300), 5)
    for view in (big[:, 1:], big[:, 4:100], big[::2, 3:40], big[2:3]):
        a, b = sffn.mx8_quantize(view), sffn.mx8_quantize(view.contiguous())
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    q = sffn.mx8_quantize(big[:, :77])
    w = sffn.mx_quantize(_rand((40, 77), 6))
    for dt in (torch.float32, torch.bfloat16):
        for c0, cols, f in ((1, 77, lambda o: sffn.mx8_dequantize(q, out=o)),
                            (3, 40, lambda o: sffn.mx_matmul(q, w, out=o)),
                            (16, 40, lambda o: sffn.mx_matmul(q, w, out=o))):
            buf = torch.full((11, 120), 7.0, dtype=dt, device="cuda")
            o = buf[1:10, c0:c0 + cols]
            assert f(o) is o
            want = (sffn.mx8_dequantize(q, dtype=dt) if cols == 77
                    else sffn.mx_matmul(q, w, dtype=dt))
            assert torch.equal(o, want)
            buf[1:10, c0:c0 + cols] = 7.0
            assert (buf == 7.0).all()
    assert sffn.mx8_quantize(big[:, :77], out=q) is q


def test_refusals():
    q8, q4 = sffn.mx8_empty(4, 64, "cuda"), sffn.mx_empty(4, 64, "cuda")
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError, match="b must be"):
        sffn.mx_matmul(q8, q8)
    with pytest.raises(ValueError, match="b must be"):
        sffn.mx_matmul(q4, q8)
    with pytest.raises(ValueError, match="columns"):
        sffn.mx_matmul(q8, sffn.mx_empty(4, 65, "cuda"))
    with pytest.raises(ValueError, match="MX8Tensor"):
        sffn.mx8_quantize(x, out=q4)
    with pytest.raises(ValueError, match="MXTensor"):
        sffn.mx_quantize(x, out=q8)
    with pytest.raises(ValueError, match="MX8Tensor"):
        sffn.mx8_dequantize(q4)
    with pytest.raises(ValueError, match="MXTensor"):
        sffn.mx_dequantize(q8)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        sffn.mx8_quantize(x.half())
    with pytest.raises(ValueError, match="dtype"):
        sffn.mx8_dequantize(q8, dtype=torch.float16)
    moe = sffn.SparseMoE(128, 32, 2, 1, weights="mxfp4")
    with pytest.raises(ValueError, match="MXTensor"):
        moe.forward(torch.zeros(1, 128, device="cuda", dtype=torch.bfloat16),
                    torch.zeros(2, 128, device="cuda", dtype=torch.bfloat16),
                    *[sffn.mx8_empty(64, 128, "cuda")] * 3)


def test_graph_and_streams():
    """Captured, replayed with new inputs between eager work; another stream
    than the default."""
    x = _rand((40, 500), 7, spread=2)
    w = sffn.mx_quantize(_rand((300, 500), 8, spread=2))
    want = [sffn.mx_matmul(sffn.mx8_quantize(x * s), w) for s in (1.0, 0.37, -5.0)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    buf = x.clone()
    with torch.cuda.stream(st):
        sffn.mx_matmul(sffn.mx8_quantize(buf), w)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            out = sffn.mx_matmul(sffn.mx8_quantize(buf), w)
    for s, ref in zip((1.0, 0.37, -5.0), want):
        buf.copy_(x * s)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        assert torch.equal(sffn.mx_matmul(sffn.mx8_quantize(buf), w), ref)


# one size for each kernel: few rows by 4 and by 8 waves, 32 x 64 and 64 x 64 tiles, 128 x 128,
# 128 x 256 and 256 x 256 ones
KERNELS = [(16, 500, 160), (16, 500, 4128), (256, 300, 160), (700, 2100, 160), (1000, 2100, 160),
           (2100, 4100, 160), (4096, 3328, 1056)]


def _device(mx, pack, codes, exps):
    return mx(*(torch.from_numpy(v).cuda() for v in pack(codes, exps)), *codes.shape)


@pytest.mark.parametrize("M,N,K", KERNELS)
def test_wide_exponents_in_every_kernel(M, N, K):
    """As test_wide_exponents_lose_nothing: multiples of 2^-10 below 2^13, of long
    rows with 256 in some runs of 8 only."""
    e = np.zeros((M, -(-K // 32)), np.int64)
    c = _wide(M, K, M + N + K, 1 if K < 300 else 32 if K > 4000 else 8)
    g = np.random.default_rng(N)
    w = np.where(g.integers(0, 2, (N, K)) == 1, 0.5, 1.5) * g.choice([-1.0, 1.0], (N, K))
    ref = torch.from_numpy(m8.values(c, e)).cuda() @ torch.from_numpy(w).cuda().t()
    assert torch.equal(ref.float().double(), ref)        # the pin's own claim
    out = sffn.mx_matmul(_device(sffn.MX8Tensor, m8.pack, c, e), sffn.mx_quantize(torch.from_numpy(w).float().cuda()))
    assert torch.equal(out.double(), ref)


@pytest.mark.parametrize("M,N,K", KERNELS)
def test_every_code_in_every_kernel(M, N, K):
    """Every e4m3 value against every e2m1 value, at several places of k; the NaN
    codes make their rows NaN."""
    va = np.array([m8.e4m3(i) for i in range(256)])
    vb = m4.values(np.arange(16, dtype=np.uint8)[:, None], np.zeros((16, 1), np.int64))[:, 0]
    for k in (0, 77, K - 1):
        for first in range(0, 256, min(M, 256)):
            ca, cb = np.zeros((M, K), np.uint8), np.zeros((N, K), np.uint8)
            ca[:, k], cb[:, k] = (first + np.arange(M)) % 256, np.arange(N) % 16
            out = sffn.mx_matmul(_device(sffn.MX8Tensor, m8.pack, ca, np.zeros((M, -(-K // 32)), np.int64)),
                                 _device(sffn.MXTensor, m4.pack, cb, np.zeros((N, -(-K // 32)), np.int64)))
            ref = torch.from_numpy(va[ca[:, k]][:, None] * vb[cb[:, k]][None]).cuda()
            assert torch.equal(torch.isnan(out), torch.isnan(ref))
            assert torch.equal(out.double().nan_to_num(), ref.nan_to_num())


@pytest.mark.parametrize("M,N,K", KERNELS)
def test_scales_in_every_kernel(M, N, K):
    """Each block of k has its own scale in either operand, in every row."""
    g = np.random.default_rng(1)
    n = -(-K // 32)
    ea, eb = g.integers(-20, 20, (M, n)), g.integers(-20, 20, (N, n))
    for b in sorted({0, 1, 2, 3, 4, n // 2, n - 2, n - 1}):
        ca, cb = np.zeros((M, K), np.uint8), np.zeros((N, K), np.uint8)
        ca[:, 32 * b + b % 32] = 56          # 1
        cb[:, 32 * b + b % 32] = 2           # 1
        out = sffn.mx_matmul(_device(sffn.MX8Tensor, m8.pack, ca, ea), _device(sffn.MXTensor, m4.pack, cb, eb))
        ref = torch.from_numpy(2.0 ** ea[:, b]).cuda()[:, None] * torch.from_numpy(2.0 ** eb[:, b]).cuda()[None]
        assert torch.equal(out.double(), ref), b
