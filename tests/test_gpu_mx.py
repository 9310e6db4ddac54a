"""MXFP4 on the GPU: quantisation and values bit for bit against the
oracle, the product against a float64 product of the same values.

The product's bound: products of two elements are exact, so only the sum
rounds. A float32 sum of K terms in any order errs by at most K half steps
of its running magnitude, which sum |a b| bounds; a truncating adder errs by
whole steps. So |got - ref| <= K 2^-23 sum |a b|, and a bfloat16 result by
half a step of itself (2^-8 relative) more."""
import numpy as np
import pytest
import torch

import unstructured_sparse_feedforward_amd as sffn
from oracle import mx_oracle as mo

pytestmark = pytest.mark.gpu


def _values(q):
    c, s = mo.unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.cols)
    return mo.values(c, s)


def _rand(shape, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp2(
        torch.randint(-12, 12, shape, generator=g).float())
    return x.to(dtype).cuda()


def _check_quantized(q, x):
    """q against the oracle of x (a CPU float64 array), codes, scales and padding."""
    codes, exps = mo.quantize(x)
    c, s = mo.pack(codes, exps)
    got_c, got_s = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    assert np.array_equal(got_c, c)
    assert np.array_equal(mo.unpack(got_c, got_s, q.cols)[1], exps)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 33), (16, 128), (17, 129), (5, 512),
                                       (33, 520), (2, 1003)])
def test_quantize(rows, cols, dtype):
    x = _rand((rows, cols), rows * 1000 + cols, dtype)
    q = sffn.mx_quantize(x)
    _check_quantized(q, x.double().cpu().numpy())
    v = sffn.mx_dequantize(q)
    assert np.array_equal(v.cpu().numpy().astype(np.float64), _values(q))
    assert torch.equal(sffn.mx_dequantize(q, dtype=torch.bfloat16).float(), v)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (32, 1), (33, 3), (128, 64), (129, 65), (257, 70),
                                       (500, 2)])
def test_quantize_transposed(rows, cols, dtype):
    x = _rand((rows, cols), rows * 1000 + cols, dtype)
    q = sffn.mx_quantize(x, transposed=True)
    assert (q.rows, q.cols) == (cols, rows)
    _check_quantized(q, x.double().cpu().numpy().T)
    # the same as the quantised copy
    r = sffn.mx_quantize(x.t().contiguous())
    assert torch.equal(q.codes, r.codes)
    assert np.array_equal(mo.unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy(), rows)[1],
                          mo.unpack(r.codes.cpu().numpy(), r.scales.cpu().numpy(), rows)[1])


@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_borders(transposed):
    """Ties and their neighbours, zeros of both signs, saturation,
    subnormals, the largest values, powers of two and their neighbours."""
    rows = []
    for s in (1.0, 2.0 ** -120, 2.0 ** 100):
        r = []
        for t in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            for v in (np.nextafter(np.float32(t), np.float32(0)), t,
                      np.nextafter(np.float32(t), np.float32(9))):
                r += [float(v) * s]
        r = (r + [0.0, -0.0, 6.0 * s, 7.9 * s, -7.0 * s, -2.5 * s] + [4.0 * s] * 32)[:32]
        r[31] = 4.0 * s
        rows.append(r)
    tiny = np.float32(2.0 ** -149)
    rows.append([float(tiny) * k for k in range(32)])
    rows.append([0.0] * 16 + [-0.0] * 16)
    rows.append([float(np.float32(3.4028235e38))] * 31 + [-1e38])
    rows.append([float(np.float32(2.0) ** (k - 20)) for k in range(32)])
    rows.append([float(np.nextafter(np.float32(2.0), np.float32(0)))] * 32)
    rows.append([2.0 ** -126, 2.0 ** -127, 2.0 ** -128, -2.0 ** -129] + [0.0] * 28)
    x = torch.tensor(np.array(rows, np.float32)).cuda()
    q = sffn.mx_quantize(x.t().contiguous(), transposed=True) if transposed else sffn.mx_quantize(x)
    _check_quantized(q, x.double().cpu().numpy())
    assert np.array_equal(sffn.mx_dequantize(q).cpu().numpy().astype(np.float64), _values(q))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_nonfinite_block(bad, transposed):
    x = _rand((5, 100), 3)
    x[2, 40] = bad
    q = sffn.mx_quantize(x.t().contiguous(), transposed=True) if transposed else sffn.mx_quantize(x)
    _check_quantized(q, x.double().cpu().numpy())
    for dt in (torch.float32, torch.bfloat16):
        v = sffn.mx_dequantize(q, dtype=dt)
        want = torch.zeros(5, 100, dtype=torch.bool, device="cuda")
        want[2, 32:64] = True
        assert torch.equal(torch.isnan(v), want)
    # in a product only the row with the block is lost
    out = sffn.mx_matmul(q, sffn.mx_quantize(_rand((7, 100), 4)))
    assert torch.isnan(out[2]).all() and torch.isfinite(out[[0, 1, 3, 4]]).all()
    out = sffn.mx_matmul(sffn.mx_quantize(_rand((70, 100), 4)), q)
    assert torch.isnan(out[:, 2]).all() and torch.isfinite(out[:, [0, 1, 3, 4]]).all()


def test_views_and_out():
    """Rows with any stride and any alignment, results into a view: what
    lies beside it is left as it was."""
    big = _rand((9, 300), 5)
    for view in (big[:, 1:], big[:, 4:100], big[::2, 3:40], big[2:3]):
        a, b = sffn.mx_quantize(view), sffn.mx_quantize(view.contiguous())
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
        a = sffn.mx_quantize(view, transposed=True)
        b = sffn.mx_quantize(view.t().contiguous())
        assert torch.equal(sffn.mx_dequantize(a), sffn.mx_dequantize(b))
    q = sffn.mx_quantize(big[:, :77])
    w = sffn.mx_quantize(_rand((40, 77), 6))
    for dt in (torch.float32, torch.bfloat16):
        for c0, cols, f in ((1, 77, lambda o: sffn.mx_dequantize(q, out=o)),
                            (8, 77, lambda o: sffn.mx_dequantize(q, out=o)),
                            (3, 40, lambda o: sffn.mx_matmul(q, w, out=o)),
                            (16, 40, lambda o: sffn.mx_matmul(q, w, out=o))):
            buf = torch.full((11, 120), 7.0, dtype=dt, device="cuda")
            o = buf[1:10, c0:c0 + cols]
            assert f(o) is o
            want = (sffn.mx_dequantize(q, dtype=dt) if cols == 77
                    else sffn.mx_matmul(q, w, dtype=dt))
            assert torch.equal(o, want)
            buf[1:10, c0:c0 + cols] = 7.0
            assert (buf == 7.0).all()
    again = sffn.mx_quantize(big[:, :77], out=q)
    assert again is q


def _assert_product(out, a, b):
    av, bv = _values(a), _values(b)
    ref, mag = av @ bv.T, np.abs(av) @ np.abs(bv).T
    tol = a.cols * 2.0 ** -23 * mag + 1e-300
    if out.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err - tol).max()


SIZES = [(1, 1, 1), (1, 16, 128), (1, 5632, 2048), (2, 17, 33), (16, 100, 1000), (17, 64, 256),
         (32, 33, 4096), (33, 48, 129), (64, 1003, 640), (65, 65, 65), (100, 200, 300),
         (128, 128, 128), (129, 257, 384), (333, 1003, 1999), (256, 256, 2048), (257, 511, 130),
         (1000, 1100, 512), (700, 2048, 1408),
         # few rows, K up to 4096 and above; long K
         (1, 300, 5000), (3, 40, 4096), (9, 64, 4097), (16, 1003, 16384), (64, 64, 16384),
         (40, 700, 8192), (2, 15, 4200)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul(M, N, K, dtype):
    a = sffn.mx_quantize(_rand((M, K), M + K))
    b = sffn.mx_quantize(_rand((N, K), N + K + 1))
    out = sffn.mx_matmul(a, b, dtype=dtype)
    _assert_product(out, a, b)
    assert torch.equal(out, sffn.mx_matmul(a, b, dtype=dtype))


@pytest.mark.parametrize("M,N,K", [
    # 128 x 256 tiles, whole and cut, K of one group, fewer and more than the ring
    (4096, 2048, 1024), (2048, 5632, 640), (2047, 2305, 128), (2500, 2000, 300), (4000, 3900, 513),
    # 256 x 256 tiles
    (4096, 4096, 2048), (3841, 3700, 1100), (8192, 5632, 1153), (40000, 300, 1280)])
def test_matmul_large(M, N, K):
    """Sizes of the large tiles; the float64 product on the GPU."""
    a = sffn.mx_quantize(_rand((M, K), 1))
    b = sffn.mx_quantize(_rand((N, K), 2))
    av, bv = sffn.mx_dequantize(a).double(), sffn.mx_dequantize(b).double()
    ref, mag = av @ bv.t(), av.abs() @ bv.abs().t()
    out = sffn.mx_matmul(a, b)
    assert ((out.double() - ref).abs() <= K * 2.0 ** -23 * mag).all()
    out16 = sffn.mx_matmul(a, b, dtype=torch.bfloat16)
    assert torch.equal(out16, out.to(torch.bfloat16))


def test_matmul_exact_integers():
    """Values whose sums float32 holds exactly come out exactly."""
    g = torch.Generator().manual_seed(0)
    for M, N, K in ((3, 50, 500), (90, 130, 700), (600, 700, 512)):
        grid = torch.tensor([0., 1., 2., 3., 4., 6.])
        av = grid[torch.randint(0, 6, (M, K), generator=g)] * (1 - 2 * torch.randint(0, 2, (M, K), generator=g))
        bv = grid[torch.randint(0, 6, (N, K), generator=g)]
        av[:, ::32] = 4.0
        bv[:, ::32] = 6.0
        a, b = sffn.mx_quantize(av.cuda()), sffn.mx_quantize(bv.cuda())
        assert torch.equal(sffn.mx_dequantize(a).cpu(), av)
        assert torch.equal(sffn.mx_matmul(a, b).cpu().double(), av.double() @ bv.double().t())


def test_matmul_empty():
    a = sffn.mx_quantize(torch.zeros(3, 0, device="cuda"))
    b = sffn.mx_quantize(torch.zeros(70, 0, device="cuda"))
    assert (sffn.mx_matmul(a, b) == 0).all() and sffn.mx_matmul(a, b).shape == (3, 70)
    assert (sffn.mx_matmul(b, b) == 0).all()
    e = sffn.mx_quantize(torch.zeros(0, 0, device="cuda"))
    assert sffn.mx_matmul(e, a).shape == (0, 3)
    assert sffn.mx_dequantize(b).shape == (70, 0)


def test_refusals_on_the_gpu():
    x = _rand((4, 64), 1)
    q = sffn.mx_quantize(x)
    for f in (lambda: sffn.mx_quantize(x.half()), lambda: sffn.mx_quantize(x.t()),
              lambda: sffn.mx_quantize(x[0]), lambda: sffn.mx_quantize(x[:, :1].expand(4, 64)),
              lambda: sffn.mx_quantize(x[:1].expand(4, 64)),
              lambda: sffn.mx_quantize(x, out=sffn.mx_quantize(x[:, :63])),
              lambda: sffn.mx_dequantize(q, dtype=torch.float16),
              lambda: sffn.mx_dequantize(q, out=torch.empty(4, 63, device="cuda")),
              lambda: sffn.mx_matmul(q, sffn.mx_quantize(x[:, :63])),
              lambda: sffn.mx_matmul(q, q, dtype=torch.int32),
              lambda: sffn.mx_matmul(q, q, out=torch.empty(4, 4)),
              lambda: sffn.mx_matmul(q, q, out=torch.empty(5, 4, device="cuda"))):
        with pytest.raises(ValueError):
            f()


def test_streams_and_graph():
    """On another stream than the default one, and captured: every replay
    with fresh inputs gives the eager result."""
    x, w = _rand((300, 512), 7), _rand((400, 512), 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        wq = sffn.mx_quantize(w)
        o1 = sffn.mx_matmul(sffn.mx_quantize(x), wq)
    torch.cuda.current_stream().wait_stream(side)
    xs = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og = sffn.mx_matmul(sffn.mx_quantize(xs), wq)
    for seed in range(4):
        xs.copy_(x if seed == 0 else _rand((300, 512), 20 + seed))
        eager = sffn.mx_matmul(sffn.mx_quantize(xs), wq)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(og, eager)
        if seed == 0:
            assert torch.equal(og, o1)


def test_gate_preactivations_into_twell():
    """A 4-bit gate product feeds the TwELL pack: the pack's actives are the
    product's positives."""
    import gpu_util as gu
    T, d, F = 70, 512, 1024
    x = torch.randn(T, d, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    w = torch.randn(F, d, device="cuda", generator=torch.Generator("cuda").manual_seed(2)) / d ** 0.5
    z = sffn.mx_matmul(sffn.mx_quantize(x), sffn.mx_quantize(w))
    ffn = sffn.SparseFFN(d, F, twell_cap=128)
    tw = gu.twell_np(ffn.pack_twell(z))
    zc = z.cpu().numpy()
    assert np.array_equal(tw["cnt"].sum(1), (zc > 0).sum(1))
    m = gu.valid_slots(tw)
    rows = np.nonzero(m)[0]
    assert np.array_equal(tw["val"][m], zc[rows, tw["idx"][m]])


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("R,K", [(3, 1), (17, 33), (5, 200), (40, 300), (70, 1185)])
def test_padding_is_written_as_zero(R, K, transposed):
    """Codes from K on and the scale bytes of blocks there, whatever the
    memory held."""
    out = sffn.mx_empty(R, K, "cuda")
    out.codes.fill_(0xFF)
    out.scales.fill_(0xFF)
    x = _rand((R, K), R + K)
    sffn.mx_quantize(x.t().contiguous() if transposed else x, transposed=transposed, out=out)
    c, s = mo.pack(*mo.quantize(x.double().cpu().numpy()))
    assert np.array_equal(out.codes.cpu().numpy(), c)
    assert np.array_equal(out.scales.cpu().numpy(), s)


@pytest.mark.parametrize("fill", [255, 254, 127])
@pytest.mark.parametrize("M,N,K", [
    # few rows, with K over four and eight waves; 32 x 64 and 64 x 64 tiles;
    # 128 x 256 and 256 x 256 tiles; one, two and three blocks of padding
    (1, 70, 1), (5, 40, 200), (16, 33, 4160), (100, 200, 300), (40, 70, 4129), (1000, 1100, 513),
    (2500, 2000, 300), (2047, 2305, 96), (3841, 3700, 1100), (4096, 4096, 2049)])
def test_scales_past_the_last_column_do_not_matter(M, N, K, fill):
    """Matrices whose scale bytes of the blocks past K are NaN's, the
    largest and 1, as memory that nobody cleared may hold: the same product
    and the same values."""
    def other(q):
        s = q.scales.clone()
        live = -(-K // 32) - (q.scales.shape[0] - 1) * 4
        assert live < 4
        s[-1, :, live:] = fill
        return sffn.MXTensor(q.codes.clone(), s, q.rows, q.cols)
    a, b = sffn.mx_quantize(_rand((M, K), 1)), sffn.mx_quantize(_rand((N, K), 2))
    want = sffn.mx_matmul(a, b)
    assert torch.isfinite(want).all()
    for p, q in ((other(a), b), (a, other(b)), (other(a), other(b))):
        assert torch.equal(sffn.mx_matmul(p, q), want)
    assert torch.equal(sffn.mx_dequantize(other(a)), sffn.mx_dequantize(a))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [
    # 8 to 16 rows of many columns: the borders at 8 rows, at K = 2048 and at
    # 224 and 448 tiles of 64 columns (7/8 of one and two rounds of the CUs), the
    # last one cut; 320 tiles do not fill theirs
    (7, 14336, 2048), (8, 14336, 2048), (8, 14336, 2047), (8, 14272, 2100), (13, 14300, 2081),
    (16, 16384, 4200), (17, 16384, 2048), (9, 16385, 2048), (12, 20480, 2176), (16, 28610, 2050)])
def test_matmul_few_rows_of_many_columns(M, N, K, dtype):
    a = sffn.mx_quantize(_rand((M, K), M + K))
    b = sffn.mx_quantize(_rand((N, K), N + K + 1))
    av, bv = sffn.mx_dequantize(a).double(), sffn.mx_dequantize(b).double()
    ref, mag = av @ bv.t(), av.abs() @ bv.abs().t()
    out = sffn.mx_matmul(a, b, dtype=dtype)
    tol = K * 2.0 ** -23 * mag
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    assert ((out.double() - ref).abs() <= tol).all()
    assert torch.equal(out, sffn.mx_matmul(a, b, dtype=dtype))


@pytest.mark.parametrize("made", [True, False])
@pytest.mark.parametrize("built", [True, False])
def test_matrices_of_inference_mode(made, built):
    """Codes and scales made in inference mode or outside, an MXTensor built
    of them in the mode or outside."""
    with torch.inference_mode(made):
        q = sffn.mx_quantize(_rand((6, 200), 1))
    with torch.inference_mode(built):
        r = sffn.MXTensor(q.codes, q.scales, 6, 200)
        out = sffn.mx_matmul(r, q)
    assert torch.equal(out, sffn.mx_matmul(q, q))
