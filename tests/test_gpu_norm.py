"""The residual norm and its gradient on the GPU against the float64 oracle.

Bounds, with u = 2^-24, half a step of float32. A row of n columns is summed
by lanes in turn, at most 16 terms a lane, then over at most 1024 lanes (64 of a
wave, then 16 waves): no term takes part in more than D = 16 + 6 + 16 = 38 additions,
taken as 46 here, the square or
product itself included. A sum of squares is thus off by at most (D + 1) u of
itself; its mean, eps, root, reciprocal and the products with s and w add
some 6 roundings: y is off by at most (D / 2 + 7) u of itself, taken here as
32 u. A result in bfloat16 is off by 2^-8 of itself more (half a step).

ds = r (g - xh c): with E = 50 the mean c is off by E u mean |g xh|, xh and g by
2 u of themselves; every further operation by half a step of its result. So
  |err| <= u (r (6 |g| + 6 |xh c| + E |xh| mean |g xh|) + 2 |ds|).
dw sums rows of dy xh, by columns: up to 512, ceil(T / (4 x 768)) rows a lane, then 3
additions over a workgroup's waves, 48 of workgroups and 15 of their sums; up to
2048, ceil(T / 512) rows (or a quarter), 3 + 32 + 15; above, ceil(T / 256) and 16 +
15; in one launch (T <= 2048) fewer. With fewer rows there are fewer workgroups, each
of one turn. xh and the product add 3 roundings, so
|err| <= (ceil(T / 256) + 69) u sum |dy xh|."""
import numpy as np
import pytest
import torch

import unstructured_sparse_feedforward_amd as sffn
from oracle import mx8_oracle as m8
from oracle import norm_oracle as no

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
COLS = [1, 2, 7, 8, 31, 32, 33, 127, 128, 129, 511, 512, 513, 1003, 1024, 1025, 2047, 2048, 2049,
        4095, 4096, 4097, 8192, 8200, 16383, 16384]


def _rand(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _check_y(y, ref, dtype):
    err = np.abs(_np(y) - ref)
    tol = 32 * U * np.abs(ref)
    if dtype == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 5])
def test_plain(rows, cols):
    x, w = _rand((rows, cols), cols), _rand((cols,), cols + 1)
    for dt in (F32, BF16):
        ref, r = no.forward(_np(x), _np(w), 1e-6)
        rstd = torch.empty(rows, device="cuda")
        _check_y(sffn.rms_norm(x, w, dtype=dt, rstd=rstd), ref, dt)
        assert (np.abs(_np(rstd) - r) <= 32 * U * r).all()
    _check_y(sffn.rms_norm(x, dtype=F32), no.forward(_np(x), None, 1e-6)[0], F32)


@pytest.mark.parametrize("cols", [1, 33, 1003, 2048, 5000, 9000])
@pytest.mark.parametrize("xd", [F32, BF16])
@pytest.mark.parametrize("rd", [F32, BF16])
@pytest.mark.parametrize("wd", [F32, BF16])
def test_residual(cols, xd, rd, wd):
    rows = 6
    x, res = _rand((rows, cols), 1, xd), _rand((rows, cols), 2, rd, 3.0)
    w = _rand((cols,), 3, wd)
    s = (x.float() + res.float()).to(rd)       # one rounding, and that to rd
    ref, r = no.forward(_np(s), _np(w), 1e-5)
    for dt in (F32, BF16):
        y, got = sffn.rms_norm(x, w, residual=res, eps=1e-5, dtype=dt)
        assert torch.equal(got, s)
        _check_y(y, ref, dt)
    # in place, and into given results
    keep = res.clone()
    out = torch.empty(rows, cols, device="cuda", dtype=BF16)
    y2, same = sffn.rms_norm(x, w, residual=keep, eps=1e-5, out=out, residual_out=keep)
    assert same is keep and y2 is out and torch.equal(keep, s) and torch.equal(out, y)


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (5, 32), (2, 100), (7, 129), (777, 1003),
                                       (4, 2000), (5, 2048), (3, 4100), (2, 8191), (2, 16384)])
def test_mxfp8(rows, cols):
    """The codes are those of the float32 result, bit for bit."""
    x, res, w = _rand((rows, cols), 5), _rand((rows, cols), 6), _rand((cols,), 7)
    x[0, cols // 2] *= 300
    y, s = sffn.rms_norm(x, w, residual=res, dtype=F32)
    q, s2 = sffn.rms_norm(x, w, residual=res, dtype="mxfp8")
    assert isinstance(q, sffn.MX8Tensor) and torch.equal(s, s2)
    ref = sffn.mx8_quantize(y)
    assert torch.equal(q.codes, ref.codes) and torch.equal(q.scales, ref.scales)
    if rows * cols < 10000:
        assert np.array_equal(q.codes.cpu().numpy()[:, :cols], m8.quantize(_np(y))[0])
    again, _ = sffn.rms_norm(x, w, residual=res, out=q)
    assert again is q


def test_rows_do_not_depend_on_each_other():
    x, w = _rand((300, 2048), 8), _rand((2048,), 9)
    y = sffn.rms_norm(x, w, dtype=F32)
    for i in (0, 1, 3, 255, 299):
        assert torch.equal(sffn.rms_norm(x[i:i + 1], w, dtype=F32), y[i:i + 1])


def test_views():
    """Any row stride, any alignment; what lies beside a result is left."""
    big = _rand((9, 3000), 10)
    bb = big.bfloat16()
    for c0, c1 in ((1, 2048), (3, 900), (5, 2998), (0, 64), (7, 8)):
        n = c1 - c0
        w = _rand((n + 1,), 11)[1:]
        x, res = bb[::2, c0:c1], big[:5, c0:c1]
        y, s = sffn.rms_norm(x.contiguous(), w, residual=res.contiguous(), dtype=BF16)
        so, yo = torch.full((5, 3001), 7.0, device="cuda"), torch.full((5, 3003), 7.0,
                                                                      device="cuda", dtype=BF16)
        a, b = sffn.rms_norm(x, w, residual=res, out=yo[:, 3:3 + n], residual_out=so[:, 1:1 + n])
        assert torch.equal(a, y) and torch.equal(b, s)
        yo[:, 3:3 + n] = 7
        so[:, 1:1 + n] = 7
        assert (yo == 7).all() and (so == 7).all()
        # the stream in place beside a column that is not part of it
        h = big.clone()
        sffn.rms_norm(x, w, residual=h[:5, c0:c1], residual_out=h[:5, c0:c1])
        assert torch.equal(h[:5, c0:c1], s)
        h[:5, c0:c1] = big[:5, c0:c1]
        assert torch.equal(h, big)


def test_special_values():
    x = torch.zeros(6, 100, device="cuda")
    x[1] = 1e-30
    x[2, 5] = float("nan")
    x[3, 6] = float("inf")
    x[4] = 1e18          # squares whose sum is near float32's largest
    x[5] = 1.0
    y = sffn.rms_norm(x, dtype=F32)
    assert (y[0] == 0).all() and torch.isnan(y[2]).all()
    assert torch.isnan(y[3, 6]) and (y[3, :6] == 0).all()
    _check_y(y[[1, 4, 5]], no.forward(_np(x[[1, 4, 5]]), None, 1e-6)[0], F32)
    # eps 0: a row of zeros has no norm, in 8 bits too, and no other row is touched
    y = sffn.rms_norm(x, eps=0.0, dtype=F32)
    assert torch.isnan(y[0]).all() and torch.isfinite(y[5]).all()
    q = sffn.rms_norm(x, eps=0.0, dtype="mxfp8")
    v = sffn.mx8_dequantize(q)
    assert torch.isnan(v[0]).all() and torch.equal(v[5], y[5]) and (q.scales[0, 5] == 119).all()


def test_n_rows():
    x, res, w = _rand((50, 700), 12), _rand((50, 700), 13), _rand((700,), 14)
    y, s = sffn.rms_norm(x, w, residual=res)
    q, _ = sffn.rms_norm(x, w, residual=res, dtype="mxfp8")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    for v, m in ((0, 0), (1, 1), (7, 7), (50, 50), (99, 50), (-3, 0)):
        n.fill_(v)
        yo = torch.full_like(y, 7)
        h = res.clone()
        rs = torch.full((50,), 7.0, device="cuda")
        sffn.rms_norm(x, w, residual=h, residual_out=h, out=yo, rstd=rs, n_rows=n)
        assert torch.equal(yo[:m], y[:m]) and (yo[m:] == 7).all() and (rs[m:] == 7).all()
        assert torch.equal(h[:m], s[:m]) and torch.equal(h[m:], res[m:])
        o = sffn.mx8_empty(50, 700, "cuda")
        o.codes.fill_(99)
        o.scales.fill_(98)
        sffn.rms_norm(x, w, residual=res, out=o, n_rows=n)
        assert torch.equal(o.codes[:m], q.codes[:m]) and (o.codes[m:] == 99).all()
        assert torch.equal(o.scales[:, :m], q.scales[:, :m]) and (o.scales[:, m:] == 98).all()


def _grads(rows, cols, dd, sd, wd=F32, di=None, seed=0):
    dy, s = _rand((rows, cols), seed + 1, dd), _rand((rows, cols), seed + 2, sd, 2.0)
    w = None if wd is None else _rand((cols,), seed + 3, wd)
    d = None if di is None else _rand((rows, cols), seed + 4, di)
    r = torch.from_numpy(no.forward(_np(s), None, 1e-6)[1]).float().cuda()
    return dy, s, r, w, d


def _check_grads(ds, dw, dy, s, r, w, d):
    n = lambda t: None if t is None else _np(t)     # noqa: E731
    ref, rdw = no.backward(n(dy), n(s), n(w), n(r), n(d))
    xh, g = n(s) * n(r)[:, None], n(dy) if w is None else n(dy) * n(w)
    m, c = np.abs(g * xh).mean(axis=1, keepdims=True), (g * xh).mean(axis=1, keepdims=True)
    tol = U * (n(r)[:, None] * (6 * np.abs(g) + 6 * np.abs(xh * c) + 50 * np.abs(xh) * m)
               + 2 * np.abs(ref))
    if ds.dtype == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert (np.abs(n(ds) - ref) <= tol).all()
    if w is None:
        assert dw is None
        return
    assert dw.dtype == F32 and dw.shape == (s.shape[1],)
    tol = (-(-s.shape[0] // 256) + 69) * U * np.abs(n(dy) * xh).sum(axis=0)
    assert (np.abs(n(dw) - rdw) <= tol).all()


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 6])
def test_gradient(rows, cols):
    a = _grads(rows, cols, F32, F32, di=F32)
    dy, s, r, w, d = a
    _check_grads(*sffn.rms_norm_backward(dy, s, r, w, dstream=d), *a)


@pytest.mark.parametrize("rows,cols", [(2, 1), (3, 7), (9, 100), (777, 1003), (2047, 8), (2048, 33),
                                       (2048, 1024), (257, 8191), (2500, 300), (2100, 2048),
                                       (1030, 4096), (600, 6000), (520, 10000)])
@pytest.mark.parametrize("dd,sd,wd,di,od", [(BF16, BF16, F32, None, BF16),
                                            (BF16, F32, BF16, BF16, F32),
                                            (F32, BF16, None, F32, F32),
                                            (F32, F32, F32, F32, BF16)])
def test_gradient_types(rows, cols, dd, sd, wd, di, od):
    a = _grads(rows, cols, dd, sd, wd, di)
    dy, s, r, w, d = a
    got = sffn.rms_norm_backward(dy, s, r, w, dstream=d, dtype=od)
    assert got[0].dtype == od
    _check_grads(*got, *a)
    again = sffn.rms_norm_backward(dy, s, r, w, dstream=d, dtype=od)
    assert torch.equal(got[0], again[0]) and (w is None or torch.equal(got[1], again[1]))


def test_gradient_against_differences():
    """The loss sum(dy y) along random directions of s and w: the central
    difference of the float64 oracle at a step of 1e-5 is off by its third
    derivative's 1e-10 and by 2^-52 / 1e-5 of the loss, below 1e-7 of the norms'
    product together; the gradient's own bound is 1e-5 of it."""
    rows, cols, h = 40, 600, 1e-5
    dy, s, r, w, _ = _grads(rows, cols, F32, F32)
    ds, dw = sffn.rms_norm_backward(dy, s, r, w)
    g = np.random.default_rng(0)
    loss = lambda a, b: (_np(dy) * no.forward(a, b, 1e-6)[0]).sum()     # noqa: E731
    for _ in range(5):
        e, f = g.standard_normal((rows, cols)), g.standard_normal(cols)
        num = (loss(_np(s) + h * e, _np(w) + h * f) - loss(_np(s) - h * e, _np(w) - h * f)) / (2 * h)
        ana = (_np(ds) * e).sum() + (_np(dw) * f).sum()
        size = np.linalg.norm(_np(ds)) * np.linalg.norm(e) + np.linalg.norm(_np(dw)) * np.linalg.norm(f)
        assert abs(num - ana) <= 2e-5 * size


def test_gradient_places():
    """In place of each operand, views, given results, no rows."""
    dy, s, r, w, d = _grads(30, 500, F32, F32, di=F32)
    ref, rdw = sffn.rms_norm_backward(dy, s, r, w, dstream=d)
    for i in range(3):
        t = [dy.clone(), s.clone(), d.clone()]
        dw = torch.empty(500, device="cuda")
        got = sffn.rms_norm_backward(t[0], t[1], r, w, dstream=t[2], out=t[i], dweight=dw)
        assert got[0] is t[i] and got[1] is dw
        assert torch.equal(t[i], ref) and torch.equal(dw, rdw)
    wide = [torch.full((30, 600), 7.0, device="cuda") for _ in range(4)]
    v = [t[:, 3:503] for t in wide]
    for a, b in zip(v, (dy, s, d)):
        a.copy_(b)
    sffn.rms_norm_backward(v[0], v[1], r, w, dstream=v[2], out=v[3])
    assert torch.equal(v[3], ref)
    v[3].fill_(7)
    assert (wide[3] == 7).all()
    e = torch.empty(0, 500, device="cuda")
    ds, dw = sffn.rms_norm_backward(e, e, torch.empty(0, device="cuda"), w)
    assert ds.shape == (0, 500) and (dw == 0).all()


@pytest.mark.parametrize("rows,cols", [(1, 8), (2, 64), (777, 1003), (1024, 2048), (2048, 1024),
                                       (2048, 512), (512, 4096), (256, 8192), (2048, 2048),
                                       (2000, 7)])
@pytest.mark.parametrize("dd,sd,od", [(F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, F32)])
def test_gradient_in_place(rows, cols, dd, sd, od):
    """ds in the place of dy or of s: dw, which reads every row of both, is the same."""
    dy, s, r, w, d = _grads(rows, cols, dd, sd, di=F32)
    ref, rdw = sffn.rms_norm_backward(dy, s, r, w, dstream=d, dtype=od)
    for i in range(2):
        if (dd, sd)[i] != od:
            continue
        for _ in range(3):
            t = [dy.clone(), s.clone()]
            got, dw = sffn.rms_norm_backward(t[0], t[1], r, w, dstream=d, out=t[i])
            assert got is t[i] and torch.equal(got, ref) and torch.equal(dw, rdw)
    # halves of the same rows: nothing in common but the span
    wide = torch.empty(rows, 2 * cols, dtype=sd, device="cuda")
    wide[:, :cols] = s
    if sd == od:
        got, dw = sffn.rms_norm_backward(dy, wide[:, :cols], r, w, dstream=d, out=wide[:, cols:])
        assert torch.equal(got, ref) and torch.equal(dw, rdw) and torch.equal(wide[:, :cols], s)


def test_empty():
    e = torch.empty(0, 500, device="cuda")
    y, s = sffn.rms_norm(e, residual=e, dtype=F32)
    assert y.shape == s.shape == (0, 500)
    assert sffn.rms_norm(torch.empty(4, 0, device="cuda")).shape == (4, 0)


def test_refusals():
    x, w = torch.zeros(4, 64, device="cuda"), torch.zeros(64, device="cuda")
    for kw, why in ((dict(residual=x[:3]), "residual must be"),
                    (dict(residual=x.half()), "residual must be float32 or bfloat16"),
                    (dict(residual_out=x), "without a residual"),
                    (dict(residual=x, residual_out=x.bfloat16()), "residual's type"),
                    (dict(weight=w[:63]), "weight must be"), (dict(weight=w.half()), "weight must"),
                    (dict(weight=torch.zeros(128, device="cuda")[::2]), "contiguous"),
                    (dict(weight=w.cpu()), "weight must"),
                    (dict(dtype=torch.float16), "dtype"), (dict(dtype="fp8"), "dtype"),
                    (dict(out=x.t()), "contiguous rows"), (dict(out=x[:2]), "out must"),
                    (dict(out=sffn.mx8_empty(4, 65, "cuda")), "out must"),
                    (dict(rstd=w), "rstd"), (dict(rstd=torch.zeros(4)), "rstd"),
                    (dict(n_rows=torch.zeros(1, device="cuda")), "n_rows")):
        with pytest.raises(ValueError, match=why):
            sffn.rms_norm(x, **kw)
    with pytest.raises(sffn.SffnError):
        sffn.rms_norm(x, eps=-1.0)
    with pytest.raises(sffn.SffnError):
        sffn.rms_norm(x, eps=float("nan"))
    with pytest.raises(sffn.SffnError):
        sffn.rms_norm(torch.zeros(1, 16385, device="cuda"))
    r = torch.zeros(4, device="cuda")
    for a, kw, why in (((x, x[:3], r), {}, "s must"), ((x, x, r[:3]), {}, "rstd"),
                       ((x, x, r), dict(dweight=w), "without a weight"),
                       ((x, x, r, w[:5]), {}, "weight must"),
                       ((x, x, r), dict(dstream=x[:1]), "dstream"),
                       ((x, x, r), dict(dtype=torch.float16), "dtype")):
        with pytest.raises(ValueError, match=why):
            sffn.rms_norm_backward(*a, **kw)
    big = torch.zeros(1, 16385, device="cuda")
    with pytest.raises(sffn.SffnError):
        sffn.rms_norm_backward(big, big, r[:1])


def test_aliases():
    """A result in x's place, the sum in x's place."""
    x, res, w = _rand((40, 300), 1), _rand((40, 300), 2), _rand((300,), 3)
    y, s = sffn.rms_norm(x, w, residual=res, dtype=F32)
    a = x.clone()
    assert sffn.rms_norm(a, w, residual=res, out=a)[0] is a and torch.equal(a, y)
    a = x.clone()
    got = sffn.rms_norm(a, w, residual=res, dtype=F32, residual_out=a)
    assert got[1] is a and torch.equal(a, s) and torch.equal(got[0], y)


def test_most_rows():
    """2^25 rows of up to 512 columns, the most of a call."""
    x = torch.ones(1 << 25, 8, dtype=BF16, device="cuda")
    y = torch.full_like(x, 7)
    sffn.rms_norm(x, eps=0.0, out=y)
    assert (y == 1).all()


def test_two_streams():
    """Calls that overlap on two streams: nothing is shared."""
    args = [_grads(n, c, BF16, F32, di=F32, seed=n) for n, c in ((3000, 1500), (300, 900))]
    want = []
    for dy, s, r, w, d in args:
        want.append((*sffn.rms_norm(dy, w, residual=s), *sffn.rms_norm_backward(dy, s, r, w, dstream=d)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = [[], []]
    for _ in range(10):
        for k, (st, (dy, s, r, w, d)) in enumerate(zip(streams, args)):
            with torch.cuda.stream(st):
                got[k].append((*sffn.rms_norm(dy, w, residual=s),
                               *sffn.rms_norm_backward(dy, s, r, w, dstream=d)))
    torch.cuda.synchronize()
    for g, ref in zip(got, want):
        for one in g:
            assert all(torch.equal(a, b) for a, b in zip(one, ref))


def test_graphs_share_nothing():
    """Two captured passes, forward and backward, replayed in turn with eager
    work between them; a stream of its own."""
    dy, s, r, w, d = _grads(600, 900, BF16, F32, di=F32)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ins, outs, graphs = [], [], []
    with torch.cuda.stream(st):
        for k in range(2):
            x, h = dy.clone(), s.clone()
            rs = torch.empty(600, device="cuda")
            run = lambda: (lambda y: (*y, *sffn.rms_norm_backward(     # noqa: E731
                dy, y[1], rs, w, dstream=d)))(sffn.rms_norm(x, w, residual=h, rstd=rs))
            run()
            st.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                outs.append(run())
            ins.append((x, h, rs))
            graphs.append(g)
    for f in (1.0, -0.5, 2.5):
        for k in (0, 1):
            ins[k][0].copy_(dy * (f + k))
            ins[k][1].copy_(s * (f - k))
        torch.cuda.synchronize()
        for k in (1, 0):
            graphs[k].replay()
        torch.cuda.synchronize()
        for k in (0, 1):
            rs = torch.empty(600, device="cuda")
            y = sffn.rms_norm(ins[k][0], w, residual=ins[k][1], rstd=rs)
            want = (*y, *sffn.rms_norm_backward(dy, y[1], rs, w, dstream=d))
            for a, b in zip(outs[k], want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [1, 8, 500, 1000, 2000, 4000, 8000, 16000])
@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-33, 1e-6, 1e30])
def test_squares_beyond_float32(cols, eps):
    """Rows whose squares float32 cannot hold, of any result type; ordinary rows
    between them as without them. Bounds as above, and r, which may be below
    float32's normals but not below 2^-128, is off by 2^-150 at most, 4 u of itself;
    below bfloat16's (float32's) normals a result by 2^-134 (2^-150) more."""
    eps = float(np.float32(eps))
    sizes = [1e-44, 1e-40, 1e-38, 1e-30, 1e-23, 1e-19, 1e-15, 1e-12, 1.0, 1e15, 1e19, 1e25, 1e30, 8e37]
    x = torch.stack([_rand((cols,), i).clamp(-4, 4) * s for i, s in enumerate(sizes)])
    x = torch.where(x == 0, torch.full_like(x, 1e-44), x)
    x = torch.cat([x, x[-3:]])
    x[-3:, ::2] *= 1e-30                          # large and small ones in one row
    x[-3:, 0] = torch.tensor([1e25, 1e30, 3e38], device="cuda")
    w = _rand((cols,), 99)
    for xd in (F32, BF16):
        xt = x.to(xd)
        if eps == 0:
            xt = xt[(xt != 0).any(1)]              # (a row of zeros has no norm)
        ref, r = no.forward(_np(xt), _np(w), eps)
        for dt in (BF16, F32):
            rs = torch.empty(len(xt), device="cuda")
            y = sffn.rms_norm(xt, w, eps=eps, dtype=dt, rstd=rs)
            tol = 36 * U * np.abs(ref) + (2.0 ** -8 * np.abs(ref) * (1 + 36 * U) if dt == BF16 else 0)
            assert (np.abs(_np(y) - ref) <= tol + 2.0 ** (-133 if dt == BF16 else -148)).all()
            fits = r < 3.4e38
            assert (np.abs(_np(rs) - r) <= 36 * U * r + 2.0 ** -148)[fits].all()
            assert torch.isinf(rs[~torch.from_numpy(fits).cuda()]).all()
        # a residual's sum, the norm in place of it
        y, s = sffn.rms_norm(torch.zeros_like(xt), w, residual=xt, eps=eps)
        assert torch.equal(s, xt) and torch.equal(y, sffn.rms_norm(xt, w, eps=eps))
    mixed = torch.cat([x, _rand((9, cols), 5)])[torch.randperm(len(x) + 9, generator=torch.Generator().manual_seed(1))]
    alone = torch.cat([sffn.rms_norm(row[None], w, eps=eps) for row in mixed])
    assert torch.equal(sffn.rms_norm(mixed, w, eps=eps), alone)


@pytest.mark.parametrize("rows,cols", [(1, 8193), (40, 16384), (600, 10000), (3, 5), (3000, 300), (2100, 2048),
                                       (1100, 4096), (700, 6000)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_gradient_in_place_by_rows(rows, cols, dt):
    """ds in the place of each operand in the kernels that form ds and dw together."""
    dy, s, r, w, d = _grads(rows, cols, dt, dt, di=dt)
    ref, rdw = sffn.rms_norm_backward(dy, s, r, w, dstream=d, dtype=dt)
    for i in range(3):
        t = [dy.clone(), s.clone(), d.clone()]
        got, dw = sffn.rms_norm_backward(t[0], t[1], r, w, dstream=t[2], out=t[i])
        assert got is t[i] and torch.equal(got, ref) and torch.equal(dw, rdw)
