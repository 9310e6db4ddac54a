"""The choice of experts on the GPU against the float64 oracle: indices
exactly, weights and gradients within bounds.

Scores are formed in 64 bits and rounded once, the weights' scale being a
float32 itself: a weight is off by at most half a step of float32, 2^-24 of
itself, and some 2^-50.

Gradients, with u = 2^-24: exponentials, quotients and products are off by at
most 8 u of themselves, sums over n terms by (7 + n / 64) u of the terms'
magnitudes; a difference g - t of such values and the product with q <= 1 then
by at most 16 (|g| + sum |g| q) q u, E <= 1024 in the sums: taken as 40 u."""
import decimal

import numpy as np
import pytest
import torch

import unstructured_sparse_feedforward_amd as sffn
from oracle import route_oracle as ro

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def _rand(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).cuda()


def _np(t):
    return None if t is None else t.double().cpu().numpy()


CASES = [  # E, k, groups, top_groups, group_best
    (1, 1, 1, 1, 1), (2, 2, 1, 1, 1), (7, 3, 1, 1, 1), (64, 6, 1, 1, 1), (65, 32, 1, 1, 1),
    (128, 8, 4, 2, 2), (200, 5, 8, 3, 1), (256, 8, 8, 4, 2), (256, 8, 8, 8, 2), (300, 10, 3, 1, 2),
    (512, 16, 64, 7, 2), (1000, 9, 1, 1, 1), (1024, 32, 16, 2, 2), (64, 4, 64, 4, 1),
    (6, 6, 3, 3, 2), (6, 2, 3, 1, 2)]


def _router(c, scores, normalize, scale=1.0):
    E, k, G, tg, gb = c
    kw = dict(sigmoid=scores == "sigmoid", groups=G, top_groups=tg, group_best=gb)
    return sffn.MoERouter(E, k, scores=scores, groups=G, top_groups=tg, group_best=gb,
                          normalize=normalize, scale=scale), kw


def _check(c, scores, normalize, scale, logits, bias):
    r, kw = _router(c, scores, normalize, scale)
    ids, p = r.forward(logits, bias)
    oi, op = ro.forward(_np(logits), c[1], bias=_np(bias), normalize=normalize, scale=scale, **kw)
    assert ids.dtype == torch.int32 and p.dtype == F32
    assert np.array_equal(ids.cpu().numpy(), oi)
    assert (np.abs(_np(p) - op) <= 1.01 * U * np.abs(op) + 1e-45).all()
    return r, ids, p


@pytest.mark.parametrize("c", CASES)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_forward(c, scores, biased):
    E = c[0]
    for T, dt, normalize, scale in ((1, F32, True, 1.0), (13, BF16, False, 2.5), (50, F32, True, 0.75)):
        logits = _rand((T, E), T + E, dt, 2.0)
        bias = _rand((E,), E, scale=0.3) if biased else None
        _check(c, scores, normalize, scale, logits, bias)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_ties(scores, biased):
    """Equal logits, biases and groups: the lower index first."""
    g = torch.Generator().manual_seed(3)
    logits = torch.randint(-1, 2, (40, 96), generator=g).float().cuda()
    bias = torch.zeros(96, device="cuda") if biased else None
    for c in ((96, 20, 1, 1, 1), (96, 8, 12, 5, 2), (96, 8, 12, 5, 1)):
        _check(c, scores, True, 1.0, logits, bias)
    # more equal ones than a wave has lanes
    even = torch.full((3, 300), 0.25, device="cuda")
    _check((300, 7, 1, 1, 1), scores, True, 1.0, even,
           torch.full((300,), 0.5, device="cuda") if biased else None)
    z = torch.zeros(2, 96, device="cuda")
    r, _ = _router((96, 5, 4, 2, 2), scores, True)
    assert r.forward(z, bias)[0].tolist() == [[0, 1, 2, 3, 4]] * 2


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_near_ties_need_64_bits(scores):
    """Scores plus bias that float32 cannot tell apart: a bias that makes up for
    the scores' difference but for 2^-40."""
    E = 64
    logits = _rand((30, E), 1)
    s = np.array([ro.choose(l, 1, scores == "sigmoid")[1] for l in _np(logits)])
    bias = (1 - s[0]).astype(np.float32)          # c of token 0: 1 but for a rounding of bias
    c = s[0] + bias.astype(np.float64)
    assert len(set(c.astype(np.float32))) < E / 4 and len(set(c)) > E / 2
    _check((E, 8, 1, 1, 1), scores, True, 1.0, logits, torch.from_numpy(bias).cuda())
    _check((E, 8, 8, 3, 2), scores, True, 1.0, logits, torch.from_numpy(bias).cuda())


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_masked_and_extreme(scores):
    """Masked experts, rows with fewer than k left, rows with none; logits far
    apart; a bias that chooses experts whose scores are nothing."""
    E, k = 40, 4
    l = _rand((8, E), 2)
    l[0, 5:] = -float("inf")
    l[1, 3:] = -float("inf")          # three left for four places
    l[2] = -float("inf")
    l[3] *= 100
    l[4] = 3.0e38
    l[5] = -3.0e38
    l[6, 1] = 600.0
    bias = _rand((E,), 4)
    for c in ((E, k, 1, 1, 1), (E, k, 5, 2, 2)):
        for normalize in (True, False):
            for b in (None, bias):
                r, ids, p = _check(c, scores, normalize, 1.0, l, b)
                assert (p[2] == 0).all() and torch.isfinite(p).all()
    far = torch.zeros(1, E, device="cuda")
    far[0, 7], far[0, 8] = 300.0, 299.0
    b = torch.zeros(E, device="cuda")
    b[20:24] = 5.0
    _, ids, p = _check((E, k, 1, 1, 1), scores, True, 1.0, far, b)
    assert ids.tolist() == [[20, 21, 22, 23]] and (p == 0.25).all()


def test_excluded_by_bias():
    """-infinity in the bias: chosen only where nothing else is left."""
    l = _rand((20, 16), 5)
    b = torch.zeros(16, device="cuda")
    b[::2] = -float("inf")
    r, _ = _router((16, 8, 1, 1, 1), "sigmoid", True)
    assert (r.forward(l, b)[0] % 2 == 1).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("c", [(100, 6, 1, 1, 1), (100, 6, 10, 3, 2)])
def test_nonfinite_stay_in_their_row(bad, c):
    l = _rand((9, 100), 6)
    b = _rand((100,), 7)
    for scores in ("softmax", "sigmoid"):
        for bias in (None, b):
            r, _ = _router(c, scores, True)
            ids, p = r.forward(l, bias)
            m = l.clone()
            m[4, 17] = bad
            i2, p2 = r.forward(m, bias)
            keep = [0, 1, 2, 3, 5, 6, 7, 8]
            assert torch.equal(ids[keep], i2[keep]) and torch.equal(p[keep], p2[keep])
            v = i2[4].tolist()
            assert len(set(v)) == 6 and min(v) >= 0 and max(v) < 100
            d = r.backward(_rand((9, 6), 8), m, i2)
            assert torch.equal(d[keep], r.backward(_rand((9, 6), 8), l, ids)[keep])


def _grad_bound(dp, l, ids, sigmoid, normalize, scale):
    l, dp = _np(l), np.abs(_np(dp)) * scale
    T, E = l.shape
    out = np.zeros((T, E))
    for t in range(T):
        s = np.array(ro._scores(l[t].tolist(), sigmoid))
        c = ids[t]
        q = s[c]
        if normalize and not sigmoid:
            q = np.array(ro._scores(l[t][c].tolist(), False))
        if sigmoid:
            z = q.sum() if normalize else 1.0
            extra = (dp[t] * q).sum() / z if normalize else 0.0
            out[t, c] = (dp[t] + extra) / z * q * (1 - q)
        elif normalize:
            out[t, c] = q * (dp[t] + (dp[t] * q).sum())
        else:
            out[t] = s * (dp[t] * q).sum()
            out[t, c] += s[c] * dp[t]
    return 40 * U * out


@pytest.mark.parametrize("c", CASES)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_backward(c, scores, normalize):
    E, k = c[:2]
    for T, dt, od, scale in ((1, F32, F32, 1.0), (13, BF16, BF16, 2.5), (30, F32, BF16, 1.5)):
        l, dp = _rand((T, E), T + E, dt, 2.0), _rand((T, k), T)
        r, kw = _router(c, scores, normalize, scale)
        ids, _ = r.forward(l, _rand((E,), 9, scale=0.3))
        d = r.backward(dp, l, ids, dtype=od)
        i = ids.cpu().numpy()
        ref = ro.backward(_np(dp), _np(l), i, kw["sigmoid"], normalize, scale)
        # The oracle's own rounding, where the gradient is 0: its Jacobians sum at
        # most E + 2 k < 2^11 products of three values up to 1, |g| and 1 / z,
        # whose factors s_e s_r / z and s_r / z are at most 1: 2^11 2^-53 of
        # sum |g|, for a few roundings a term 2^-40.
        tol = _grad_bound(dp, l, i, kw["sigmoid"], normalize, scale) + \
            2.0 ** -40 * scale * np.abs(_np(dp)).sum(axis=1, keepdims=True)
        if od == BF16:
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol) + 2.0 ** -134
        assert d.dtype == od and (np.abs(_np(d) - ref) <= tol).all()


def test_backward_against_differences():
    """The weights' central differences (step 1e-5, in float64, off by about
    1e-9) in random directions, the choice held."""
    g = np.random.default_rng(0)
    for c in ((30, 5, 1, 1, 1), (64, 6, 8, 3, 2)):
        for scores in ("softmax", "sigmoid"):
            for normalize in (True, False):
                r, kw = _router(c, scores, normalize, 1.25)
                l, dp = _rand((4, c[0]), 1), _rand((4, c[1]), 2)
                ids, _ = r.forward(l)
                d = _np(r.backward(dp, l, ids))
                i = ids.cpu().numpy()
                for _ in range(3):
                    e = g.standard_normal((4, c[0]))
                    f = lambda h: sum(np.dot(_np(dp)[t], ro.weights(     # noqa: E731
                        _np(l)[t] + h * e[t], i[t], kw["sigmoid"], normalize, 1.25)) for t in range(4))
                    num = (f(1e-5) - f(-1e-5)) / 2e-5
                    assert abs(num - (d * e).sum()) <= 1e-5 * (np.abs(d * e).sum() + 1e-3)


def test_backward_of_masked():
    l = _rand((4, 40), 2)
    l[0, 5:] = -float("inf")
    l[1] = -float("inf")
    for scores in ("softmax", "sigmoid"):
        for normalize in (True, False):
            r, _ = _router((40, 4, 1, 1, 1), scores, normalize)
            ids, _ = r.forward(l)
            d = r.backward(_rand((4, 4), 3), l, ids)
            assert torch.isfinite(d).all() and (d[0, 5:] == 0).all() and (d[1] == 0).all()


def test_bad_indices_are_not_chosen():
    l, dp = _rand((3, 40), 2), _rand((3, 4), 3)
    for scores in ("softmax", "sigmoid"):
        for normalize in (True, False):
            r, kw = _router((40, 4, 1, 1, 1), scores, normalize)
            ids = torch.tensor([[1, -1, 40, 3], [-5, 1 << 30, -1, -1], [0, 1, 2, 39]],
                               dtype=torch.int32, device="cuda")
            d = r.backward(dp, l, ids)
            ref = ro.backward(_np(dp), _np(l), ids.cpu().numpy(), kw["sigmoid"], normalize, 1.0)
            assert np.allclose(_np(d), ref, rtol=1e-5, atol=1e-6)


def test_views_out_n_tokens():
    big = _rand((50, 100), 4)
    l = big[::2, 3:67]
    r, _ = _router((64, 6, 8, 4, 2), "sigmoid", True)
    ids, p = r.forward(l.contiguous())
    i2, p2 = r.forward(l)
    assert torch.equal(ids, i2) and torch.equal(p, p2)
    dp = _rand((25, 6), 5)
    d = r.backward(dp, l, ids)
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    for v, m in ((0, 0), (1, 1), (9, 9), (25, 25), (77, 25), (-1, 0)):
        n.fill_(v)
        out = (torch.full_like(ids, 77), torch.full_like(p, 7.0))
        got = r.forward(l, n_tokens=n, out=out)
        assert got[0] is out[0] and got[1] is out[1]
        assert torch.equal(out[0][:m], ids[:m]) and (out[0][m:] == 77).all()
        assert torch.equal(out[1][:m], p[:m]) and (out[1][m:] == 7).all()
        buf = torch.full((25, 80), 7.0, device="cuda")
        o = buf[:, 5:69]
        assert r.backward(dp, l, ids, n_tokens=n, out=o) is o
        assert torch.equal(o[:m], d[:m])
        o[:m] = 7
        assert (buf == 7).all()


def _plain(l, c, scores, bias, normalize):
    """The definition in float64 torch operations."""
    E, k, G, tg, gb = c
    l = l.double()
    s = torch.softmax(l, 1) if scores == "softmax" else torch.sigmoid(l)
    ch = s if bias is None else s + bias.double()
    key = l if bias is None else ch
    if tg < G:
        g = ch.view(-1, G, E // G).sort(dim=2, descending=True).values[:, :, :gb].sum(2)
        kept = g.sort(dim=1, descending=True, stable=True).indices[:, :tg]
        keep = torch.zeros_like(g, dtype=torch.bool).scatter_(1, kept, True)
        key = key.masked_fill(~keep.repeat_interleave(E // G, 1), -float("inf"))
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    p = s.gather(1, ids)
    return ids, p / p.sum(1, keepdim=True) if normalize else p


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("c", [(64, 6, 1, 1, 1), (64, 15, 16, 5, 2), (60, 8, 4, 2, 2), (5, 2, 1, 1, 1),
                               (64, 16, 1, 1, 1), (96, 5, 1, 1, 1), (128, 31, 32, 11, 2),
                               (128, 8, 4, 2, 1), (256, 8, 8, 4, 2)])
def test_many_tokens(c, scores, biased):
    """Several tokens a wave, the last wave's not all there; against sorting,
    bfloat16 logits (with ties, of groups too) as well."""
    for T, dt, normalize in ((20001, F32, True), (9003, BF16, False), (5000, BF16, True)):
        l = _rand((T, c[0]), 6, dt)
        bias = _rand((c[0],), 7, scale=0.2) if biased else None
        r, _ = _router(c, scores, normalize)
        ids, p = r.forward(l, bias)
        oi, op = _plain(l, c, scores, bias, normalize)
        assert torch.equal(ids.long(), oi)
        assert ((p.double() - op).abs() <= 1.01 * U * op).all()


def test_many_tokens_masked_and_counted():
    """Several tokens a wave with masked experts, rows without any, equal ones
    throughout, and fewer tokens than rows."""
    for c in ((64, 6, 1, 1, 1), (64, 6, 8, 3, 2), (128, 8, 1, 1, 1)):
        T, E, k = 9000, c[0], c[1]
        l = _rand((T, E), 3)
        l[::7] = -float("inf")
        l[1::7, k - 2:] = -float("inf")
        l[2::7] = 0.5
        l[3::7, 5] = float("nan")
        bias = _rand((E,), 4, scale=0.2)
        bias[::3] = 0
        for scores in ("softmax", "sigmoid"):
            for b in (None, bias, torch.zeros_like(bias)):
                r, kw = _router(c, scores, True)
                ids, p = r.forward(l, b)
                for rows in (slice(0, 28), slice(T - 28, T)):
                    keep = [i for i in range(28) if (i + (0 if rows.start == 0 else T - 28)) % 7 != 3]
                    oi, op = ro.forward(_np(l[rows])[keep], k, bias=_np(b), **kw)
                    assert np.array_equal(ids[rows].cpu().numpy()[keep], oi)
                    assert (np.abs(_np(p[rows])[keep] - op) <= 1.01 * U * op + 1e-45).all()
                n = torch.full((1,), 4097, dtype=torch.int32, device="cuda")
                out = (torch.full_like(ids, 77), torch.full_like(p, 7.0))
                r.forward(l, b, n_tokens=n, out=out)
                assert torch.equal(out[0][:4097], ids[:4097]) and (out[0][4097:] == 77).all()
                assert (out[1][4097:] == 7).all()


def test_empty_and_refusals():
    r = sffn.MoERouter(8, 2)
    ids, p = r.forward(torch.empty(0, 8, device="cuda"))
    assert ids.shape == p.shape == (0, 2)
    assert r.backward(p, torch.empty(0, 8, device="cuda"), ids).shape == (0, 8)
    l = torch.zeros(3, 8, device="cuda")
    for f, why in ((lambda: r.forward(l[:, :7]), "logits must"), (lambda: r.forward(l.half()), "float32"),
                   (lambda: r.forward(l[0]), "logits must"), (lambda: r.forward(l.cpu()), "GPU"),
                   (lambda: r.forward(l.t().contiguous().t()), "contiguous rows"),
                   (lambda: r.forward(l, l[0, :7]), "bias"),
                   (lambda: r.forward(l, l[0].bfloat16()), "bias"),
                   (lambda: r.forward(l, n_tokens=l[0]), "n_tokens"),
                   (lambda: r.forward(l, out=(ids, p)), "ids must"),
                   (lambda: r.backward(p, l, ids), "dprobs must")):
        with pytest.raises(ValueError, match=why):
            f()


def test_graph():
    l, dp = _rand((70, 64), 7), _rand((70, 6), 8)
    b = _rand((64,), 9)
    r, _ = _router((64, 6, 8, 4, 2), "sigmoid", True)
    buf = l.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        r.forward(buf, b)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            ids, p = r.forward(buf, b)
            d = r.backward(dp, buf, ids)
    for f in (1.0, -1.0, 0.3):
        buf.copy_(l * f)
        g.replay()
        torch.cuda.synchronize()
        i2, p2 = r.forward(buf, b)
        assert torch.equal(ids, i2) and torch.equal(p, p2)
        assert torch.equal(d, r.backward(dp, buf, i2))


def test_most_tokens():
    """2^25 tokens, the most of a call: a window at each end and in the middle against
    the same window alone, and nothing left out."""
    T, E, k = 1 << 25, 8, 2
    logits = torch.randn(T, E, generator=torch.Generator(device="cuda").manual_seed(1),
                         device="cuda", dtype=torch.float32)
    r = sffn.MoERouter(E, k)
    out = (torch.full((T, k), -7, dtype=torch.int32, device="cuda"),
           torch.full((T, k), float("nan"), device="cuda"))
    ids, probs = r.forward(logits, out=out)
    assert (ids >= 0).all() and not probs.isnan().any()
    dl = r.backward(torch.ones_like(probs), logits, ids, out=torch.full_like(logits, float("nan")))
    assert not dl.isnan().any()
    for a in (0, T // 2 - 500, T - 1000):
        i, p = r.forward(logits[a:a + 1000])
        assert torch.equal(i, ids[a:a + 1000])
        # (so few tokens take a kernel of other lanes, whose sums have another order: E + k
        # roundings and an exponential's at each side)
        assert torch.allclose(p, probs[a:a + 1000], rtol=2 * (E + k + 4) * 2.0 ** -24, atol=0)


def _sigmoid_gradient(dp, l, ids, scale):
    """(the gradient of normalised sigmoid weights, its bound) of one token, from
    the definition with 60 digits. Bound: q = s / S is the 64-bit one rounded, the
    scores' gradient and sums as in the head of this file, 40 u q (1 - s) (|g| +
    sum |g| q); a q below float32's smallest normal is off by 2^-150 itself."""
    D = decimal.Decimal
    with decimal.localcontext() as c:
        c.prec = 60
        s = [1 / (1 + (-D(float(v))).exp()) for v in l]
        g = [D(float(v)) * D(scale) for v in dp]
        S = sum(s[e] for e in ids)
        t = sum(gr * s[e] for gr, e in zip(g, ids)) / S
        ta = sum(abs(gr) * s[e] for gr, e in zip(g, ids)) / S
        d, b = np.zeros(len(l)), np.zeros(len(l))
        for gr, e in zip(g, ids):
            d[e] = float((gr - t) / S * s[e] * (1 - s[e]))
            b[e] = float((abs(gr) + ta) * (D(40 * U) * s[e] / S * (1 - s[e]) + D(2) ** -148))
    return d, b


@pytest.mark.parametrize("top", [-30.0, -80.0, -86.0, -87.2, -88.0, -88.5, -90.0, -100.0, -103.5, -300.0,
                                 -700.0])
@pytest.mark.parametrize("by", [1.0, 65536.0])
def test_backward_of_far_logits(top, by):
    """Normalised sigmoid weights of experts whose scores float32 cannot hold, as
    the forward pass forms them; beside ordinary ones; loss scaling."""
    E, k, scale = 40, 4, 2.5
    l = _rand((6, E), 3, scale=0.5) + top
    l[4, 7:9] = torch.tensor([0.5, -1.0])          # ordinary ones, and others with them
    l[5, 3] = 90.0
    r, _ = _router((E, k, 1, 1, 1), "sigmoid", True, scale)
    ids, p = r.forward(l)
    assert (torch.abs(p.sum(1) - scale) < 1e-5).all()
    dp = by * _rand((6, k), 4)
    d = _np(r.backward(dp, l, ids))
    for t in range(6):
        ref, bound = _sigmoid_gradient(_np(dp)[t], _np(l)[t], ids[t].tolist(), scale)
        assert (np.abs(d[t] - ref) <= bound).all(), (t, d[t][ids[t].tolist()], ref[ids[t].tolist()])
    # weights that are not normalised: s (1 - s) g, as far as float32 holds it
    r, _ = _router((E, k, 1, 1, 1), "sigmoid", False, scale)
    d = _np(r.backward(dp, l, ids))
    for t in range(6):
        for g, e in zip(_np(dp)[t], ids[t].tolist()):
            v = _np(l)[t, e]
            ref = scale * g * np.exp(-abs(v)) / (1 + np.exp(-abs(v))) ** 2
            assert abs(d[t, e] - ref) <= 40 * U * abs(ref) + 2.0 ** -149


def test_backward_where_every_score_is_0():
    """Logits whose scores are 0 in 64 bits too: the weights are, and their gradient."""
    r, _ = _router((8, 2, 1, 1, 1), "sigmoid", True)
    l = torch.tensor([[-709.78], [-709.79], [-800.0], [-float("inf")]], device="cuda").repeat(1, 8)
    ids, p = r.forward(l)
    d = r.backward(torch.tensor([[1.0, -2.0]] * 4, device="cuda"), l, ids)
    assert (p[0] == 0.5).all() and (p[1:] == 0).all()
    # q = 1/2 each, g - sum g q = 1.5 and -1.5
    assert d[0, :2].tolist() == [0.75, -0.75] and (d[0, 2:] == 0).all() and (d[1:] == 0).all()


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("c,T", [((64, 6, 1, 1, 1), 5000), ((64, 6, 8, 3, 2), 5000), ((60, 15, 4, 2, 1), 5003),
                                 ((128, 8, 1, 1, 1), 9000), ((128, 9, 16, 5, 2), 9001),
                                 ((256, 8, 8, 4, 2), 700), ((1000, 20, 1, 1, 1), 90)])
def test_many_near_ties(c, T, scores):
    """Scores plus bias that 32 bits cannot tell apart, of all experts of every
    other token: tokens of one wave need 64 bits one after the other."""
    E = c[0]
    g = torch.Generator().manual_seed(E + T)
    u, noise = torch.rand(E, generator=g).double(), torch.rand(T, E, generator=g).double()
    if scores == "sigmoid":
        bias = (0.5 * u).float()
        s = 0.9 - bias.double() + 1e-7 * noise
        l = torch.log(s / (1 - s)).float()
    else:
        bias = (0.5 / E * u).float()
        s = (1 + bias.double().sum()) / E - bias.double() + 1e-9 * noise
        l = torch.log(s).float()
    l[1::4] = torch.randn(l[1::4].shape, generator=g)
    l[3::4] = torch.randn(l[3::4].shape, generator=g)
    l, bias = l.cuda(), bias.cuda()
    near = (torch.softmax(l[:1].double(), 1) if scores == "softmax" else torch.sigmoid(l[:1].double())) + bias
    assert len(set(near[0].tolist())) == E and near.max() - near.min() < 2.0 ** -20
    r, _ = _router(c, scores, True)
    for b in (bias, None):
        ids, p = r.forward(l, b)
        oi, op = _plain(l, c, scores, b, True)
        assert torch.equal(ids.long(), oi)
        assert ((p.double() - op).abs() <= 1.01 * U * op).all()


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_backward_in_place(scores, normalize):
    for (E, k), dt in (((64, 6), F32), ((300, 8), BF16), ((1000, 20), F32)):
        r, _ = _router((E, k, 1, 1, 1), scores, normalize)
        l, dp = _rand((700, E + 5), 1, dt)[:, 2:2 + E], _rand((700, k), 2)
        ids, _ = r.forward(l)
        d = r.backward(dp, l, ids, dtype=dt)
        assert r.backward(dp, l, ids, out=l) is l and torch.equal(d, l)
