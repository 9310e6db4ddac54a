"""The operators around the layers together: the expert layer with experts
that a router has chosen, whole blocks (norm, router, experts, norm, 8-bit
product) eager and captured, and the stack with its fused norm."""
import numpy as np
import pytest
import torch

import unstructured_sparse_feedforward_amd as sffn
from oracle import moe_oracle as mo
from oracle import norm_oracle as no
from oracle import route_oracle as ro
from test_gpu_moe import make, value
from unstructured_sparse_feedforward_amd import workloads as wl
from unstructured_sparse_feedforward_amd.stack import FFNStack

pytestmark = pytest.mark.gpu


def _np(t):
    return t.double().cpu().numpy()


def _ref(layer, x, ws, ids, probs, monkeypatch):
    """y and the oracle's bound for given experts: every expert with the sum of
    the weights that a token gives it."""
    E, F, d = layer.n_experts, layer.d_ff, layer.d
    T, k = ids.shape
    dense = np.zeros((T, E))
    for t in range(T):
        for r in range(k):
            if 0 <= ids[t, r] < E:
                dense[t, ids[t, r]] += probs[t, r]
    w = [value(v, E, F, d) for v in ws]
    out = []
    for p in (dense, np.abs(dense)):
        with monkeypatch.context() as m:
            m.setattr(mo, "route", lambda *a: (np.tile(np.arange(E), (T, 1)), p))
            out.append(mo.forward(_np(x), np.zeros((E, d)), *w, E))
    return out[0][0], out[1][3]


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,d,F,E,k,gated", [
    (1, 128, 32, 1, 1, True), (1, 1024, 352, 10, 3, True), (1, 256, 96, 8, 8, False),
    (2, 128, 64, 30, 2, False), (13, 640, 352, 10, 3, True), (16, 512, 160, 64, 6, True),
    (64, 256, 64, 16, 2, True), (100, 128, 96, 130, 32, True), (256, 256, 32, 7, 3, False)])
def test_chosen_experts(T, d, F, E, k, gated, weights, monkeypatch):
    layer, x, wr, ws = make(T, d, F, E, k, gated, weights)
    g = np.random.default_rng(T + E)
    for kind in ("distinct", "any"):
        # any: the same expert again, indices that are none, weights of both signs and 0
        ids = (np.stack([g.permutation(E)[:k] for _ in range(T)]) if kind == "distinct"
               else g.integers(-2, E + 2, (T, k))).astype(np.int32)
        p = g.standard_normal((T, k)).astype(np.float32)
        if kind == "any":
            p[g.random((T, k)) < 0.1] = 0.0
            ids[T // 2] = -1 if T > 1 else ids[0]
        chosen = (torch.from_numpy(ids).cuda(), torch.from_numpy(p).cuda())
        y = layer.forward(x, None, *ws, chosen=chosen)
        ry, bound = _ref(layer, x, ws, ids, p, monkeypatch)
        err = np.abs(_np(y) - ry)
        assert (err <= bound).all()
        if kind == "any" and T > 1:
            assert (y[T // 2] == 0).all()
        assert torch.equal(y, layer.forward(x, None, *ws, chosen=chosen))


def test_all_pairs_one_expert(monkeypatch):
    """256 tokens that name one expert 32 times over."""
    layer, x, wr, ws = make(256, 128, 32, 32, 32, True, "bf16")
    ids = np.full((256, 32), 5, np.int32)
    p = np.random.default_rng(0).standard_normal((256, 32)).astype(np.float32)
    y = layer.forward(x, None, *ws, chosen=(torch.from_numpy(ids).cuda(), torch.from_numpy(p).cuda()))
    one = p[:, 0].copy()
    for r in range(1, 32):
        one = one + p[:, r]
    ry, bound = _ref(layer, x, ws, ids[:, :1], one[:, None], monkeypatch)
    assert (np.abs(_np(y) - ry) <= bound).all()


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
def test_routers_own_choice(weights):
    """The layer's own experts and weights, given back to it."""
    for T, E, k in ((1, 64, 6), (3, 64, 6), (40, 8, 2)):
        layer, x, wr, ws = make(T, 256, 96, E, k, True, weights)
        y, ids, probs = layer.forward(x, wr, *ws, return_routing=True)
        z = layer.forward(x, None, *ws, chosen=(ids, probs))
        # the same pairs; a single token's sums may be cut otherwise
        assert torch.equal(y, z) if T > 1 else torch.allclose(y, z, rtol=1e-4, atol=1e-5)


def test_chosen_with_n_tokens():
    layer, x, wr, ws = make(20, 256, 64, 16, 4, True, "bf16")
    r = sffn.MoERouter(16, 4, scores="sigmoid")
    logits = x.float() @ wr.float().t()
    full = r.forward(logits)
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    for m in (0, 1, 7, 20):
        n.fill_(m)
        ids = torch.full((20, 4), 123456, dtype=torch.int32, device="cuda")
        probs = torch.full((20, 4), float("nan"), device="cuda")
        r.forward(logits, n_tokens=n, out=(ids, probs))
        y = torch.full((20, 256), 7.0, device="cuda")
        layer.forward(x, None, *ws, y=y, n_tokens=n, chosen=(ids, probs))
        want = layer.forward(x[:m], None, *ws, chosen=(full[0][:m], full[1][:m]))
        assert torch.allclose(y[:m], want, rtol=1e-4, atol=1e-5) and (y[m:] == 7).all()


def test_chosen_refusals():
    layer, x, wr, ws = make(3, 128, 32, 4, 2, True, "bf16")
    ids, p = sffn.MoERouter(4, 2).forward(x.float() @ wr.float().t())
    for kw, why in ((dict(chosen=(ids, p), w_router=wr), "no w_router"),
                    (dict(chosen=(ids, p), return_routing=True), "no w_router"),
                    (dict(chosen=(ids, p), routing=(ids, p)), "no w_router"),
                    (dict(chosen=(ids.long(), p)), "chosen ids"),
                    (dict(chosen=(ids, p.double())), "chosen probs"),
                    (dict(chosen=(ids[:2], p)), "chosen ids"), (dict(), "w_router is missing")):
        with pytest.raises(ValueError, match=why):
            layer.forward(**{**dict(x=x, w_router=None, w_gate=ws[0], w_up=ws[1], w_down=ws[2]), **kw})


class Block:
    """h += experts(norm(h)); h += W_d4 ReLU(W_g4 norm8(h)), in 8 by 4 bits."""

    def __init__(self, T, d=256, F=96, E=16, k=4):
        self.layer, _, self.wr, self.ws = make(T, d, F, E, k, True, "mxfp4")
        g = torch.Generator("cuda").manual_seed(1)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")     # noqa: E731
        self.n1, self.n2 = 1 + 0.1 * r(d), 1 + 0.1 * r(d)
        self.router = sffn.MoERouter(E, k, scores="sigmoid", groups=4, top_groups=2, group_best=2,
                                     scale=1.5)
        self.bias = 0.1 * r(E)
        self.wg, self.wd = r(512, d) / d ** 0.5, r(d, 512) / 512 ** 0.5
        self.g4, self.d4 = sffn.mx_quantize(self.wg), sffn.mx_quantize(self.wd)

    def __call__(self, h, y, n=None, record=None):
        """h and y, the last block's output, float32: h + y goes through."""
        x, h = sffn.rms_norm(y, self.n1, residual=h, n_rows=n)
        logits = x.float() @ self.wr.float().t()
        chosen = self.router.forward(logits, self.bias, n_tokens=n)
        m = self.layer.forward(x, None, *self.ws, n_tokens=n, chosen=chosen)
        q, h2 = sffn.rms_norm(m, self.n2, residual=h, dtype="mxfp8", n_rows=n)
        z = sffn.mx_matmul(q, self.g4)
        a = sffn.mx8_quantize(torch.relu(z))
        out = sffn.mx_matmul(a, self.d4)
        if record is not None:
            record.update(x=x, h=h, logits=logits, chosen=chosen, m=m, q=q, h2=h2, z=z, a=a)
        return h2, out


def test_block_stage_by_stage(monkeypatch):
    T = 24
    b = Block(T)
    g = torch.Generator("cuda").manual_seed(5)
    h, y = (torch.randn(T, 256, generator=g, device="cuda") for _ in range(2))
    s = {}
    h2, out = b(h, y, record=s)
    u = 2.0 ** -24
    assert torch.equal(s["h"], h + y)
    ref = no.forward(_np(s["h"]), _np(b.n1), 1e-6)[0]
    assert (np.abs(_np(s["x"]) - ref) <= (2.0 ** -8 + 33 * u) * np.abs(ref)).all()
    ids, p = ro.forward(_np(s["logits"]), 4, sigmoid=True, bias=_np(b.bias), groups=4, top_groups=2,
                        group_best=2, scale=1.5)
    assert np.array_equal(s["chosen"][0].cpu().numpy(), ids)
    assert (np.abs(_np(s["chosen"][1]) - p) <= 1.01 * u * p).all()
    ry, bound = _ref(b.layer, s["x"], b.ws, ids, _np(s["chosen"][1]), monkeypatch)
    assert (np.abs(_np(s["m"]) - ry) <= bound).all()
    assert torch.equal(s["h2"], s["h"] + s["m"]) and h2 is s["h2"]
    n2 = sffn.rms_norm(s["h2"], b.n2, dtype=torch.float32)
    assert torch.equal(s["q"].codes, sffn.mx8_quantize(n2).codes)
    for a, w, o in ((s["q"], b.g4, s["z"]), (s["a"], b.d4, out)):
        va, vw = _np(sffn.mx8_dequantize(a)), _np(sffn.mx_dequantize(w))
        assert (np.abs(_np(o) - va @ vw.T) <= 2 * va.shape[1] * 2.0 ** -23
                * (np.abs(va) @ np.abs(vw).T)).all()


def test_block_captured_with_fewer_rows():
    """One graph of 24 rows serves batches of any size; rows behind the last do
    not disturb the others, whatever they hold."""
    T = 24
    b = Block(T)
    g = torch.Generator("cuda").manual_seed(6)
    h, y = (torch.zeros(T, 256, device="cuda") for _ in range(2))
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    n.fill_(T)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b(h, y, n)
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            h2, out = b(h, y, n)
    for m in (T, 1, 9, 0, 23):
        nh, ny = (torch.randn(T, 256, generator=g, device="cuda") for _ in range(2))
        nh[m:] = float("nan")
        h.copy_(nh)
        y.copy_(ny)
        n.fill_(m)
        graph.replay()
        torch.cuda.synchronize()
        eh, eo = b(h, y, n)
        assert torch.equal(h2[:m], eh[:m]) and torch.equal(out[:m], eo[:m])
        assert torch.isfinite(out[:m]).all()


def test_stack_with_fused_norm():
    T = 256
    Ws = [wl.stack_layer(i).replace(T=T) for i in (0, 5, 11)]
    inps = [wl.make_inputs(W, seed=3, layer=i) for i, W in enumerate(Ws)]
    bf = lambda a: torch.from_numpy((a.view(np.uint32) >> 16).astype(np.uint16).view(   # noqa: E731
        np.int16)).view(torch.bfloat16).cuda()
    weights = [tuple(bf(getattr(i, k)) for k in ("w_gate", "w_up", "w_down")) for i in inps]
    keep = torch.from_numpy((~inps[0].outlier).astype(np.float32)).to(torch.bfloat16).cuda()
    h0 = torch.from_numpy(inps[0].x).cuda()
    stack = FFNStack(weights, Ws, T, fused_norm=True)
    stack.choose_modes(h0, keep)
    rec = []
    h = stack.forward(h0, keep, record=rec)
    stack.check()
    ref = h0.clone()
    for x, y, _ in rec:
        want = no.forward(_np(ref[:, 1:]), None, 1e-6)[0]
        err = np.abs(_np(x[:, 1:]) - want)
        assert (err <= (2.0 ** -8 + 33 * 2.0 ** -24) * np.abs(want)).all()
        assert torch.equal(x[:, 0], keep)
        ref += y
    assert torch.equal(h, ref)
    # the other way to the same: their layers' inputs differ in bf16 roundings alone
    other = FFNStack(weights, Ws, T)
    other.modes = stack.modes
    first = []
    other.forward(h0, keep, record=first)
    assert (np.abs(_np(first[0][0]) - _np(rec[0][0])) <= 2.0 ** -7 * np.abs(_np(rec[0][0]))).all()
