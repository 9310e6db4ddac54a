"""The expert layer on the GPU against its float64 oracle, within the bound
that the oracle derives for float32 sums."""
import math

import numpy as np
import pytest
import torch

import moe_pins as mp
import unstructured_sparse_feedforward_amd as sffn
from oracle import moe_oracle as mo

pytestmark = pytest.mark.gpu


def make(T, d, F, E, k, gated, weights, active=0.5, seed=0, normalize=True):
    """Layer and inputs; ``active``: the expected fraction of active neurons,
    by a gate threshold on column 0 of x (always 1)."""
    g = torch.Generator("cuda").manual_seed(seed + 1000 * T + d + F + E + k)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = r(T, d)
    x[:, 0] = 1.0
    tau = math.sqrt(2) * float(torch.erfinv(torch.tensor(1 - 2 * active)))
    wg = r(E, F, d) / math.sqrt(d)
    wg[:, :, 0] = -tau
    wu = r(E, F, d) / math.sqrt(d) if gated else None
    wd = r(E, F, d) / math.sqrt(F)
    bf = lambda t: None if t is None else t.to(torch.bfloat16)
    x, wr, ws = bf(x), bf(r(E, d) / math.sqrt(d)), [bf(w) for w in (wg, wu, wd)]
    layer = sffn.SparseMoE(d, F, E, k, gated=gated, normalize=normalize, weights=weights)
    if weights == "mxfp4":
        ws = [None if w is None else sffn.mx_quantize(w.view(E * F, d)) for w in ws]
    return layer, x, wr, ws


def value(w, E, F, d):
    if w is None:
        return None
    v = sffn.mx_dequantize(w) if isinstance(w, sffn.MXTensor) else w
    return v.double().cpu().numpy().reshape(E, F, d)


def ref(layer, x, wr, ws):
    E, F, d = layer.n_experts, layer.d_ff, layer.d
    return mo.forward(x.double().cpu().numpy(), wr.double().cpu().numpy(),
                      *[value(w, E, F, d) for w in ws], layer.top_k, layer.normalize)


def check(layer, x, wr, ws, out):
    y, ids, probs = out
    ry, rids, rp, bound = ref(layer, x, wr, ws)
    assert np.array_equal(ids.cpu().numpy(), rids)
    # exponential and quotient: a few steps of 2^-23 of the weight
    assert (np.abs(probs.double().cpu().numpy() - rp) <= 64 * 2.0 ** -23 * rp).all()
    err = np.abs(y.double().cpu().numpy() - ry)
    assert (err <= bound).all(), (err / np.maximum(bound, 1e-300)).max()


CASES = [
    # T, d, F, E, k, gated
    (1, 128, 32, 1, 1, True), (1, 1024, 352, 10, 3, True), (1, 256, 96, 8, 8, False),
    (2, 128, 64, 3, 2, False), (13, 640, 352, 10, 3, False), (13, 640, 352, 10, 3, True),
    (16, 512, 160, 64, 6, True), (17, 384, 32, 5, 1, True), (33, 256, 128, 4, 4, True),
    (64, 2048, 64, 16, 2, True), (100, 128, 96, 130, 32, True), (256, 256, 32, 7, 3, False),
    (256, 128, 160, 2, 2, True), (5, 8192, 32, 2, 1, True)]


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,d,F,E,k,gated", CASES)
def test_forward(T, d, F, E, k, gated, weights):
    print(T, d, F, E, k, gated, weights, flush=True)
    layer, x, wr, ws = make(T, d, F, E, k, gated, weights, normalize=(T + k) % 2 == 0)
    out = layer.forward(x, wr, *ws, return_routing=True)
    check(layer, x, wr, ws, out)
    again = layer.forward(x, wr, *ws)
    assert torch.equal(again, out[0])


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
@pytest.mark.parametrize("active", [0.002, 0.03, 0.2])
@pytest.mark.parametrize("T", [1, 12, 40])
def test_sparse_activations(T, active, weights):
    layer, x, wr, ws = make(T, 256, 1024, 6, 2, True, weights, active=active)
    check(layer, x, wr, ws, layer.forward(x, wr, *ws, return_routing=True))


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
def test_long_slices(weights):
    """Enough experts and neurons for the longest slices, in full and cut
    (1000 = 7 * 128 + 104 neurons would not be a multiple of 32: 1120 =
    8 * 128 + 96)."""
    layer, x, wr, ws = make(24, 128, 1120, 64, 8, True, weights, active=0.1)
    check(layer, x, wr, ws, layer.forward(x, wr, *ws, return_routing=True))


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
def test_nothing_active(weights):
    """Every pre-activation negative: zeros, not what the buffer held."""
    layer, x, wr, ws = make(9, 256, 64, 4, 2, True, "bf16")
    ws[0] = -torch.ones_like(ws[0]).abs()
    x = x.abs()
    if weights == "mxfp4":
        layer = sffn.SparseMoE(256, 64, 4, 2, weights="mxfp4")
        ws = [sffn.mx_quantize(w.view(-1, 256)) for w in ws]
    y = torch.full((9, 256), 7.0, device="cuda")
    layer.forward(x, wr, *ws, y=y)
    assert (y == 0).all()


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,d,F,E,k,gated", [
    # more neurons than the down product lists at a time, and the most
    (3, 128, 8224, 2, 2, True), (40, 128, 8224, 2, 1, False), (2, 128, 65536, 1, 1, True)])
def test_many_neurons(T, d, F, E, k, gated, weights):
    print(T, d, F, E, k, gated, weights, flush=True)
    layer, x, wr, ws = make(T, d, F, E, k, gated, weights, active=0.3)
    check(layer, x, wr, ws, layer.forward(x, wr, *ws, return_routing=True))


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,d,F,E,k,gated", [
    # an expert's tokens and neurons over several workgroups: all in one expert,
    # uneven blocks, ranges of neurons that the last one cuts
    (128, 128, 2080, 1, 1, True), (33, 256, 4128, 2, 1, True), (200, 128, 2048, 3, 2, False),
    (17, 128, 5632, 1, 1, True), (1, 128, 4128, 8, 2, True), (256, 128, 96, 1, 1, True),
    (70, 128, 64, 2, 2, True)])
def test_few_experts(T, d, F, E, k, gated, weights):
    print(T, d, F, E, k, gated, weights, flush=True)
    layer, x, wr, ws = make(T, d, F, E, k, gated, weights, active=0.3)
    out = layer.forward(x, wr, *ws, return_routing=True)
    check(layer, x, wr, ws, out)
    assert torch.equal(layer.forward(x, wr, *ws), out[0])
    # the same call with fewer valid tokens than it was planned for
    n = torch.tensor([T // 3 + 1], dtype=torch.int32, device="cuda")
    m = int(n)
    y = torch.full((T, d), 7.0, device="cuda")
    layer.forward(x, wr, *ws, y=y, n_tokens=n, routing=(out[1], out[2]))
    assert (y[m:] == 7).all()
    check(layer, x[:m], wr, ws, (y[:m], out[1][:m], out[2][:m]))


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 2, 1), (1, 64, 32), (1, 65, 2), (1, 127, 31), (1, 128, 32),
                                   (1, 129, 32), (1, 300, 5), (1, 1024, 32), (3, 1024, 32),
                                   (9, 16, 4), (9, 17, 4)])
def test_many_experts(T, E, k, normalize):
    """Around the sizes at which another kernel routes."""
    print(T, E, k, normalize, flush=True)
    layer, x, wr, ws = make(T, 128, 32, E, k, True, "bf16", normalize=normalize)
    check(layer, x, wr, ws, layer.forward(x, wr, *ws, return_routing=True))


@pytest.mark.parametrize("T", [1, 5])
def test_extreme_logits(T):
    """Logits so far apart that the smaller weights vanish, and all of them
    negative: exact zeros, no NaN."""
    layer, x, wr, ws = make(T, 128, 32, 40, 4, True, "bf16")
    wr.zero_()
    wr[:, 0] = -1e4 * torch.arange(1, 41, device="cuda").bfloat16()
    y, ids, probs = layer.forward(x, wr, *ws, return_routing=True)
    assert ids.tolist() == [[0, 1, 2, 3]] * T and probs.tolist() == [[1.0, 0.0, 0.0, 0.0]] * T
    check(layer, x, wr, ws, (y, ids, probs))


def test_everyone_to_one_expert():
    """All 256 tokens in one expert's list, none in the others'."""
    layer, x, wr, ws = make(256, 128, 96, 9, 1, True, "bf16")
    wr.zero_()
    wr[4, 0] = 1.0
    out = layer.forward(x, wr, *ws, return_routing=True)
    assert (out[1] == 4).all() and (out[2] == 1).all()
    check(layer, x, wr, ws, out)


@pytest.mark.parametrize("k", [1, 3, 70])
def test_ties_go_to_the_lowest(k):
    layer, x, wr, ws = make(6, 128, 32, 100, min(k, 32), False, "bf16")
    wr.zero_()
    wr[70:, 0] = 1.0        # thirty equal winners, then seventy equal others
    out = layer.forward(x, wr, *ws, return_routing=True)
    want = (list(range(70, 100)) + list(range(70)))[:layer.top_k]
    assert out[1].tolist() == [want] * 6
    check(layer, x, wr, ws, out)


def test_negative_zero_ties():
    layer, x, wr, ws = make(3, 128, 32, 4, 2, False, "bf16")
    wr.zero_()
    wr[0] = -0.0
    x[:] = 1.0
    x[:, 1] = -1.0
    _, ids, _ = layer.forward(x, wr, *ws, return_routing=True)
    assert ids.tolist() == [[0, 1]] * 3


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("normalize", [True, False])
def test_nonfinite_token(bad, normalize):
    """A NaN or infinity in one token's row: its own row is lost, the others
    are right, and its experts are valid. (Not bit for bit as without it:
    the neurons that only this token kept active take positions in the
    others' float32 sums, whose order the oracle's bound leaves open.)"""
    layer, x, wr, ws = make(20, 256, 96, 5, 2, True, "bf16", normalize=normalize)
    x[7, 3] = bad
    y, ids, probs = layer.forward(x, wr, *ws, return_routing=True)
    keep = [t for t in range(20) if t != 7]
    check(layer, x[keep], wr, ws, (y[keep], ids[keep], probs[keep]))
    if math.isnan(bad):
        assert torch.isnan(y[7]).all() and ids[7].tolist() == [0, 1]
    else:
        assert not torch.isfinite(y[7]).any()
    assert ((ids >= 0) & (ids < 5)).all() and (ids[:, 0] != ids[:, 1]).all()


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
@pytest.mark.parametrize("n", [-3, 0, 1, 11, 30, 99])
def test_padded_batch(n, weights):
    """Rows from n_tokens on: not read (they hold NaN), not written."""
    layer, x, wr, ws = make(30, 256, 96, 5, 2, True, weights)
    v = min(max(n, 0), 30)
    x[v:] = float("nan")
    y = torch.full((30, 256), 7.0, device="cuda")
    ids = torch.full((30, 2), -9, dtype=torch.int32, device="cuda")
    probs = torch.full((30, 2), 5.0, device="cuda")
    nt = torch.tensor([n], dtype=torch.int32, device="cuda")
    layer.forward(x, wr, *ws, y=y, n_tokens=nt, routing=(ids, probs))
    assert (y[v:] == 7).all() and (ids[v:] == -9).all() and (probs[v:] == 5).all()
    if v:
        check(layer, x[:v], wr, ws, (y[:v], ids[:v], probs[:v]))


def test_workspace_contents_do_not_matter():
    layer, x, wr, ws = make(12, 256, 96, 5, 2, True, "bf16")
    import ctypes
    from unstructured_sparse_feedforward_amd import binding as B
    nb = layer.workspace_bytes(12)
    outs = []
    for fill in (0, 255):
        buf = torch.full((nb,), fill, dtype=torch.uint8, device="cuda")
        y = torch.empty(12, 256, device="cuda")
        w = B.SffnMoeWeights(wr.data_ptr(), *[t.data_ptr() for t in ws], None, None, None)
        st = layer.lib.sffn_moe_forward(ctypes.byref(layer.desc), x.data_ptr(), ctypes.byref(w), 12,
                                        None, y.data_ptr(), None, None, buf.data_ptr(), nb,
                                        B._stream())
        assert st == B.SFFN_OK
        outs.append(y)
    assert torch.equal(*outs) and torch.isfinite(outs[0]).all()


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
def test_graphs_and_streams(weights):
    """Two captured graphs of one layer, replayed in turn with other inputs
    and token counts and eager work between, and two streams at once."""
    layer, x, wr, ws = make(20, 256, 160, 8, 2, True, weights)
    xs, n = x.clone(), torch.tensor([20], dtype=torch.int32, device="cuda")
    ya, yb = torch.zeros(20, 256, device="cuda"), torch.zeros(7, 256, device="cuda")
    layer.forward(xs, wr, *ws, y=ya, n_tokens=n)
    torch.cuda.synchronize()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        layer.forward(xs, wr, *ws, y=ya, n_tokens=n)
    with torch.cuda.graph(gb):
        layer.forward(xs[:7], wr, *ws, y=yb)
    for i, m in enumerate((20, 3, 17, 1)):
        xs.copy_(torch.roll(x, i, 0))
        n.fill_(m)
        ya.fill_(7.0)
        eager = layer.forward(xs, wr, *ws, n_tokens=n)
        small = layer.forward(xs[:7].contiguous(), wr, *ws)
        ga.replay()
        gb.replay()
        torch.cuda.synchronize()
        assert torch.equal(ya[:m], eager[:m]) and (ya[m:] == 7).all()
        assert torch.equal(yb, small)
    xs.copy_(x)
    want = layer.forward(x, wr, *ws)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(4):
        for s in sides:
            with torch.cuda.stream(s):
                outs.append(layer.forward(x, wr, *ws))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_refusals_on_the_gpu():
    layer, x, wr, ws = make(4, 256, 96, 5, 2, True, "bf16")
    q, _, _, qs = make(4, 256, 96, 5, 2, True, "mxfp4")
    ng = sffn.SparseMoE(256, 96, 5, 2, gated=False)
    one = torch.tensor([1], dtype=torch.int32, device="cuda")
    for f in (lambda: layer.forward(x.float(), wr, *ws), lambda: layer.forward(x[:, :128], wr, *ws),
              lambda: layer.forward(x, wr[:4], *ws), lambda: layer.forward(x, wr, ws[0], None, ws[2]),
              lambda: layer.forward(x, wr, *qs), lambda: q.forward(x, wr, *ws),
              lambda: ng.forward(x, wr, *ws), lambda: layer.forward(x, wr, ws[0][:, :64], *ws[1:]),
              lambda: layer.forward(x, wr, *ws, y=torch.empty(4, 256, device="cuda").bfloat16()),
              lambda: layer.forward(x, wr, *ws, n_tokens=one.long()),
              lambda: layer.forward(x, wr, *ws, n_tokens=one.cpu()),
              lambda: layer.forward(x, wr, *ws, n_tokens=one.expand(2)),
              lambda: layer.forward(x.repeat(65, 1), wr, *ws),
              lambda: layer.forward(x, wr, *ws, routing=(one, one))):
        with pytest.raises(ValueError):
            f()
    odd = torch.empty(4 * 256 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(4, 256)
    for f in (lambda: layer.forward(odd, wr, *ws),
              lambda: layer.forward(x, wr, *ws, y=torch.empty(1025, device="cuda")[1:].view(4, 256))):
        with pytest.raises(sffn.SffnError):
            f()
    assert layer.forward(x[:0], wr, *ws).shape == (0, 256)


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("T,d,F", [(1, 128, 32), (4, 128, 128), (5, 256, 96), (16, 128, 64),
                                   (40, 256, 256), (200, 128, 128)])
def test_h_enters_the_down_product_with_24_bits(T, d, F, gated, weights):
    """Results that float32 holds exactly and that need every bit of h."""
    x, gate, up, down, y = mp.hidden_24_bits(T, d, F, gated, seed=T + d)
    bf = lambda a: torch.from_numpy(a).cuda().to(torch.bfloat16)
    # two experts; the second, which these are, has the larger logit
    ws = [None if w is None else torch.stack([bf(np.flip(w, 0).copy()), bf(w)])
          for w in (gate, up, down)]
    wr = torch.zeros(2, d, device="cuda", dtype=torch.bfloat16)
    wr[1, 3] = 1.0
    if weights == "mxfp4":
        ws = [None if w is None else sffn.mx_quantize(w.view(2 * F, d)) for w in ws]
    layer = sffn.SparseMoE(d, F, 2, 1, gated=gated, weights=weights)
    out, ids, probs = layer.forward(bf(x), wr, *ws, return_routing=True)
    assert (ids == 1).all() and (probs == 1).all()
    assert np.array_equal(out.double().cpu().numpy(), y)


# the kernels that route: the hidden kernel (one token, up to 128 experts), the
# router's with the logits in it (up to 16 experts) and without
ROUTES = [(1, 2), (1, 16), (1, 17), (1, 64), (1, 65), (1, 128), (1, 129), (1, 1024), (5, 2), (5, 16),
          (5, 17), (5, 300), (3, 1024)]


@pytest.mark.parametrize("d", [128, 640, 8192])
@pytest.mark.parametrize("T,E", ROUTES)
def test_logits_in_64_bits(T, E, d):
    """Two logits that 32 bits do not tell apart: the larger one, of higher
    index, comes first."""
    if E * d > 1 << 18:
        E = (1 << 18) // d      # (the weights stay small)
    w, want = mp.near_tie(E, d)
    layer, x, wr, ws = make(T, d, 32, E, 2, True, "bf16")
    x.zero_()
    x[:, [0, d - 1]] = 1.0
    wr.copy_(torch.from_numpy(w))
    out = layer.forward(x, wr, *ws, return_routing=True)
    assert out[1].tolist() == [want] * T
    check(layer, x, wr, ws, out)


@pytest.mark.parametrize("T,E", ROUTES)
def test_logits_are_summed_in_one_order(T, E):
    """Products too far apart for exact sums: a lane's columns are added in
    ascending order, whichever kernel routes."""
    layer, x, wr, ws = make(T, 128, 32, E, 2, True, "bf16")
    x.zero_()
    x[:, :3] = 1.0
    wr.zero_()
    wr[:, 0] = -1.0
    wr[0, :3] = torch.tensor([1.0, 2.0 ** 60, -2.0 ** 60])      # (1 + 2^60) - 2^60 = 0
    wr[E - 1, :3] = torch.tensor([2.0 ** 60, -2.0 ** 60, 1.0])  # 1
    _, ids, _ = layer.forward(x, wr, *ws, return_routing=True)
    assert ids.tolist() == [[E - 1, 0]] * T


@pytest.mark.parametrize("active", [0.1, 0.8])
@pytest.mark.parametrize("T,d,F,E,k,gated,weights", [
    # the longest slices (64 neurons of bf16, 128 of codes): every wave a tile
    # of its own, and with eight in ten active more than 64 neurons of codes in
    # the up product. One block of 16 tokens a pass, the last slice cut (32 of
    # 64, 96 of 128) and whole, d of one step and of many
    (64, 128, 1120, 128, 8, True, "bf16"), (64, 128, 1120, 128, 8, True, "mxfp4"),
    (64, 128, 1152, 128, 8, True, "bf16"), (64, 128, 1152, 128, 8, True, "mxfp4"),
    (64, 128, 1120, 128, 8, False, "bf16"), (64, 128, 1120, 128, 8, False, "mxfp4"),
    # a single token
    (1, 128, 4064, 32, 32, True, "bf16"), (1, 128, 4064, 32, 32, True, "mxfp4"),
    (1, 1024, 4064, 32, 32, True, "bf16"), (1, 1024, 4096, 32, 32, True, "mxfp4"),
    # a unit for each pair of several tokens
    (3, 128, 1440, 128, 32, True, "bf16"), (3, 128, 1440, 128, 32, True, "mxfp4"),
    # two blocks a pass, one pass and several
    (128, 128, 1120, 128, 16, True, "bf16"), (128, 128, 1120, 128, 16, True, "mxfp4"),
    (200, 128, 4064, 32, 4, True, "bf16"), (200, 128, 4064, 32, 4, True, "mxfp4"),
    (128, 128, 1152, 128, 16, False, "mxfp4")])
def test_longest_slices(T, d, F, E, k, gated, weights, active):
    print(T, d, F, E, k, gated, weights, active, flush=True)
    layer, x, wr, ws = make(T, d, F, E, k, gated, weights, active=active)
    out = layer.forward(x, wr, *ws, return_routing=True)
    check(layer, x, wr, ws, out)
    assert torch.equal(layer.forward(x, wr, *ws), out[0])


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,E,k,n", [
    # a single token routed by the hidden kernel and by its own; a unit for each
    # pair of fewer tokens than the call's, and of none
    (1, 8, 2, 0), (1, 8, 2, 1), (1, 130, 3, 0), (1, 130, 3, 1), (4, 64, 6, 0), (4, 64, 6, 1),
    (4, 64, 6, 3), (5, 200, 32, 2)])
def test_padded_batch_of_few_tokens(T, E, k, n, weights):
    layer, x, wr, ws = make(T, 256, 96, E, k, True, weights)
    x[n:] = float("nan")
    y = torch.full((T, 256), 7.0, device="cuda")
    ids = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    probs = torch.full((T, k), 5.0, device="cuda")
    nt = torch.tensor([n], dtype=torch.int32, device="cuda")
    layer.forward(x, wr, *ws, y=y, n_tokens=nt, routing=(ids, probs))
    assert (y[n:] == 7).all() and (ids[n:] == -9).all() and (probs[n:] == 5).all()
    if n:
        check(layer, x[:n], wr, ws, (y[:n], ids[:n], probs[:n]))
