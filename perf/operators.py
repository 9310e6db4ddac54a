"""What the measurement of the 4-bit and expert operators runs.

Three operators of the library:

``quantize``   values to microscaled 4-bit floating point (MXFP4: elements
               of 1 sign, 2 exponent and 1 mantissa bit, one power-of-two
               scale for every 32 of them along the contracted axis) and
               back to the values the codes stand for;
``matmul``     the product of two MXFP4 matrices, out = a b^T;
``moe``        a whole mixture-of-experts layer for a few tokens: router,
               top-k selection, the selected ReLU experts, their weighted
               sum; expert weights in bfloat16 or MXFP4.

``run`` computes them in elementary torch operations where ``own`` is
false, and through the library's public entry points where it is true.
``exact`` is each operator's definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 32                      # elements that share one MXFP4 scale


# ---------------------------------------------------------------- cases

def _quantize(name, rows, cols, dtype, transposed):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "dtype": dtype,
            "transposed": transposed}


def _matmul(name, M, N, K, out):
    return {"name": name, "op": "matmul", "M": M, "N": N, "K": K, "out": out}


def _moe(name, T, d, F, E, k, gated, weights, active, normalize):
    return {"name": name, "op": "moe", "T": T, "d": d, "F": F, "E": E, "k": k, "gated": gated,
            "weights": weights, "active": active, "normalize": normalize}


def listed():
    return [
        # the activations of one decoding step of eight sequences
        _quantize("quantize_decode", 8, 2048, "bf16", False),
        # odd sizes: a block that the row's end cuts, rows that no vector load divides
        _quantize("quantize_ragged", 777, 1003, "f32", False),
        # a prompt batch's activations
        _quantize("quantize_prompt", 8192, 2048, "bf16", False),
        # W_down as it is stored, [F, d], contracted over F: the other axis
        _quantize("quantize_w_down", 5632, 2048, "f32", True),
        # gate pre-activations of one token
        _matmul("matmul_decode", 1, 5632, 2048, "f32"),
        # odd sizes in every direction
        _matmul("matmul_ragged", 333, 1003, 1999, "f32"),
        # the down projection of a short prompt
        _matmul("matmul_short", 512, 2048, 5632, "bf16"),
        # the gate pre-activations of a prompt batch, float32 for the TwELL pack
        _matmul("matmul_prompt", 8192, 5632, 2048, "f32"),
        # one token, fine-grained experts, no L1 penalty on the activations
        # (911 of 5632 neurons active)
        _moe("moe_token", 1, 2048, 1408, 64, 6, True, "bf16", 0.16, True),
        # a small non-gated layer of odd sizes, as in a draft model
        _moe("moe_odd", 13, 640, 352, 10, 3, False, "mxfp4", 0.5, False),
        # a decoding batch over 4-bit experts
        _moe("moe_decode_mxfp4", 32, 2048, 1408, 64, 6, True, "mxfp4", 0.16, True),
        # the layer's full-size experts, trained with an L1 penalty (29 of
        # 5632 active), one decoding batch
        _moe("moe_batch", 64, 2048, 5632, 16, 2, True, "bf16", 0.005, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "moe", "moe"])
    if op == "quantize":
        while True:
            r, c = _log(rng, 1, 16384), _log(rng, 1, 8192)
            if r * c <= 8192 * 2048:
                break
        return {k: v for k, v in _quantize("", r, c, rng.choice(["bf16", "f32"]),
                                           rng.random() < 0.4).items() if k != "name"}
    if op == "matmul":
        while True:
            M, N, K = _log(rng, 1, 8192), _log(rng, 1, 16384), _log(rng, 1, 16384)
            if M * N * K <= 8192 * 5632 * 2048 and M * N <= 8192 * 5632:
                break
        return {k: v for k, v in _matmul("", M, N, K, rng.choice(["bf16", "f32"])).items()
                if k != "name"}
    while True:
        d, F = 128 * _log(rng, 1, 32), 32 * _log(rng, 1, 176)
        E = _log(rng, 1, 128)
        if d * F * E <= 2048 * 5632 * 16:
            break
    k = rng.randint(1, min(E, 8))
    return {k_: v for k_, v in _moe("", _log(rng, 1, 128), d, F, E, k, rng.random() < 0.7,
                                    rng.choice(["bf16", "mxfp4"]),
                                    rng.choice([0.005, 0.02, 0.16, 0.5]),
                                    rng.random() < 0.5).items() if k_ != "name"}


# ---------------------------------------------------------------- work

def _mx_bytes(rows, cols):
    return rows * cols / 2 + rows * math.ceil(cols / BLOCK)


def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        e = 2 if case["dtype"] == "bf16" else 4
        # the input, the codes and scales written and read, the values
        mx = (_mx_bytes(case["cols"], case["rows"]) if case["transposed"]
              else _mx_bytes(case["rows"], case["cols"]))
        return {"bytes": 2 * n * e + 2 * mx, "flops": 4 * n}
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": _mx_bytes(M, K) + _mx_bytes(N, K) + M * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    T, d, F, E, k, a = (case[x] for x in ("T", "d", "F", "E", "k", "active"))
    pairs = T * k
    # experts that some token selects, and neurons that are active for some
    # token of theirs, in expectation; every selected expert's gate is read
    # in whole, up and down only for active neurons
    touched = E * (1 - (1 - k / E) ** T)
    union = 1 - (1 - a) ** (pairs / touched)
    wb = 2 if case["weights"] == "bf16" else 17 / 32
    rest = 2 if case["gated"] else 1
    return {"bytes": touched * F * d * wb * (1 + rest * union) + E * d * 2 + T * d * (2 + 4)
            + T * k * 8,
            "flops": 2 * T * E * d + 2 * pairs * d * F * (1 + rest * a)}


# ---------------------------------------------------------------- inputs

def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + salt)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def _quantize_plain(x):
    """x [R, K] -> (signed multiples of the block scale [R, K], scale
    exponents [R, ceil(K / 32)]): the exponent of the block's largest
    magnitude less 2 (the exponent of the largest element, 6 = 1.5 * 4), to
    the nearest element, ties to the even code, saturating at 6."""
    R, K = x.shape
    nb = (K + BLOCK - 1) // BLOCK
    xp = torch.zeros(R, nb * BLOCK, device=x.device, dtype=torch.float32)
    xp[:, :K] = x
    xb = xp.view(R, nb, BLOCK)
    amax = xb.abs().amax(dim=2)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, torch.full_like(amax, -127).int())
    e = e.clamp(-127, 127)
    v = torch.ldexp(xb, -e[:, :, None])
    a = v.abs()
    step = 0.5 + 0.5 * (a >= 2) + 1.0 * (a >= 4)
    q = torch.clamp(torch.round(a / step) * step, max=6.0)
    q = torch.where(v < 0, -q, q)
    return q.view(R, nb * BLOCK)[:, :K].contiguous(), e


def _packed_plain(x):
    # the multiples are small: bfloat16 holds them
    q, e = _quantize_plain(x)
    return q.to(torch.bfloat16), e


def _values_plain(q, e):
    R, K = q.shape
    s = e.repeat_interleave(BLOCK, dim=1)[:, :K]
    return torch.ldexp(q, s)


def _expert_weights(case, seed):
    """w_gate, w_up (or None), w_down, each [E, F, d] bfloat16 in the
    library's neuron-major layout. Column 0 of the gate meets an input that
    is always 1 and sets the fraction of active neurons."""
    d, F, E, a = case["d"], case["F"], case["E"], case["active"]
    tau = math.sqrt((d - 1) / d) * math.sqrt(2) * float(torch.erfinv(torch.tensor(1 - 2 * a,
                                                                                  dtype=torch.float64)))
    out = []
    for salt, scale, used in ((11, d, True), (12, d, case["gated"]), (13, F, True)):
        if not used:
            out.append(None)
            continue
        g = _gen(seed, salt)
        w = torch.empty(E, F, d, device=DEV, dtype=torch.bfloat16)
        for i in range(E):
            w[i] = _randn(g, F, d) / math.sqrt(scale)
        if salt == 11:
            w[:, :, 0] = -tau
        out.append(w)
    return out


def prepare(case, seed):
    g = _gen(seed, 1)
    st = {"case": case}
    if own:
        import unstructured_sparse_feedforward_amd as sffn
    if case["op"] == "quantize":
        x = _randn(g, case["rows"], case["cols"])
        # a few large entries, as activations have
        x = x * (1 + 15 * (torch.rand(x.shape, generator=g, device=DEV) < 0.002))
        st["x"] = x.to(_TORCH[case["dtype"]])
    elif case["op"] == "matmul":
        for key, rows in (("a", case["M"]), ("b", case["N"])):
            x = _randn(g, rows, case["K"])
            if key == "b":
                x = x / math.sqrt(case["K"])
            st[key] = sffn.mx_quantize(x) if own else _quantize_plain(x)
    else:
        x = _randn(g, case["T"], case["d"])
        x[:, 0] = 1.0
        st["x"] = x.to(torch.bfloat16)
        st["router"] = (_randn(g, case["E"], case["d"]) / math.sqrt(case["d"])).to(torch.bfloat16)
        ws = _expert_weights(case, seed)
        if case["weights"] == "mxfp4":
            E, F, d = case["E"], case["F"], case["d"]
            if own:
                ws = [w if w is None else sffn.mx_quantize(w.view(E * F, d)) for w in ws]
            else:
                # one expert at a time: the float32 copies stay small
                ws = [w if w is None else [_packed_plain(w[i]) for i in range(E)] for w in ws]
        st["weights"] = ws
        if own:
            st["layer"] = sffn.SparseMoE(case["d"], case["F"], case["E"], case["k"],
                                         gated=case["gated"], normalize=case["normalize"],
                                         weights=case["weights"])
    return st


# ---------------------------------------------------------------- run

def _weight32(w, i):
    if isinstance(w, list):
        q, e = w[i]
        return _values_plain(q.float(), e)
    return w[i].float()


def _moe_plain(st):
    case = st["case"]
    x, k = st["x"].float(), case["k"]
    # 64 bits: two experts' logits may lie closer than 32 bits resolve
    logits = st["router"].double() @ st["x"].double().t()
    logits = logits.t().contiguous()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = ids[:, :k]
    p = torch.exp(top - top[:, :1])
    total = (p[:, :k] if case["normalize"] else p).sum(dim=1, keepdim=True)
    p = (p[:, :k] / total).float()
    dense = torch.zeros(x.shape[0], case["E"], device=x.device)
    dense.scatter_(1, ids, p)
    y = torch.zeros_like(x)
    wg, wu, wd = st["weights"]
    for i in range(case["E"]):
        z = x @ _weight32(wg, i).t()
        h = torch.where(z > 0, z, torch.zeros_like(z))
        if wu is not None:
            h = h * (x @ _weight32(wu, i).t())
        y += dense[:, i:i + 1] * (h @ _weight32(wd, i))
    return y, ids.int(), p


def run(state):
    case = state["case"]
    if own:
        import unstructured_sparse_feedforward_amd as sffn
        if case["op"] == "quantize":
            q = sffn.mx_quantize(state["x"], transposed=case["transposed"])
            return sffn.mx_dequantize(q, dtype=state["x"].dtype)
        if case["op"] == "matmul":
            return sffn.mx_matmul(state["a"], state["b"], dtype=_TORCH[case["out"]])
        return state["layer"].forward(state["x"], state["router"], *state["weights"],
                                      return_routing=True)
    if case["op"] == "quantize":
        x = state["x"].t() if case["transposed"] else state["x"]
        return _values_plain(*_quantize_plain(x)).to(state["x"].dtype)
    if case["op"] == "matmul":
        a, b = _values_plain(*state["a"]), _values_plain(*state["b"])
        return (a @ b.t()).to(_TORCH[case["out"]])
    return _moe_plain(state)


# ---------------------------------------------------------------- exact

_E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _exact_values(x):
    """The MXFP4 values of x [R, K] (64-bit tensor): for each block the
    scale from the logarithm of its largest magnitude, then the nearest of
    the eight magnitudes by distance, of two at the same distance the one
    with the even code."""
    grid = torch.from_numpy(_E2M1).to(x.device)
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=x.device)    # even codes first
    out = torch.empty_like(x)
    for k0 in range(0, x.shape[1], BLOCK):
        b = x[:, k0:k0 + BLOCK]
        amax = b.abs().max(dim=1, keepdim=True).values
        safe = torch.where(amax > 0, amax, torch.ones_like(amax))
        e = torch.floor(torch.log2(safe))
        # the logarithm may round up to a whole number just below it
        e = torch.where(torch.exp2(e) > safe, e - 1, e)
        e = torch.where(torch.exp2(e + 1) <= safe, e + 1, e) - 2
        s = torch.exp2(e.clamp(-127, 127))
        dist = ((b.abs() / s)[:, :, None] - grid[order]).abs()
        out[:, k0:k0 + BLOCK] = torch.sign(b) * grid[order[dist.argmin(dim=2)]] * s
    return out


def _exact_weight(w, i, packed):
    w = w[i].double()
    return _exact_values(w) if packed else w


def exact(case, seed):
    global own
    was, own = own, False
    try:
        if case["op"] != "moe":
            g = _gen(seed, 1)
            if case["op"] == "quantize":
                x = prepare(case, seed)["x"].double()
                return _exact_values(x.t().contiguous() if case["transposed"] else x)
            v = {}
            for key, rows in (("a", case["M"]), ("b", case["N"])):
                x = _randn(g, rows, case["K"])
                v[key] = _exact_values((x / math.sqrt(case["K"]) if key == "b" else x).double())
            return v["a"] @ v["b"].t()
        st = prepare(dict(case, weights="bf16"), seed)
        packed = case["weights"] == "mxfp4"
    finally:
        own = was
    x, wr = st["x"].double(), st["router"].double()
    T, E, k = case["T"], case["E"], case["k"]
    logits = (x[:, None, :] * wr[None, :, :]).sum(dim=2).cpu().numpy() if T * E * case["d"] < 1 << 27 \
        else (x @ wr.t()).cpu().numpy()
    ids = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -logits), axis=1)[:, :k]
    chosen = np.take_along_axis(logits, ids, 1)
    m = logits.max(axis=1, keepdims=True)
    p = np.exp(chosen - m) / (np.exp(chosen - m) if case["normalize"]
                              else np.exp(logits - m)).sum(axis=1, keepdims=True)
    y = torch.zeros(T, case["d"], device=DEV, dtype=torch.float64)
    for i in np.unique(ids):
        t, r = np.nonzero(ids == i)
        rows = torch.from_numpy(t).to(DEV)
        wg, wu, wd = st["weights"]
        z = x[rows] @ _exact_weight(wg, i, packed).t()
        h = z.clamp_min(0)
        if wu is not None:
            h = h * (x[rows] @ _exact_weight(wu, i, packed).t())
        h = h * torch.from_numpy(p[t, r]).to(DEV)[:, None]
        y.index_add_(0, rows, h @ _exact_weight(wd, i, packed))
    return y, torch.from_numpy(ids.astype(np.int32)), torch.from_numpy(p)
