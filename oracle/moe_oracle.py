"""The expert layer in float64 numpy, token by token and expert by expert,
and a bound on what a float32 evaluation of it may differ by."""
import numpy as np


def route(x, w_router, k, normalize):
    """ids [T, k] in descending order of the logits (ties: the lower expert
    first) and the softmax weights [T, k]."""
    T, E = x.shape[0], w_router.shape[0]
    ids = np.zeros((T, k), np.int64)
    probs = np.zeros((T, k))
    for t in range(T):
        l = w_router @ x[t]
        order = sorted(range(E), key=lambda e: (-l[e], e))
        ids[t] = order[:k]
        ex = np.exp(l - l.max())
        probs[t] = ex[ids[t]] / (ex[ids[t]].sum() if normalize else ex.sum())
    return ids, probs


def forward(x, w_router, w_gate, w_up, w_down, k, normalize=True):
    """x [T, d], w_router [E, d], w_gate, w_up (or None), w_down [E, F, d].
    Returns (y, ids, probs, bound): |y' - y| <= bound for a y' with
    float32 sums in any order (d, then F, then k terms and at most F / 32
    partial sums; a sum of n terms errs by at most n 2^-23 of the sum of
    magnitudes, truncating adders included) and h rounded to 2^-23 of
    itself (the product of z and u, and its sum of three bf16 parts, each
    to half a step of 24 bits). The bound on h covers a z whose sign the rounding flips."""
    ids, probs = route(x, w_router, k, normalize)
    T, d = x.shape
    F = w_gate.shape[1]
    y, bound = np.zeros((T, d)), np.zeros((T, d))
    eps = 2.0 ** -23
    for t in range(T):
        for r in range(k):
            e = ids[t, r]
            z = w_gate[e] @ x[t]
            dz = d * eps * (np.abs(w_gate[e]) @ np.abs(x[t]))
            a = np.where(z > 0, z, 0.0)
            if w_up is None:
                u, du = np.ones(F), np.zeros(F)
            else:
                u = w_up[e] @ x[t]
                du = d * eps * (np.abs(w_up[e]) @ np.abs(x[t]))
            h = a * u
            dh = a * du + (np.abs(u) + du) * dz + eps * np.abs(h)
            y[t] += probs[t, r] * (h @ w_down[e])
            mag = (np.abs(h) + dh) @ np.abs(w_down[e])
            # the weights' exponential and quotient: a few units of 2^-23
            bound[t] += probs[t, r] * (dh @ np.abs(w_down[e])
                                       + (F + k * (F // 32) + 64) * eps * mag)
    return y, ids, probs, bound
