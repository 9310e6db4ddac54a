"""Inputs of the expert layer for which the results are known exactly, and
differ if the logits or h carry fewer bits than they are said to."""
import numpy as np


def hidden_24_bits(T, d, F, gated, seed=0):
    """x [T, d], gate, up (None), down [F, d] and y [T, d], all float64 and
    exact in bfloat16 (x and weights) and in MXFP4 (weights; every block's
    values lie within a factor of 8 of each other or are 0).

    x of token t is (a, b 2^-8, c 2^-16, 1, 0, ..) with whole a of 128 .. 255
    and b, c of 0 .. 255, c odd, so that z = x . s (1, 1, 1, 0, ..) = s v for a
    v of exactly 24 significant bits, in any order of summation. u, when
    gated, is a power of two, and a neuron's row of the down matrix is one
    power of two in a column of its own: y is h times that, without any
    rounding in float32. F <= d."""
    assert F <= d
    r = np.random.default_rng(seed)
    x = np.zeros((T, d))
    x[:, 0] = r.integers(128, 256, T)
    x[:, 1] = r.integers(0, 256, T) * 2.0 ** -8
    x[:, 2] = (r.integers(0, 128, T) * 2 + 1) * 2.0 ** -16
    x[:, 3] = 1.0
    s = 2.0 ** r.integers(-3, 4, F)
    gate, up, down = np.zeros((F, d)), np.zeros((F, d)), np.zeros((F, d))
    gate[:, :3] = s[:, None]
    up[:, 3] = 2.0 ** r.integers(-2, 3, F) * r.choice([-1.0, 1.0], F)
    col = r.permutation(d)[:F]
    down[np.arange(F), col] = 2.0 ** r.integers(-3, 4, F)
    h = x @ gate.T
    if gated:
        h = h * (x @ up.T)
    y = np.zeros((T, d))
    y[:, col] = h * down[np.arange(F), col]
    return x, gate, up if gated else None, down, y


def bf16(v):
    """float64 to the nearest bfloat16, ties to even (no NaN or overflow)."""
    b = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + (b >> 16 & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def near_tie(E, d):
    """Router rows [E, d] for an x of ones at columns 0 and d - 1 (0
    elsewhere), exact in bfloat16: the last expert's logit is 2^-40 above
    the second one's (the first's, if there are two), which a sum in 32 bits
    does not see; all others' are 0. ids of the two largest."""
    low, high = (1 if E > 2 else 0), E - 1
    w = np.zeros((E, d))
    w[[low, high], 0] = 1.0
    w[high, d - 1] = 2.0 ** -40
    return w, [high, low]
