"""MXFP4 in float64 numpy, from its definition (the OCP Microscaling
format with e2m1 elements and e8m0 scales): scalar loops over blocks,
nearest element by distance. Shares no code with the library."""
import math

import numpy as np

BLOCK = 32
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def nearest_code(v):
    """Code 0..7 of the magnitude nearest to v >= 0; of two at the same
    distance the even code; 6 for everything above."""
    best = min(abs(v - g) for g in GRID)
    near = [c for c, g in enumerate(GRID) if abs(v - g) == best]
    return near[0] if len(near) == 1 else next(c for c in near if c % 2 == 0)


def block_exponent(b):
    """Exponent of the block's scale; None for a block with inf or NaN."""
    b = np.asarray(b, np.float64)
    if not np.isfinite(b).all():
        return None
    m = float(np.abs(b).max()) if b.size else 0.0
    if m == 0.0:
        return -127
    return min(max(math.frexp(m)[1] - 1 - 2, -127), 127)


def quantize(x):
    """x [R, K] -> (codes [R, K] of 0..15 with the sign in bit 3, exponents
    [R, ceil(K / 32)], 128 for a NaN block)."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    nb = -(-K // BLOCK)
    codes = np.zeros((R, K), np.uint8)
    exps = np.zeros((R, nb), np.int64)
    for r in range(R):
        for i in range(nb):
            b = x[r, i * BLOCK:(i + 1) * BLOCK]
            e = block_exponent(b)
            if e is None:
                exps[r, i] = 128
                continue
            exps[r, i] = e
            for j, v in enumerate(b):
                c = nearest_code(abs(v) * 2.0 ** -e)
                codes[r, i * BLOCK + j] = c | (8 if math.copysign(1.0, v) < 0 else 0)
    return codes, exps


def values(codes, exps):
    """The float64 values of codes [R, K] with exponents [R, blocks]."""
    mag = np.asarray(GRID)[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    e = np.repeat(exps, BLOCK, axis=1)[:, :codes.shape[1]]
    return np.where(e == 128, np.nan, mag * 2.0 ** np.where(e == 128, 0, e).astype(np.float64))


def pack(codes, exps):
    """The library's layout: (codes [R, Kp / 2], scales [Kp / 128, R, 4]),
    the scale bytes of blocks past K as 0."""
    R, K = codes.shape
    Kp = -(-K // 128) * 128
    c = np.zeros((R, Kp), np.uint8)
    c[:, :K] = codes
    s = np.zeros((R, Kp // 32), np.uint8)
    s[:, :exps.shape[1]] = exps + 127
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8), np.ascontiguousarray(
        s.reshape(R, Kp // 128, 4).transpose(1, 0, 2))


def unpack(codes, scales, K):
    """The inverse of pack."""
    R = codes.shape[0]
    c = np.zeros((R, codes.shape[1] * 2), np.uint8)
    c[:, 0::2] = codes & 15
    c[:, 1::2] = codes >> 4
    s = scales.transpose(1, 0, 2).reshape(R, -1).astype(np.int64) - 127
    return c[:, :K], s[:, :-(-K // BLOCK)]
