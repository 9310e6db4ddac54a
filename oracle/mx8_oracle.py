"""MXFP8 in float64 numpy, from its definition (the OCP Microscaling format
with e4m3 elements and e8m0 scales): scalar loops over blocks, nearest
element by distance. Shares no code with the library."""
import math

import numpy as np

BLOCK = 32


def e4m3(c):
    """The value of a code 0 .. 255 (NaN for 0x7F and 0xFF)."""
    s, e, m = c >> 7, (c >> 3) & 15, c & 7
    if e == 15 and m == 7:
        return math.nan
    v = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
    return -v if s else v


GRID = np.array([e4m3(c) for c in range(127)])


def nearest_code(v):
    """Code 0 .. 126 of the magnitude nearest to v >= 0; of two at the same
    distance the even code; 448 for everything above."""
    d = np.abs(GRID - v)
    near = np.flatnonzero(d == d.min())
    return int(near[0] if len(near) == 1 else next(c for c in near if c % 2 == 0))


def quantize(x):
    """x [R, K] -> (codes [R, K], exponents [R, ceil(K / 32)], 128 for a block
    with an infinity or a NaN, whose codes are 0)."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    codes = np.zeros((R, K), np.uint8)
    exps = np.zeros((R, -(-K // BLOCK)), np.int64)
    for r in range(R):
        for i in range(exps.shape[1]):
            b = x[r, i * BLOCK:(i + 1) * BLOCK]
            if not np.isfinite(b).all():
                exps[r, i] = 128
                continue
            m = float(np.abs(b).max())
            e = -127 if m == 0 else min(max(math.frexp(m)[1] - 1 - 8, -127), 127)
            exps[r, i] = e
            for j, v in enumerate(b):
                c = nearest_code(abs(v) * 2.0 ** -e)
                codes[r, i * BLOCK + j] = c | (128 if math.copysign(1.0, v) < 0 else 0)
    return codes, exps


def values(codes, exps):
    """The float64 values of codes [R, K] with exponents [R, blocks]."""
    v = np.array([e4m3(c) for c in range(256)])[codes]
    e = np.repeat(exps, BLOCK, axis=1)[:, :codes.shape[1]]
    return np.where(e == 128, np.nan, v * 2.0 ** np.where(e == 128, 0, e).astype(np.float64))


def pack(codes, exps):
    """The library's layout: (codes [R, Kp], scales [Kp / 128, R, 4])."""
    R, K = codes.shape
    Kp = -(-K // 128) * 128
    c = np.zeros((R, Kp), np.uint8)
    c[:, :K] = codes
    s = np.zeros((R, Kp // 32), np.uint8)
    s[:, :exps.shape[1]] = exps + 127
    return c, np.ascontiguousarray(s.reshape(R, Kp // 128, 4).transpose(1, 0, 2))


def unpack(codes, scales, K):
    """The inverse of pack."""
    s = scales.transpose(1, 0, 2).reshape(codes.shape[0], -1).astype(np.int64) - 127
    return codes[:, :K], s[:, :-(-K // BLOCK)]
