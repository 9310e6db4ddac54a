"""The residual norm and its gradient in float64 numpy, from the formulas.
Shares no code with the library."""
import numpy as np


def forward(s, weight, eps):
    """(y, r) of the rows s [T, n]."""
    s = np.asarray(s, np.float64)
    r = 1 / np.sqrt((s * s).mean(axis=1) + eps)
    y = s * r[:, None]
    return (y if weight is None else y * np.asarray(weight, np.float64)), r


def backward(dy, s, weight, r, dstream=None):
    """(ds, dweight) by the chain rule, r [T] as given."""
    dy, s, r = (np.asarray(v, np.float64) for v in (dy, s, r))
    xh = s * r[:, None]
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    ds = r[:, None] * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    if dstream is not None:
        ds = ds + np.asarray(dstream, np.float64)
    return ds, (dy * xh).sum(axis=0)
