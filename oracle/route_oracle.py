"""The choice of experts and its gradient in float64, token by token, from the
definition. Shares no code with the library."""
import math

import numpy as np


def _scores(l, sigmoid):
    if sigmoid:
        return [1 / (1 + math.exp(-v)) if v >= 0 else math.exp(v) / (1 + math.exp(v)) for v in l]
    m = max(l)
    if m == -math.inf:
        return [0.0] * len(l)
    e = [math.exp(v - m) for v in l]
    z = math.fsum(e)
    return [v / z for v in e]


def choose(l, k, sigmoid=False, bias=None, groups=1, top_groups=1, group_best=1):
    """The ids of one token's experts, and all scores."""
    E = len(l)
    l = [float(v) for v in l]
    s = _scores(l, sigmoid)
    c = s if bias is None else [a + float(b) for a, b in zip(s, bias)]
    key = l if bias is None else c
    per = E // groups
    allowed = range(E)
    if top_groups < groups:
        score = [sum(sorted(c[g * per:(g + 1) * per], reverse=True)[:group_best])
                 for g in range(groups)]
        kept = sorted(range(groups), key=lambda g: (-score[g], g))[:top_groups]
        allowed = [e for e in range(E) if e // per in kept]
    return sorted(allowed, key=lambda e: (-key[e], e))[:k], s


def forward(logits, k, sigmoid=False, bias=None, groups=1, top_groups=1, group_best=1,
            normalize=True, scale=1.0):
    ids, probs = [], []
    for l in np.asarray(logits, np.float64):
        i, s = choose(l, k, sigmoid, bias, groups, top_groups, group_best)
        probs.append(weights(l, i, sigmoid, normalize, scale))
        ids.append(i)
    return np.array(ids, np.int32).reshape(-1, k), np.array(probs).reshape(-1, k)


def weights(l, ids, sigmoid, normalize, scale):
    """The weights of one token's chosen experts, as a function of its
    logits."""
    l = [float(v) for v in l]
    if normalize and not sigmoid:
        p = _scores([l[e] for e in ids], False)
    else:
        s = _scores(l, sigmoid)
        p = [s[e] for e in ids]
        if normalize:
            z = math.fsum(p)
            p = [v / z if z else 0.0 for v in p]
    return [scale * v for v in p]


def backward(dprobs, logits, ids, sigmoid, normalize, scale):
    """dlogits by the Jacobian of each token's weights, element by element."""
    out = np.zeros(np.shape(logits))
    for t, l in enumerate(np.asarray(logits, np.float64)):
        s = _scores([float(v) for v in l], sigmoid)
        E = len(l)
        # J[j][e] = d s_j / d l_e
        if sigmoid:
            J = np.diag([v * (1 - v) for v in s])
        else:
            J = np.diag(s) - np.outer(s, s)
        c = [e for e in ids[t] if 0 <= e < E]
        d = [dprobs[t][r] for r, e in enumerate(ids[t]) if 0 <= e < E]
        z = math.fsum(s[e] for e in c)
        for i, (e, g) in enumerate(zip(c, d)):
            if not normalize:
                out[t] += scale * g * J[e]
            elif z:
                out[t] += scale * g * (J[e] / z - s[e] / z ** 2 * sum(J[q] for q in c))
    return out
