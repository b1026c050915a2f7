"""Plain 64-bit forms of the int8 products and the expert operators, on numpy
arrays, for the tests."""
import math

import numpy as np

MAX = np.finfo(np.float64).max


def quantize(x):
    """(codes, fp32 scales) of fp32 rows.  The quotient of two fp32 values is
    either exactly halfway between two integers below 128 or further than
    2^-33 (relative) from it, so a float64 quotient rounds as the real one."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(1)
    s = (amax.astype(np.float64) / 127.0).astype(np.float32)
    s = np.where(amax > 0, np.maximum(s, np.float32(2.0 ** -126)), np.float32(0.0))
    bad = ~np.isfinite(x).all(1)
    with np.errstate(all="ignore"):
        q = np.rint(x.astype(np.float64) / s.astype(np.float64)[:, None])
    q = np.where((bad | (amax == 0))[:, None], 0.0, q)
    return q.astype(np.int8), np.where(bad, np.float32(np.nan), s).astype(np.float32)


def erfc(x):
    return np.vectorize(math.erfc)(x)


def product(a, a_s, b, b_s, bias=None, act=False):
    """(result, tolerance of the fp32 evaluation) in float64.

    The integer sum is rounded to fp32 once and multiplied twice: at most
    3 * 2^-24 of the product p; the bias adds one rounding of y.  GELU is
    y/2 (1 + erf(y / sqrt 2)) with an erf good to 1.5e-7 plus at most 12
    roundings of values of at most 1, so its own error is at most
    |y|/2 (1.5e-7 + 12 * 2^-24) and one rounding; its slope is below 1.13."""
    u = 2.0 ** -24
    p = (a.astype(np.float64) @ b.astype(np.float64).T) * a_s.astype(np.float64)[:, None] * b_s.astype(np.float64)[None, :]
    tol = 3.01 * u * np.abs(p)
    y = p
    if bias is not None:
        y = y + bias.astype(np.float64)[None, :]
        tol = tol + 1.01 * u * np.abs(y)
    if act:
        g = 0.5 * y * erfc(-y / math.sqrt(2.0))
        tol = 1.13 * tol + 0.5 * np.abs(y) * (1.5e-7 + 12 * u) + 2.01 * u * np.abs(g)
        y = g
    return y, tol


def half_step(dtype):
    import torch

    return torch.finfo(dtype).eps / 2


def scores(x, score):
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        if score == "softmax":
            m = x.max(-1, keepdims=True)
            e = np.exp(x - np.where(m == -np.inf, 0.0, m))
            return e / e.sum(-1, keepdims=True)
        return 1.0 / (1.0 + np.exp(-x))


def route(logits, k, score, bias=None, groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0):
    """ids, weights by the definition, one token at a time."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    ids = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k))
    per = E // groups
    for t in range(T):
        s = scores(x[t], score)
        out = x[t] == -np.inf
        nan_row = score == "softmax" and (np.isnan(x[t]).any() or x[t].max() == np.inf)
        # where the score is the whole key, the logit orders alike and does not saturate
        key = x[t].copy() if bias is None and group_top == 1 else s + (0 if bias is None else np.asarray(bias, np.float64))
        if nan_row:
            key[:] = np.nan
        key = np.where(np.isnan(key), -MAX, key)
        key[out] = -np.inf
        if groups > 1:
            g = np.full(groups, -np.inf)
            for i in range(groups):
                best = sorted(key[i * per:(i + 1) * per], reverse=True)[:group_top]
                best = [b for b in best if b > -np.inf]
                if best:
                    with np.errstate(over="ignore"):
                        g[i] = max(float(np.sum(best)), -MAX)
            kept = sorted(range(groups), key=lambda i: (-g[i], i))[:top_groups]
            for i in range(groups):
                if i not in kept:
                    key[i * per:(i + 1) * per] = -np.inf
        chosen = [e for e in sorted(range(E), key=lambda e: (-key[e], e)) if key[e] > -np.inf][:k]
        w = chosen_weights(x[t], chosen, score, renormalize, scale)
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = np.nan if nan_row else w
    return ids, weights


def chosen_weights(x, chosen, score, renormalize, scale):
    if not chosen:
        return np.zeros(0)
    l = x[chosen]
    with np.errstate(all="ignore"):
        if not renormalize:
            return scale * scores(x, score)[chosen]
        # logarithms of the scores up to a constant: the ratio survives underflow
        ls = l if score == "softmax" else np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))
        p = np.exp(ls - ls.max())
        return scale * p / p.sum()


def route_backward(logits, ids, dw, score, renormalize=True, scale=1.0):
    """(gradient, magnitude of the terms it is a sum of)."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        at = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        if not at:
            continue
        c = ids[t, at]
        g = np.asarray(dw[t], np.float64)[at] * scale
        s = scores(x[t], score)
        if renormalize:
            w = chosen_weights(x[t], list(c), score, True, 1.0)
            own = w * (g - (w * g).sum())
            big = w * (np.abs(g) + (w * np.abs(g)).sum())
            if score == "sigmoid":
                own, big = own * scores(-x[t][c], score), big * scores(-x[t][c], score)
        elif score == "softmax":
            dot, adot = (g * s[c]).sum(), (np.abs(g) * s[c]).sum()
            d[t], mag[t] = -s * dot, s * adot
            own, big = g * s[c], np.abs(g) * s[c]
        else:
            own = g * s[c] * scores(-x[t][c], score)
            big = np.abs(own)
        np.add.at(d[t], c, own)
        np.add.at(mag[t], c, big)
    return d, mag


def plan(ids, experts):
    flat = np.asarray(ids).reshape(-1)
    order = np.full(flat.size, -1, np.int32)
    position = np.full(flat.size, -1, np.int32)
    offsets = np.zeros(experts + 1, np.int32)
    p = 0
    for e in range(experts):
        offsets[e] = p
        at = np.nonzero(flat == e)[0]
        order[p:p + at.size] = at
        position[at] = np.arange(p, p + at.size)
        p += at.size
    offsets[experts] = p
    return offsets, order, position.reshape(np.asarray(ids).shape)
