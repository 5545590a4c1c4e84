"""Plain top-k routing in 64 bits (numpy, one token at a time): the definition that
the CUDA router is compared with.  Shares no code with it."""
from __future__ import annotations

import numpy as np


def scores64(z, kind):
    """Scores of one token's logits (fp64, -inf: score 0)."""
    if kind == "sigmoid":
        return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
    live = z > -np.inf
    s = np.zeros_like(z)
    if live.any():
        e = np.exp(z[live] - z[live].max())
        s[live] = e / e.sum()
    return s


def clean(logits):
    """Logits as the router reads them: NaN counts as -inf, +inf as the largest fp32 value."""
    z = np.asarray(logits, np.float64).copy()
    z[np.isnan(z)] = -np.inf
    return np.minimum(z, float(np.finfo(np.float32).max))


def choose(z, k, kind, bias, n_group, topk_group):
    """Chosen experts of one token, best first (shorter than k where too few can be chosen)."""
    E = len(z)
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    with np.errstate(invalid="ignore"):
        c = scores64(z, kind) + b
    ok = (z > -np.inf) & ~np.isnan(b) & (b > -np.inf)
    if bias is None and n_group == 1:
        c = z
    per = E // n_group
    if topk_group < n_group:
        values = []
        for g in range(n_group):
            best = sorted((c[e] for e in range(g * per, (g + 1) * per) if ok[e]), reverse=True)[:2]
            values.append(sum(best) if best else -np.inf)
        kept = sorted(range(n_group), key=lambda g: (-values[g], g))[:topk_group]
        ok = ok & np.isin(np.arange(E) // per, kept)
    order = sorted((e for e in range(E) if ok[e]), key=lambda e: (-c[e], e))
    return order[:k]


def weights64(z, ids, kind, renorm, scale):
    """Weights of the chosen experts of one token, fp64."""
    if not len(ids):
        return np.zeros(0)
    zi = z[list(ids)]
    if renorm:
        # relative to the largest chosen logit, in logarithms: nothing underflows
        ls = zi if kind == "softmax" else -np.logaddexp(0, -zi)
        r = np.exp(ls - ls.max())
        return r / r.sum() * scale
    return scores64(z, kind)[list(ids)] * scale


def route(logits, k, kind="softmax", bias=None, n_group=1, topk_group=None, renorm=True, scale=1.0):
    """(gates [T, E], ids [T, k], weights [T, k]) in fp64."""
    T, E = logits.shape
    gates, ids, w = np.zeros((T, E)), -np.ones((T, k), np.int64), np.zeros((T, k))
    for t in range(T):
        z = clean(logits[t])
        got = choose(z, k, kind, bias, n_group, n_group if topk_group is None else topk_group)
        v = weights64(z, got, kind, renorm, scale)
        ids[t, : len(got)] = got
        w[t, : len(got)] = v
        gates[t, got] = v
    return gates, ids, w


def backward(logits, ids, d_weights, kind="softmax", renorm=True, scale=1.0):
    """(d_logits [T, E], the size of the terms that add up in each element), fp64."""
    T, E = logits.shape
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        z = clean(logits[t])
        at = [int(i) for i in ids[t]]
        s = scores64(z, kind)
        live = [i for i, e in enumerate(at) if 0 <= e < E and z[e] > -np.inf]
        if not live:
            continue
        e = np.array([at[i] for i in live])
        dw = np.asarray(d_weights[t], np.float64)[live] * scale
        if renorm:
            p = weights64(z, e, kind, True, 1.0)
            v, mag = p * (dw - (dw * p).sum()), p * (np.abs(dw) + (np.abs(dw) * p).sum())
            if kind == "sigmoid":
                v, mag = v * (1 - s[e]), mag * (1 - s[e])
            np.add.at(out[t], e, v)
            np.add.at(size[t], e, mag)
            continue
        ds, dabs = np.zeros(E), np.zeros(E)
        np.add.at(ds, e, dw)
        np.add.at(dabs, e, np.abs(dw))
        if kind == "sigmoid":
            out[t], size[t] = ds * s * (1 - s), dabs * s * (1 - s)
        else:
            out[t], size[t] = s * (ds - (dw * s[e]).sum()), s * (dabs + (np.abs(dw) * s[e]).sum())
    return out, size
