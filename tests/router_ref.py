"""The router in 64 bits, token by token, from its definition; shares no code with the library."""

import numpy as np

U32 = 2.0 ** -24


def clean(l):
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    return np.minimum(l, float(np.finfo(np.float32).max))


def scores(l, kind):
    """[T, E] scores; 0 where masked."""
    l = clean(l)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return np.where(l == -np.inf, 0.0, np.where(l > 0, 1 / (1 + np.exp(-l)), np.exp(np.minimum(l, 0)) / (1 + np.exp(np.minimum(l, 0)))))
        top = l.max(1, keepdims=True)
        e = np.where(l == -np.inf, 0.0, np.exp(l - np.where(np.isfinite(top), top, 0)))
        s = e.sum(1, keepdims=True)
        return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def choose(l, bias, kind, K, groups=1, top_groups=1):
    l = clean(l)
    s = scores(l, kind)
    T, E = l.shape
    if bias is None and (groups == 1 or groups == top_groups):
        key = l.copy()                                   # the logits' order is the scores'
    else:
        key = s if bias is None else s + bias.astype(np.float64)
        key = np.where((l == -np.inf) | np.isnan(key), -np.inf, key)
    out = np.zeros((T, K), dtype=np.int32)
    gs = E // groups
    for t in range(T):
        live = range(E)
        if groups > 1:
            total = []
            for g in range(groups):
                two = sorted((k for k in key[t, g * gs:(g + 1) * gs] if k > -np.inf), reverse=True)[:2]
                total.append(sum(two) if two else -np.inf)
            best = sorted(range(groups), key=lambda g: (-total[g], g))[:top_groups]
            live = [e for e in range(E) if e // gs in best]
        out[t] = sorted(live, key=lambda e: (-key[t, e], e))[:K]
    return out


def spread(l, ids):
    """How far the exponentials' arguments reach: their rounding counts that often."""
    x = np.take_along_axis(clean(l), ids, 1)
    x = np.where(np.isfinite(x), x, np.nan)
    with np.errstate(all="ignore"):
        s = np.nanmax(np.abs(x), 1, keepdims=True, initial=0) * 2
    return np.minimum(np.nan_to_num(s), 220.0)


def weights(l, ids, kind, normalize, scale):
    """(weights, bound): each score is an exponential (2 ulp, of an argument rounded once), a sum of up to E terms
    or one more exponential, and three roundings; a sum over K of them, one division and two products."""
    s = np.take_along_axis(scores(l, kind), ids, 1)
    if normalize:
        x = np.take_along_axis(clean(l), ids, 1)
        # of the ratios, where the scores themselves are too small for 64 bits
        z = np.minimum(x, 0) if kind == "sigmoid" else x
        with np.errstate(all="ignore"):
            m = z.max(1, keepdims=True)
            a = np.exp(z - np.where(np.isfinite(m), m, 0)) / (1 + np.exp(-np.abs(x)) if kind == "sigmoid" else 1.0)
        a = np.where(x == -np.inf, 0.0, a)
        t = a.sum(1, keepdims=True)
        s = np.divide(a, t, out=np.zeros_like(a), where=t > 0)
    w = scale * s
    return w, (16 + l.shape[1] + 2 * ids.shape[1] + 2 * spread(l, ids)) * U32 * np.abs(w) + abs(scale) * 2.0 ** -125


def gradient(l, ids, g_w, kind, normalize, scale):
    """(gradient [T, E], bound) of the logits; every sum's terms count by their magnitudes."""
    T, E = l.shape
    s = scores(l, kind)
    lc = clean(l)
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        k = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        i = ids[t, k]
        g = scale * g_w[t, k].astype(np.float64) * (lc[t, i] > -np.inf)
        p = s[t, i]
        if normalize:
            p = weights(l[t:t + 1], i[None], kind, True, 1.0)[0][0] if len(k) else p
        dot, mdot = (g * p).sum(), (np.abs(g) * p).sum()
        if kind == "sigmoid" and not normalize:
            dot = mdot = 0.0
        one = (1 - p) if kind == "sigmoid" and not normalize else (1 - s[t, i]) if kind == "sigmoid" else np.ones(len(k))
        if kind == "sigmoid":
            x = lc[t, i]
            with np.errstate(over="ignore"):
                one = np.where(x > 0, np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))), 1 / (1 + np.exp(-np.abs(x))))
        if kind == "softmax" and not normalize:
            out[t] -= s[t] * dot
            mag[t] += s[t] * mdot
            np.add.at(out[t], i, p * g)
            np.add.at(mag[t], i, p * np.abs(g))
        else:
            np.add.at(out[t], i, p * (g - dot) * one)
            np.add.at(mag[t], i, p * (np.abs(g) + mdot) * one)
    n = 32 + 2 * E + 4 * ids.shape[1]
    sp = spread(l, np.where((ids >= 0) & (ids < E), ids, 0))
    if kind == "softmax" and not normalize:
        sp = np.maximum(sp, spread(l, np.tile(np.arange(E), (T, 1))))
    return out, (n + 4 * sp) * U32 * mag + 2.0 ** -120
