"""Routing by scores, and low-rank adapters, in float64 (oracle; test-only).

The pages give 384 experts with 8 active per token and no scoring rule; the
rules here are additions.  With l the logits and b a bias: s is the row's softmax
or the sigmoid of l, c = s + b.  An expert whose l or c is NaN or -inf is not
available.  A group (E / groups consecutive experts) is worth the sum of its
`best` largest available c; the `keep` groups worth most stay.  Of their
available experts the k of the largest c (of the largest l without a bias) are
taken; equal values go by the lower index.  Weights are s, or s over the sum of
the taken, times scale; a place that nothing is left for holds -1 and 0."""

import numpy as np


def scores(logits, sigmoid):
    """float64[T, E] of one row each; NaN and -inf count as no logit at all."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    with np.errstate(all="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-l))
        top = l.max(1, keepdims=True)
        p = np.where(l == top, 1.0, np.exp(l - top))
        p = np.where(l > -np.inf, p, 0.0)
        return np.where(p.sum(1, keepdims=True) > 0, p / p.sum(1, keepdims=True), 0.0)


def log_scores(l, sigmoid):
    """log s of float64 logits, up to a row's constant (softmax)."""
    with np.errstate(all="ignore"):
        return np.minimum(l, 0.0) - np.log1p(np.exp(-np.abs(l))) if sigmoid else l


def _best_first(values):
    """Indices by descending value, the lower first on equal ones."""
    return sorted(range(len(values)), key=lambda i: (-values[i], i))


def route(logits, k, bias=None, sigmoid=True, groups=1, keep=1, best=2, norm=True, scale=1.0):
    """-> (ids int32[T, k], weights float64[T, k]), token by token."""
    logits = np.asarray(logits, np.float32)
    T, E = logits.shape
    size = E // groups
    s_all = scores(logits, sigmoid)
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float32).astype(np.float64)
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        l, s = logits[t].astype(np.float64), s_all[t]
        c = s + b
        ok = (l > -np.inf) & (c > -np.inf)              # False for NaN
        worth = []
        for g in range(groups):
            of = sorted((c[e] for e in range(g * size, (g + 1) * size) if ok[e]), reverse=True)
            worth.append(sum(of[1:best], of[0]) if of else -np.inf)
        stay = set(_best_first(worth)[:keep])
        rank = c if bias is not None else l + 0.0
        left = [e for e in range(E) if ok[e] and e // size in stay]
        left.sort(key=lambda e: (-rank[e], e))
        left = left[:k]
        n = len(left)
        if not n:
            continue
        ids[t, :n] = left
        if norm:
            z = log_scores(l[left], sigmoid)
            with np.errstate(all="ignore"):
                p = np.where(z == z.max(), 1.0, np.exp(z - z.max()))
            w[t, :n] = p / p.sum() * scale
        else:
            w[t, :n] = s[left] * scale
    return ids, w


def lora(x, slots, a, b, y, scale=None):
    """float64: y[m] + scale_s b_s (a_s x_m), s = slots[m]; rows of other slots are y's."""
    out = np.array(y, np.float64)
    for m, s in enumerate(slots):
        if 0 <= s < len(a):
            t = np.asarray(a[s], np.float64) @ np.asarray(x[m], np.float64)
            out[m] += (1.0 if scale is None else float(scale[s])) * (np.asarray(b[s], np.float64) @ t)
    return out


def lora_magnitudes(x, slots, a, b, scale=None):
    """(sum |b| |scale| sum |a x|, sum |b| |scale a x|) per element of y: what fp32 sums' errors go by."""
    full, outer = (np.zeros((len(slots), b.shape[1])) for _ in range(2))
    for m, s in enumerate(slots):
        if 0 <= s < len(a):
            f = 1.0 if scale is None else abs(float(scale[s]))
            ax = np.asarray(a[s], np.float64) * np.asarray(x[m], np.float64)
            full[m] = np.abs(b[s]) @ np.abs(ax).sum(1) * f
            outer[m] = np.abs(b[s]) @ np.abs(ax.sum(1)) * f
    return full, outer
