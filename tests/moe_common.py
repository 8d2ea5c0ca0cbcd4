"""Routing to experts and the combination of their rows from their definitions in 64
bits (numpy), one token at a time, for the tests; shares nothing with the library."""
import numpy as np


def scores(l, kind):
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = l.max()
        if m == -np.inf:
            return np.zeros_like(l)
        e = np.exp(l - m)
        return e / e.sum()


def best_first(key, count):
    """Indices of the `count` largest entries that are above -inf, the lowest index first among equals."""
    order = sorted((i for i in range(len(key)) if key[i] > -np.inf), key=lambda i: (-key[i], i))
    return order[:count]


def route(logits, top, score="softmax", bias=None, groups=1, groups_kept=None, group_best=1, renormalise=False,
          scale=1.0):
    """(experts, weights) of logits [tokens, E], float64."""
    tokens, count = logits.shape
    experts, weights = np.full((tokens, top), -1), np.zeros((tokens, top))
    kept = groups if groups_kept is None else groups_kept
    for t in range(tokens):
        l = logits[t]
        if np.isnan(l).any() or (l == np.inf).any():
            weights[t] = np.nan
            continue
        s = scores(l, score)
        key = s.copy() if bias is None else s + bias
        key[(l == -np.inf) | ~(key > -np.inf)] = -np.inf
        if groups > 1:
            parts = key.reshape(groups, -1)
            total = np.full(groups, -np.inf)
            for g in range(groups):
                two = parts[g][best_first(parts[g], group_best)]
                if len(two):
                    total[g] = two.sum()
            for g in set(range(groups)) - set(best_first(total, kept)):
                parts[g] = -np.inf
            key = parts.reshape(-1)
        chosen = best_first(key, top)
        w = s[chosen]
        if renormalise:
            w = w / w.sum() if w.sum() > 0 else 0.0 * w
        experts[t, :len(chosen)], weights[t, :len(chosen)] = chosen, w * scale
    return experts, weights


def order(experts, count):
    """(offsets, rows, slots) of experts [tokens, top]."""
    tokens, top = experts.shape
    rows, slots, offsets = np.full(tokens * top, -1), np.full((tokens, top), -1), np.zeros(count + 1, dtype=int)
    at = 0
    for e in range(count):
        offsets[e] = at
        for t, j in np.argwhere(experts == e):
            rows[at], slots[t, j] = t, at
            at += 1
    offsets[count] = at
    return offsets, rows, slots


def combine(y, slots, weights, add=None):
    """(out, sum of magnitudes), float64."""
    tokens = slots.shape[0]
    out = np.zeros((tokens, y.shape[1])) if add is None else add.copy()
    size = np.abs(out)
    for t in range(tokens):
        for s, w in zip(slots[t], weights[t]):
            v = w * (y[s] if 0 <= s < len(y) else np.zeros(y.shape[1]))
            out[t] += v
            size[t] += np.abs(v)
    return out, size
