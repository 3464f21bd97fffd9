"""Plain fp64 forms of routing by scores with a bias and groups, of its gates
and of their gradient (numpy, one token after the other)."""

import numpy as np


def scores(l, score):
    """Scores of one token's logits; those of -infinity and NaN are 0."""
    l = np.where(np.isnan(l), -np.inf, np.asarray(l, dtype=np.float64))
    if score == "sigmoid":
        u = np.exp(-np.abs(l))
        return np.where(l >= 0, 1.0, u) / (1.0 + u)
    top = l.max()
    if np.isinf(top):
        e = (l == top).astype(np.float64) if top > 0 else np.zeros(len(l))
    else:
        e = np.exp(l - top)
    return e / e.sum() if e.sum() > 0 else e


def choose(l, k, score, bias, groups, top_groups, group_score):
    """Expert ids of one token, best first."""
    l = np.where(np.isnan(l), -np.inf, np.asarray(l, dtype=np.float64))
    s, E = scores(l, score), len(l)
    with np.errstate(invalid="ignore"):
        c = l.copy() if bias is None else s + np.asarray(bias, dtype=np.float64)
    c[np.isnan(c) | (l == -np.inf)] = -np.inf
    best = list(range(E))
    if groups > 1:
        size = E // groups
        per = c.reshape(groups, size)
        if group_score == "max":
            worth = per.max(1)
        else:
            two = np.where(c == -np.inf, -np.inf, s if bias is None else c).reshape(groups, size)
            with np.errstate(invalid="ignore"):
                worth = np.sort(two, 1)[:, -2:].sum(1)
            worth = np.where(np.isnan(worth), -np.inf, worth)
        kept = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
        best = [e for e in range(E) if e // size in kept]
    return sorted(best, key=lambda e: (-c[e], e))[:k]


def gates(l, ids, score, renorm, scale):
    """Gates of one token's experts ids."""
    if renorm and score == "softmax":
        g = scores(np.asarray(l)[ids], score)      # the softmax over the chosen ones
    else:
        g = scores(l, score)[ids]
        if renorm:
            g = g / g.sum() if g.sum() > 0 else np.zeros(len(g))
    return scale * g


def route(logits, k, score="softmax", bias=None, groups=1, top_groups=None, group_score="max", renorm=True, scale=1.0):
    """(ids [T, k], gates [T, k])."""
    top = groups if top_groups is None else top_groups
    ids = [choose(l, k, score, bias, groups, top, group_score) for l in logits]
    g = [gates(l, i, score, renorm, scale) for l, i in zip(logits, ids)]
    return np.array(ids, dtype=np.int64).reshape(-1, k), np.array(g, dtype=np.float64).reshape(-1, k)


def sort_pairs(ids, E):
    """(offsets, sorted_pairs, pair_pos) of the stable counting sort."""
    flat = np.asarray(ids).reshape(-1)
    order = np.argsort(flat, kind="stable")
    pos = np.empty_like(order)
    pos[order] = np.arange(len(order))
    return np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))]), order, pos


def route_grad(logits, ids, d_gates, score="softmax", renorm=True, scale=1.0):
    """(d_logits [T, E], and the sum of the magnitudes of each entry's terms);
    ids outside [0, E) are no experts."""
    logits = np.asarray(logits, dtype=np.float64)
    out, mag = np.zeros(logits.shape), np.zeros(logits.shape)
    for t, l in enumerate(logits):
        l = np.where(np.isnan(l), -np.inf, l)
        s = scores(l, score)
        ok = [j for j, e in enumerate(ids[t]) if 0 <= e < len(l)]
        e, dg = np.asarray(ids[t])[ok], np.asarray(d_gates[t], dtype=np.float64)[ok]
        if score == "softmax" and not renorm:
            d, a = np.zeros(len(l)), np.zeros(len(l))
            np.add.at(d, e, scale * dg)
            np.add.at(a, e, abs(scale * dg))
            mean = scale * (dg * s[e]).sum()
            out[t] = s * (d - mean)
            mag[t] = s * (a + abs(scale) * abs(dg * s[e]).sum())
            continue
        if renorm:
            w = gates(l, e, score, True, 1.0) if len(e) else s[e]
            v = (dg - (dg * w).sum()) * w
            m = (abs(dg) + abs(dg * w).sum()) * w
        else:
            v, m = dg * s[e], abs(dg) * s[e]
        if score == "sigmoid":
            rest = scores(-l, "sigmoid")[e]
            v, m = v * rest, m * rest
        np.add.at(out[t], e, scale * v)
        np.add.at(mag[t], e, abs(scale) * m)
    return out, mag


def route_grad_apart(logits, ids, d_gates, score="softmax", renorm=True, scale=1.0):
    """route_grad for distinct ids in [0, E) and finite logits, written so that
    nothing cancels where one expert has nearly all the weight: the differences
    of what experts bring are weighted, not the difference of the weighted taken.
    (d_logits [T, E], and the sum of the magnitudes of each entry's weighted
    differences)."""
    logits = np.asarray(logits, dtype=np.float64)
    out, mag = np.zeros(logits.shape), np.zeros(logits.shape)
    for t, l in enumerate(logits):
        e, dg = np.asarray(ids[t]), scale * np.asarray(d_gates[t], dtype=np.float64)
        if score == "softmax" and not renorm:
            s, v = scores(l, score), np.zeros(len(l))
            v[e] = dg
            apart = v[:, None] - v[None, :]
            out[t], mag[t] = s * (apart @ s), s * (abs(apart) @ s)
            continue
        if renorm:
            w = gates(l, e, score, True, 1.0)
            apart = dg[:, None] - dg[None, :]
            v, m = w * (apart @ w), w * (abs(apart) @ w)
        else:
            v, m = dg * scores(l, score)[e], abs(dg) * scores(l, score)[e]
        rest = scores(-l, "sigmoid")[e] if score == "sigmoid" else 1.0
        out[t][e], mag[t][e] = v * rest, m * rest
    return out, mag
