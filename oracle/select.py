"""Expert selection from router scores and its backward, in float64.

Test infrastructure only (see the package header).

    p = sigmoid(s) or softmax(s);  key = p + bias  (without a bias: the order of s, in which p grows)
    group score = sum of the group_top best keys of a group, experts with s = -inf left out
    ids = the k best keys of the groups_kept best groups, ties to the lower index
    w = scale * p_i / (sum of the k p), or scale * p_i

A token at a time, written as the definition reads. NaN scores count as -inf. The backward goes by the
chain rule step by step: dL/dw -> dL/dp of the slots -> dL/ds over all experts.

Pins: tests/test_oracle_around.py (brute-force enumeration, central differences)."""

from __future__ import annotations

import numpy as np


def probabilities(s: np.ndarray, score: str) -> np.ndarray:
    """p of one token's scores (float64, NaN already -inf)."""
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-s))
    top = s.max()
    if top == -np.inf:
        return np.zeros_like(s)
    with np.errstate(invalid="ignore"):
        z = np.where(s == top, 1.0, np.exp(np.where(s == top, 0.0, s - top)))
    return z / z.sum()


def _clean(scores) -> np.ndarray:
    s = np.array(scores, dtype=np.float64)
    s[np.isnan(s)] = -np.inf
    return s


def forward(scores, k, score="sigmoid", bias=None, groups=1, kept=None, group_top=1, renorm=True, scale=1.0):
    """(ids int64 [Q, k], weights [Q, k])."""
    s_all = _clean(scores)
    q, e = s_all.shape
    kept = groups if kept is None else kept
    size = e // groups
    ids = np.zeros((q, k), dtype=np.int64)
    w = np.zeros((q, k))
    for t in range(q):
        s = s_all[t]
        p = probabilities(s, score)
        key = p if bias is None else np.where(np.isnan(bias), -np.inf, p + bias)
        key = np.where(s == -np.inf, -np.inf, key)
        rank = s if bias is None else key
        group_score = []
        for g in range(groups):
            pick = rank if group_top == 1 else key
            best = sorted((v for v in pick[g * size:(g + 1) * size] if v > -np.inf), reverse=True)[:group_top]
            group_score.append(sum(best) if best else -np.inf)
        inside = sorted(range(groups), key=lambda g: (-group_score[g], g))[:kept]
        open_ = [i for g in sorted(inside) for i in range(g * size, (g + 1) * size)]
        chosen = sorted(open_, key=lambda i: (-rank[i], i))[:k]
        ids[t] = chosen
        w[t] = _weights(s[chosen], p[chosen], score, renorm, scale)
    return ids, w


def _weights(s, p, score, renorm, scale):
    if not renorm:
        return scale * p
    top = s.max() if len(s) else -np.inf
    if top == -np.inf:
        return np.zeros_like(p)
    if score == "softmax":
        with np.errstate(invalid="ignore"):
            u = np.where(s == top, 1.0, np.exp(np.where(s == top, 0.0, s - top)))
    else:  # sigmoid scaled by exp(-min(top, 0)): the same ratios, no common underflow
        u = np.exp(np.minimum(s, 0) - min(top, 0)) / (1 + np.exp(-np.abs(s)))
    return scale * u / u.sum()


def backward(scores, ids, grad_route, score="sigmoid", renorm=True, scale=1.0):
    """dL/dscores [Q, E]; ids outside [0, E) contribute nothing."""
    s_all = _clean(scores)
    ids = np.asarray(ids)
    g_all = np.asarray(grad_route, dtype=np.float64)
    q, e = s_all.shape
    out = np.zeros((q, e))
    for t in range(q):
        s = s_all[t]
        slots = [(int(i), g) for i, g in zip(ids[t], g_all[t]) if 0 <= i < e]
        if not slots:
            continue
        at = np.array([i for i, _ in slots])
        g = np.array([v for _, v in slots])
        p = probabilities(s, score)
        share = _weights(s[at], p[at], score, renorm, 1.0)  # w / scale
        with np.errstate(over="ignore"):
            slope = 1.0 / (1.0 + np.exp(s)) if score == "sigmoid" else None  # d log p / ds = 1 - p
        # d log p of a slot carries share * g (minus the renormalisation's mean)
        dlog = scale * share * (g - (share * g).sum() if renorm else g)
        dlog = np.where(s[at] == -np.inf, 0.0, dlog)
        if score == "sigmoid":
            np.add.at(out[t], at, dlog * slope[at])
        else:
            np.add.at(out[t], at, dlog)
            if not renorm:
                out[t] -= p * dlog.sum()
    return out
