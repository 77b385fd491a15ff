"""Float64 oracle of moe_route_experts (softmax or sigmoid scores, bias, groups)."""
from __future__ import annotations

import numpy as np

SOFTMAX, SIGMOID = 0, 1


def scores(logits, scoring):
    """s [T, E]; a logit of -inf has score 0."""
    z = np.asarray(logits, dtype=np.float64)
    with np.errstate(over="ignore"):
        if scoring == SIGMOID:
            return 1.0 / (1.0 + np.exp(-z))
    top = z.max(axis=1, keepdims=True)
    e = np.exp(z - np.where(np.isneginf(top), 0.0, top))
    den = e.sum(axis=1, keepdims=True)
    return e / np.where(den > 0, den, 1.0)


def log_scores(logits, scoring):
    """log s [T, E], which does not underflow (-inf for a logit of -inf)."""
    z = np.asarray(logits, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if scoring == SIGMOID:
            return -np.logaddexp(0.0, -z)
        top = z.max(axis=1, keepdims=True)
        top = np.where(np.isneginf(top), 0.0, top)
        return z - top - np.log(np.exp(z - top).sum(axis=1, keepdims=True))


def route_experts(logits, k, scoring=SOFTMAX, bias=None, n_group=1, topk_group=1, group_best=1,
                  renormalize=True, scale=1.0):
    """(ids [T, k] int32, weights [T, k] float64)"""
    z = np.asarray(logits, dtype=np.float64)
    T, E = z.shape
    s, ls = scores(z, scoring), log_scores(z, scoring)
    c = s if bias is None else s + np.asarray(bias, dtype=np.float64)
    c = np.where(np.isneginf(z), -np.inf, c)
    order = z if bias is None else c                   # the score grows with the logit
    S = E // n_group
    ids, w = np.zeros((T, k), dtype=np.int32), np.zeros((T, k))
    for t in range(T):
        value = []
        for g in range(n_group):
            live = sorted((v for v in c[t, g * S:(g + 1) * S] if v > -np.inf), reverse=True)
            value.append(sum(live[:group_best]) if live else -np.inf)
        stay = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
        left = [order[t, e] if e // S in stay and c[t, e] > -np.inf else -np.inf for e in range(E)]
        ids[t] = sorted(range(E), key=lambda e: (-left[e], e))[:k]
        live = np.array([left[e] > -np.inf for e in ids[t]])
        if renormalize and live.any():                 # ratios of scores, whatever their size
            lc = np.where(live, ls[t, ids[t]], -np.inf)
            chosen = np.exp(lc - lc.max())
            chosen = chosen / chosen.sum()
        else:
            chosen = np.where(live, s[t, ids[t]], 0.0)
        w[t] = chosen * scale
    return ids, w
