"""The router: logits to expert ids and gates, in 64 bits.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

score s = softmax(x) or 1 / (1 + exp(-x)); choice c = s + bias (the logits themselves without a bias and
with groups scored by their best expert), -inf where x or bias is -inf; the experts outside the
topk_group best groups (sum of their group_top largest c) get c = -inf; the ids are the k largest c,
ties to the lowest index; the gates are their scores, 0 where c = -inf.
"""
from __future__ import annotations

import numpy as np


def _first(v: np.ndarray, k: int) -> list:
    """Indices of the k largest, descending, ties to the lowest index (one row, brute force)."""
    left = list(range(len(v)))
    out = []
    for _ in range(k):
        best = left[0]
        for i in left:
            if v[i] > v[best]:
                best = i
        out.append(best)
        left.remove(best)
    return out


def gate(x: np.ndarray, k: int, sigmoid: bool, bias=None, n_group=1, topk_group=1, group_top=1, renorm=True,
         scale=1.0):
    x = np.asarray(x, dtype=np.float64)
    T, E = x.shape
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    ids = np.zeros((T, k), dtype=np.int32)
    gates = np.zeros((T, k))
    for t in range(T):
        with np.errstate(over="ignore", invalid="ignore"):
            if sigmoid:
                s = 1 / (1 + np.exp(-x[t]))
            else:
                p = np.exp(x[t] - x[t].max())
                s = p / p.sum()
        c = s + b if bias is not None or (n_group > 1 and group_top == 2) else x[t].copy()
        c[(x[t] == -np.inf) | (b == -np.inf)] = -np.inf
        if n_group > 1:
            g = c.reshape(n_group, -1)
            score = np.sort(g, axis=1)[:, -group_top:].sum(1)
            keep = _first(score, topk_group)
            c = np.where(np.isin(np.arange(E) // (E // n_group), keep), c, -np.inf)
        ids[t] = _first(c, k)
        w = np.where(c[ids[t]] > -np.inf, s[ids[t]], 0.0)
        if renorm:
            # (scores that underflow together keep their ratios)
            if sigmoid:
                xi = x[t][ids[t]]
                live = c[ids[t]] > -np.inf
                m = min(0.0, xi[live].max()) if live.any() else 0.0
                with np.errstate(over="ignore", invalid="ignore"):
                    w = np.where(live, np.where(xi > 0, s[ids[t]], np.exp(xi - m) / (1 + np.exp(np.minimum(xi, 0)))), 0.0)
            elif (c[ids[t]] > -np.inf).any():
                live = c[ids[t]] > -np.inf
                xi = x[t][ids[t]]
                w = np.where(live, np.exp(xi - xi[live].max()), 0.0)
            w = w / w.sum() if w.sum() > 0 else w * 0
        gates[t] = w * scale
    return ids, gates
