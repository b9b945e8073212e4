"""Rows of logits in float64: draws under top-k, top-p and min-p, largest logits, distillation (test infrastructure; never
product code).

A row's tokens stand in order of (logit descending, id ascending).  The pages evaluate at temperature 1.0 ([DFlash] and
[DDTree] "실험 결과") and say that the drafter learns from the target with early positions counting more ([DFlash] "학습
방식도 추론 시나리오에 맞춰 바꿨다"); they state neither the cuts nor a loss, so both are the plain ones.
"""
from __future__ import annotations

import math

import numpy as np


def order(row) -> np.ndarray:
    """Token ids in order; masked tokens (-inf) are not in it."""
    row = np.asarray(row, np.float64)
    ids = np.lexsort((np.arange(row.size), -row))
    return ids[row[ids] > -np.inf]


def kept(row, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(ids that stay, their probabilities among each other)."""
    row = np.asarray(row, np.float64)
    ids = order(row)
    if temperature == 0 or ids.size == 0:
        return ids[:1], np.ones(min(1, ids.size))
    if top_k > 0:
        ids = ids[:top_k]
    x = (row[ids] - row[ids[0]]) / float(temperature)
    w = np.exp(x)
    n = ids.size
    if top_p < 1:
        before = np.concatenate(([0.0], np.cumsum(w)[:-1]))
        n = min(n, int((before < float(top_p) * w.sum()).sum()))
    if min_p > 0:
        n = min(n, int((w >= float(min_p)).sum()))
    return ids[:n], w[:n] / w[:n].sum()


def draw(row, u, **settings):
    """(token, ln of its probability among the kept, kept tokens); (-1, -inf, 0) where nothing is left."""
    ids, p = kept(row, **settings)
    if ids.size == 0:
        return -1, -math.inf, 0
    at = min(int((np.cumsum(p) <= float(u)).sum()), ids.size - 1)
    return int(ids[at]), math.log(p[at]), ids.size


def top(row, K, temperature=1.0):
    """(ids, values, log-sum) of the K first tokens; -1 and -inf behind the last one."""
    row = np.asarray(row, np.float64)
    ids = order(row)
    lse = -math.inf
    if ids.size:
        x = row[ids] / temperature
        lse = x[0] + math.log(np.exp(x - x[0]).sum())
    ids = ids[:K]
    pad = K - ids.size
    return (np.concatenate((ids, np.full(pad, -1))).astype(np.int32), np.concatenate((row[ids], np.full(pad, -np.inf))), lse)


def teacher(ids, vals, lse, temperature):
    """(listed ids, their probabilities, mass of the others) of one list."""
    on = np.asarray(ids) >= 0
    ids, v = np.asarray(ids)[on], np.asarray(vals, np.float64)[on] / temperature
    if lse is None:
        v = v - (v.max() + math.log(np.exp(v - v.max()).sum()))
        return ids, np.exp(v), 0.0
    t = np.exp(v - float(lse))
    return ids, t, max(0.0, 1.0 - t.sum())


def distill(z, ids, vals, lse, temperature, weight=1.0):
    """(loss, gradient by z, stats) of one student row; `lse` that of the list's own row, None: the list is all there is.
    Sums are relative to the row's largest logit: what lies 745 temperatures below it is 0 here."""
    z = np.asarray(z, np.float64)
    ids, t, rho = teacher(ids, vals, lse, temperature)
    m = z.max()
    e = np.exp((z - m) / temperature)
    other = np.ones(z.size, bool)
    other[ids] = False
    S, R = e.sum(), e[other].sum()
    kl = 0.0
    with np.errstate(divide="ignore"):
        for i, ti in zip(ids, t):
            if ti > 0:
                kl += ti * (math.log(ti) - ((z[i] - m) / temperature - math.log(S)))
        if rho > 0:
            kl += rho * (math.log(rho) - np.log(R / S))
        stats = np.array([m, math.log(S), np.log(R), 0.0])
    grad = e / S - (rho * e / R if rho > 0 and R > 0 else 0.0)
    grad[ids] = e[ids] / S - t
    return weight * kl, weight / temperature * grad, stats
