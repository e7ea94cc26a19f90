"""CPU oracle of the operators around the experts and of the adapters (test infrastructure only,
plain numpy in float64, one row at a time).

  route     s = softmax or sigmoid of the logits, c = s + bias; groups by their largest c or the sum
            of their two largest; the k largest c of the groups kept; weights from s
  group     the slots of each expert in turn, each expert's in their order
  combine   sum_j w_j y[position_j] (+ residual), and the sum of the terms' magnitudes
  lora      base + scale (x A^T) B^T, with the magnitudes its error bound needs
"""
from __future__ import annotations

import numpy as np


def _largest(values, n):
    """Indices of the n largest finite-or-larger values, the lowest index first among equal ones."""
    order = sorted((i for i, v in enumerate(values) if v > -np.inf), key=lambda i: (-values[i], i))
    return order[:n]


def route_row(l, k, bias=None, sigmoid=False, groups=1, topk_groups=1, best=1, renormalize=True, scale=1.0):
    """Experts (list, -1 where none is left) and weights (list) of one row of float64 logits."""
    E = len(l)
    if np.isnan(l).any() or (not sigmoid and np.isposinf(l).any()):
        return list(range(k)), [np.nan] * k
    open_ = l > -np.inf
    with np.errstate(over="ignore", under="ignore"):
        if sigmoid:
            s = np.where(l > 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
        else:
            s = np.exp(l - l[open_].max()) if open_.any() else np.zeros(E)
            s = s / s.sum() if open_.any() else s
    c = s.copy() if bias is None else s + bias
    if np.isnan(c[open_]).any():
        return list(range(k)), [np.nan] * k
    if bias is None and (groups == 1 or best == 1):
        c = l.copy()                       # the same order, without the scores' rounding
    c[~open_] = -np.inf
    if groups > 1:
        per = E // groups
        value = []
        for g in range(groups):
            top = sorted((v for v in c[g * per:(g + 1) * per] if v > -np.inf), reverse=True)[:best]
            value.append(sum(top) if top else -np.inf)
        # (a group with nothing left may be among the kept: it adds nothing)
        kept = sorted(range(groups), key=lambda g: (-value[g], g))[:topk_groups]
        for g in range(groups):
            if g not in kept:
                c[g * per:(g + 1) * per] = -np.inf
    chosen = _largest(c, k)
    w = s[chosen]
    if renormalize and chosen:
        if sigmoid:                        # s up to a common factor, which cancels
            top = min(l[chosen].max(), 0.0)
            with np.errstate(over="ignore"):
                w = np.array([1 / (1 + np.exp(-v)) if v > 0 else np.exp(v - top) / (1 + np.exp(v)) for v in l[chosen]])
        else:
            w = np.exp(l[chosen] - l[chosen].max())
        w = w / w.sum()
    pad = k - len(chosen)
    return chosen + [-1] * pad, [float(v) * scale for v in w] + [0.0] * pad


def route(l, k, **kw):
    rows = [route_row(r, k, **kw) for r in np.asarray(l, np.float64)]
    return (np.array([r[0] for r in rows], np.int32).reshape(-1, k),
            np.array([r[1] for r in rows], np.float64).reshape(-1, k))


def group_rows(ids, E):
    """rows, offsets, position as lowbit_group_rows writes them."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    rows, offsets, position = [], [0], np.full(T * k, -1, np.int32)
    for e in range(E):
        for s in np.flatnonzero(flat == e):
            position[s] = len(rows)
            rows.append(s // k)
        offsets.append(len(rows))
    rows += [s // k for s in np.flatnonzero((flat < 0) | (flat >= E))]
    return np.array(rows, np.int32).reshape(-1), np.array(offsets, np.int32), position.reshape(T, k)


def combine(y, position, weights, residual=None):
    """(out, sum of the terms' magnitudes), float64."""
    T, k = position.shape
    out = np.zeros((T, y.shape[1])) if residual is None else residual.astype(np.float64).copy()
    A = np.abs(out)
    for t in range(T):
        for p, w in zip(position[t], weights[t].astype(np.float64)):
            if p < 0:
                continue
            row = y[p] if p < y.shape[0] else np.full(y.shape[1], np.nan)
            out[t] += w * row
            A[t] += np.abs(w * row)
    return out, A


def lora(x, a, b, scales, ids, base=None):
    """float64 arrays: y, and per output sum_j |s b_j| * (sum_k |x a_j|), sum_j |s b_j t_j| and
    sum_j |s b_j| * max_j |t_j|.  ids: each row's adapter, or -1."""
    M, N = x.shape[0], b.shape[1]
    y = np.zeros((M, N)) if base is None else base.astype(np.float64).copy()
    At, Ab, Am = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
    for l in range(a.shape[0]):
        at = np.flatnonzero(ids == l)
        if len(at):
            s = 1.0 if scales is None else float(scales[l])
            t = x[at] @ a[l].T
            y[at] += s * (t @ b[l].T)
            absb = np.abs(s * b[l]).T
            At[at] = (np.abs(x[at]) @ np.abs(a[l]).T) @ absb
            Ab[at] = np.abs(t) @ absb
            Am[at] = np.abs(t).max(1, keepdims=True) * absb.sum(0)
    return y, At, Ab, Am
