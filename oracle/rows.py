"""Oracle of the row operators: pairs sorted by expert with dropped pairs, token rows brought to
their pairs' rows and back with weights, and the gradients.  float64, written from the definitions,
one pair at a time."""
from __future__ import annotations

import numpy as np


def permute_capacity(ids, E: int, capacity: int = 0):
    """(expert_offsets [E+1], sorted_pair [P], pair_to_row [P], expert_list [E+1]): pairs with an id
    outside 0..E-1, or with `capacity` earlier pairs of the same id (capacity > 0), are dropped:
    pair_to_row -1, and behind the kept ones in sorted_pair, ascending.  expert_list is defined up to
    entry expert_list[0]; the rest is 0 here."""
    ids = np.asarray(ids).reshape(-1)
    of = [[] for _ in range(E)]
    lost = []
    for p, e in enumerate(ids):
        if 0 <= e < E and (capacity == 0 or len(of[e]) < capacity):
            of[e].append(p)
        else:
            lost.append(p)
    offsets = np.concatenate([[0], np.cumsum([len(v) for v in of])]).astype(np.int32)
    kept = [p for v in of for p in v]
    row = np.full(ids.size, -1, np.int32)
    row[kept] = np.arange(len(kept))
    active = [e for e in range(E) if of[e]]
    lst = np.zeros(E + 1, np.int32)
    lst[0] = len(active)
    lst[1:1 + len(active)] = active
    return offsets, np.array(kept + lost, np.int32), row, lst


def sort_rows(x, w, row, k: int, rows):
    """rows[row[p]] = w_p x[p // k] into a copy of `rows`; w None: weight 1."""
    rows = np.array(rows, np.float64)
    for p, r in enumerate(row):
        if r >= 0:
            rows[r] = x[p // k] * (1.0 if w is None else w[p])
    return rows


def unsort_rows(rows, w, row, T: int, k: int, residual=None):
    """out[t] = sum_j w_p rows[row[p]] (+ residual[t])."""
    out = np.zeros((T, rows.shape[1])) if residual is None else np.array(residual, np.float64)
    for p, r in enumerate(row):
        if r >= 0:
            out[p // k] += rows[r] * (1.0 if w is None else w[p])
    return out


def pair_dots(rows, x, row, k: int):
    """dw_p = <rows[row[p]], x[p // k]>, 0 without a row: the weights' gradient of both directions."""
    return np.array([float(np.dot(rows[r], x[p // k])) if r >= 0 else 0.0 for p, r in enumerate(row)])


def route_topk_bwd(dw, w, ids, T: int, E: int, k: int):
    """d_logits [T][E] of w = softmax over the k chosen logits."""
    out = np.zeros((T, E))
    for t in range(T):
        wt, dt = w[t * k:(t + 1) * k], dw[t * k:(t + 1) * k]
        s = float(np.dot(wt, dt))
        for j in range(k):
            e = ids[t * k + j]
            if 0 <= e < E:
                out[t, e] += wt[j] * (dt[j] - s)
    return out
