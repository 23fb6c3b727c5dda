"""Plain numpy float64 oracle of the paged cache: rows of a page table, decode
attention over the rows held with its weights, and eviction by accumulated
attention weight.  Test infrastructure only; one function per step, no
blocking, nothing shared with the CUDA path."""
from __future__ import annotations

import numpy as np


def rows(pool: np.ndarray, table_row: np.ndarray, h: int, n: int, n_pages: int):
    """The first n rows of one (sequence, KV head): pool [n_pages, heads, page,
    d], and a mask of those whose page id is valid (the others are zero)."""
    page = pool.shape[2]
    out, ok = np.zeros((n, pool.shape[3])), np.zeros(n, dtype=bool)
    for r in range(n):
        p = int(table_row[r // page])
        if 0 <= p < n_pages:
            out[r], ok[r] = pool[p, h, r % page], True
    return out, ok


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, ok: np.ndarray, scale: float):
    """q [g, d] over rows k, v [n, d] with ok set: (out [g, d], lse [g], the
    weights' sum over the g heads [n])."""
    g = q.shape[0]
    out, lse, weight = np.zeros((g, v.shape[1])), np.full(g, -np.inf), np.zeros(len(k))
    if not ok.any():
        return out, lse, weight
    for j in range(g):
        s = scale * (k[ok] @ q[j])
        m = s.max()
        e = np.exp(s - m)
        lse[j] = m + np.log(e.sum())
        p = e / e.sum()
        out[j] = p @ v[ok]
        weight[ok] += p
    return out, lse, weight


def keep(mass: np.ndarray, pos: np.ndarray, seen: int, budget: int, sinks: int, recent: int) -> np.ndarray:
    """Mask of the rows kept: protected ones first, then mass descending (NaN
    lowest), ties to the lower row; everything when at most `budget` rows."""
    n = len(mass)
    if n <= budget:
        return np.ones(n, dtype=bool)

    def rank(r):
        protected = pos[r] < sinks or pos[r] >= seen - recent
        m = float(mass[r])
        nan = m != m
        return (not protected, nan and not protected, 0.0 if protected or nan else -m, r)

    kept = np.zeros(n, dtype=bool)
    kept[sorted(range(n), key=rank)[:budget]] = True
    return kept


def moves(kept: np.ndarray, budget: int) -> np.ndarray:
    """[(source, destination)]: the k-th kept row at or past the budget goes to
    the k-th slot below it that was not kept."""
    if len(kept) <= budget:
        return np.zeros((0, 2), dtype=np.int32)
    src = [r for r in range(budget, len(kept)) if kept[r]]
    dst = [r for r in range(budget) if not kept[r]]
    assert len(src) == len(dst)
    return np.array(list(zip(src, dst)), dtype=np.int32).reshape(-1, 2)
