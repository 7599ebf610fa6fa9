"""Plain CPU oracle of drafting over a budget of cache pages, in fp64.

TEST INFRASTRUCTURE ONLY: the tests call this; the product library never does.
It shares no code with the HIP library.

The C ABI header states the definitions: bounds of a page's keys, the score
that they give a page, and the lists of pages that key heads attend over.
"""
from __future__ import annotations

import numpy as np


def bounds(keys):
    """(least, largest) [Hkv, D] of one page's keys [tokens, Hkv, D]; NaN where
    a value is."""
    return keys.min(0), keys.max(0)


def scores(q, k_min, k_max):
    """Scores of pages [F] for one key head: q [rows, D], bounds [F, D]."""
    with np.errstate(invalid="ignore"):
        up, down = np.maximum(q, 0.0).sum(0), np.minimum(q, 0.0).sum(0)
        s = np.zeros(len(k_min))
        for d in range(q.shape[1]):
            s += up[d] * k_max[:, d] + down[d] * k_min[:, d]
    return np.where(np.isnan(s), np.inf, s)


def choose(score, budget, first, last):
    """Ascending indices of the chosen pages."""
    F = len(score)
    if F <= budget:
        return list(range(F))
    kept = set(range(first)) | set(range(F - last, F))
    rest = sorted((i for i in range(F) if i not in kept), key=lambda i: (-score[i], i))
    return sorted(kept | set(rest[:budget - len(kept)]))


def select(q, k_min, k_max, table, ctx_len, n_nodes, budget, page, first, last, width):
    """(lists [R, Hkv, width], listed tokens [R]); q [R, M, Hq, D] and bounds
    [P, Hkv, D] in fp64."""
    R, M, Hq, D = q.shape
    P, Hkv = k_min.shape[:2]
    G = Hq // Hkv
    lists, length = np.full((R, Hkv, width), -1, np.int32), np.zeros(R, np.int32)
    for r in range(R):
        n, c = int(n_nodes[r]), int(ctx_len[r])
        if not 0 <= n <= M or c < 0 or c + n > table.shape[1] * page:
            length[r] = -1
            continue
        if n == 0:
            continue
        mine = table[r, :(c + n - 1) // page + 1]
        if ((mine < 0) | (mine >= P)).any():
            length[r] = -1
            continue
        F = c // page
        for g in range(Hkv):
            rows = q[r, :n, g * G:(g + 1) * G].reshape(-1, D)
            got = choose(scores(rows, k_min[mine[:F], g], k_max[mine[:F], g]), budget, first, last)
            entries = np.concatenate([mine[got], mine[F:]])
            lists[r, g, :len(entries)] = entries
            length[r] = len(got) * page + c % page
    return lists, length
