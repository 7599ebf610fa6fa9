"""Plain CPU oracle of truncated draws: sorted rows of whole-number weights.

TEST INFRASTRUCTURE ONLY: the tests call this; the product library never does.
It shares no code with the HIP library.
"""
from __future__ import annotations

import math

import numpy as np

UNIT = 2.0 ** 44


def kept(x, t, k=0, p=1.0, min_p=0.0):
    """(mask of kept ids, int64 weights of all ids) of one row in fp64."""
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        fall = (x - x.max()) / (t if t else 1.0)
    w = np.rint(np.exp(fall) * UNIT).astype(np.int64)
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    n = len(order)
    if t == 0:
        n = 1
    else:
        if k > 0:
            n = min(n, k)
        left = n
        if p < 1:
            need = math.ceil(p * float(w[order[:n]].sum()))
            n = min(n, int(np.searchsorted(np.cumsum(w[order[:n]]), need)) + 1)
        if min_p > 0:
            # (e^y >= p is y >= ln p; e^y itself rounds to 1 where |y| < 2^-53)
            n = min(n, int((fall[order[:left]] >= math.log(min_p)).sum()))
    mask = np.zeros(len(x), bool)
    mask[order[:n]] = True
    return mask, w


def draw(x, t, u, k=0, p=1.0, min_p=0.0):
    """(token, log q, kept ids) of one row."""
    mask, w = kept(x, t, k, p, min_p)
    if t == 0:
        return int(np.argmax(x)), 0.0, 1
    w = np.where(mask, w, 0)
    total = float(w.sum())
    i = int(np.searchsorted(np.cumsum(w), math.floor(u * total), side="right"))
    return i, (float(x[i]) - float(np.max(x))) / t - math.log(total / UNIT), int(mask.sum())
