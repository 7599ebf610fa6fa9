"""Pins of the page oracle (CPU): hand-made choices and the bound's meaning."""
import numpy as np

from cache_util import bf16
from oracle import cache as oc
from oracle import pages as op


def test_a_score_bounds_every_key_of_the_page():
    g = np.random.default_rng(1)
    keys, q = g.standard_normal((20, 16, 1, 8)), g.standard_normal((5, 8))
    lo, hi = zip(*(op.bounds(k) for k in keys))
    s = op.scores(q, np.array(lo)[:, 0], np.array(hi)[:, 0])
    for p in range(20):
        corner = np.where(q.T > 0, hi[p].T, lo[p].T)                # the box's best corner of every row
        assert np.isclose(s[p], (corner.T * q).sum())
        assert (keys[p, :, 0] @ q.T).sum(1).max() <= s[p] + 1e-12


def test_a_score_of_rounded_bounds():
    """e4m3 pages: values are fp32 products code * scale, their bounds rounded to bf16
    (half a step: 2^-8 of each).  The score bounds q . k up to that of its terms, and no
    better."""
    g = np.random.default_rng(2)
    codes, scale = oc.quantise(g.standard_normal((50, 16, 1, 64)).astype(np.float32) * 3)
    keys = (codes.astype(np.float32) * scale[..., None]).astype(np.float64)
    q = g.standard_normal((5, 64))
    lo, hi = (np.array(b)[:, 0] for b in zip(*(op.bounds(k) for k in keys)))
    kept = [bf16(b).double().numpy() for b in (lo, hi)]
    up, down = np.maximum(q, 0).sum(0), np.minimum(q, 0).sum(0)
    slack = 2.0 ** -8 * (np.abs(up * hi) + np.abs(down * lo)).sum(1)
    s, exact = op.scores(q, *kept), op.scores(q, lo, hi)
    assert (np.abs(s - exact) <= slack + 1e-12).all()
    assert ((keys[:, :, 0] @ q.T).sum(2).max(1) <= s + slack + 1e-12).all()
    one = np.zeros((1, 64))
    one[0, 0] = 1.0                                                 # a single dimension: the largest value itself
    below = op.scores(one, *kept) < hi[:, 0]
    assert below.any() and not below.all()


def test_choice_by_hand():
    s = np.array([0.0, 5.0, 1.0, 5.0, 5.0, -1.0, 9.0])
    assert op.choose(s, 7, 0, 0) == list(range(7)) and op.choose(s, 9, 1, 1) == list(range(7))
    assert op.choose(s, 1, 0, 0) == [6]
    assert op.choose(s, 3, 0, 0) == [1, 3, 6]                       # the lower of equal ones
    assert op.choose(s, 4, 1, 1) == [0, 1, 3, 6]
    assert op.choose(s, 2, 1, 1) == [0, 6] and op.choose(s, 0, 0, 0) == []
    nan = op.scores(np.ones((1, 2)), np.zeros((3, 2)), np.array([[1.0, 2], [np.nan, 0], [np.inf, 1]]))
    assert nan.tolist() == [3.0, np.inf, np.inf] and op.choose(nan, 1, 0, 0) == [1]


def test_lists_by_hand():
    q = np.array([[[[1.0, -1.0]]]])                                 # one row
    lo, hi = np.zeros((9, 1, 2)), np.zeros((9, 1, 2))
    hi[[4, 7, 2], 0, 0] = [1.0, 3.0, 2.0]
    lo[2, 0, 1] = -4.0                                              # page 2: 2 + 4
    table = np.array([[4, 7, 2, 8, 5]])
    lists, n = op.select(q, lo, hi, table, [50], [1], 1, 16, 0, 0, 4)
    assert lists.tolist() == [[[2, 8, -1, -1]]] and n.tolist() == [16 + 2]
    lists, n = op.select(q, lo, hi, table, [48], [1], 2, 16, 0, 0, 4)
    assert lists.tolist() == [[[7, 2, 8, -1]]] and n.tolist() == [32]
    lists, n = op.select(q, lo, hi, table, [48], [0], 2, 16, 0, 0, 4)
    assert (lists == -1).all() and n.tolist() == [0]
    lists, n = op.select(q, lo, hi, np.array([[4, 99, 2, 8, 5]]), [48], [1], 2, 16, 0, 0, 4)
    assert (lists == -1).all() and n.tolist() == [-1]
