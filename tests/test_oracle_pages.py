"""Pins of the page oracle (CPU): hand-made choices and the bound's meaning."""
import numpy as np

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
