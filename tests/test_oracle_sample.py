"""Pins of the truncated-draw oracle (CPU): rows by hand, torch's softmax."""
import numpy as np
import torch

from oracle import sample as osm

ROW = np.log(np.array([0.1, 0.4, 0.2, 0.2, 0.05, 0.05]))


def ids(x, *a, **k):
    return np.flatnonzero(osm.kept(x, *a, **k)[0]).tolist()


def test_prefixes_by_hand():
    assert ids(ROW, 1.0) == [0, 1, 2, 3, 4, 5]
    assert ids(ROW, 1.0, k=2) == [1, 2]                             # the lower of equal ones
    assert ids(ROW, 1.0, k=3) == [1, 2, 3] and ids(ROW, 1.0, k=99) == [0, 1, 2, 3, 4, 5]
    assert ids(ROW, 1.0, p=0.39) == [1] and ids(ROW, 1.0, p=0.41) == [1, 2]
    assert ids(ROW, 1.0, p=0.79) == [1, 2, 3] and ids(ROW, 1.0, p=0.81) == [0, 1, 2, 3]
    assert ids(ROW, 1.0, min_p=0.49) == [1, 2, 3] and ids(ROW, 1.0, min_p=0.51) == [1]
    assert ids(ROW, 1.0, min_p=1.0) == [1] and ids(ROW, 0.0) == [1]
    assert ids(ROW, 1.0, k=3, p=0.74) == [1, 2]                     # of 0.8: 0.592
    assert ids(ROW, 0.5, p=0.6) == [1] and ids(ROW, 2.0, p=0.7) == [0, 1, 2, 3]
    assert ids(np.array([3.0, -np.inf, 3.0]), 1.0) == [0, 2]
    assert ids(np.array([3.0, 3.0, 3.0, 3.0]), 1.0, p=0.5) == [0, 1]


def test_draws_by_hand():
    got = [osm.draw(ROW, 1.0, u)[0] for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.71, 0.96, 0.999)]
    assert got == [0, 0, 1, 1, 2, 3, 5, 5]
    assert [osm.draw(ROW, 1.0, u, k=2)[0] for u in (0.0, 0.66, 0.67)] == [1, 1, 2]
    tok, lq, n = osm.draw(ROW, 1.0, 0.9, k=2)
    assert (tok, n) == (2, 2) and abs(lq - np.log(1 / 3)) < 1e-12
    assert osm.draw(ROW, 0.0, 0.99) == (1, 0.0, 1)


def test_probabilities_are_the_softmax():
    g = np.random.default_rng(0)
    x = g.standard_normal(500) * 3
    mask, w = osm.kept(x, 0.7, k=40)
    want = torch.softmax(torch.from_numpy(x / 0.7).masked_fill(~torch.from_numpy(mask), -np.inf), 0).numpy()
    assert mask.sum() == 40 and set(np.flatnonzero(mask)) == set(torch.from_numpy(x).topk(40).indices.tolist())
    got = np.where(mask, w, 0) / w[mask].sum()
    assert np.abs(got - want).max() < 1e-12
    for u in g.random(50):
        tok, lq, _ = osm.draw(x, 0.7, u, k=40)
        assert np.isclose(lq, np.log(want[tok]), atol=1e-11)
        assert want[:tok].sum() - 1e-12 <= u <= want[:tok + 1].sum() + 1e-12
