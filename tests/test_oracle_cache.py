"""Pins of the paged-cache oracle (CPU): hand-made values and identities."""
import numpy as np
import torch

from oracle import cache as oc


def test_e4m3_rounding_agrees_with_every_code_and_midpoint():
    codes = torch.arange(0, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    codes = codes.astype(np.float64)                      # 0 .. 448, ascending
    assert codes[-1] == 448.0 and np.array_equal(oc.e4m3_round(codes), codes)
    mid = (codes[1:] + codes[:-1]) / 2
    even = np.where(np.arange(len(mid)) % 2 == 0, codes[:-1], codes[1:])
    assert np.array_equal(oc.e4m3_round(mid), even)
    assert np.array_equal(oc.e4m3_round(-mid), -even)
    assert np.array_equal(oc.e4m3_round(np.nextafter(mid, 1e9)), codes[1:])
    assert np.array_equal(oc.e4m3_round(np.nextafter(mid, 0)), codes[:-1])


def test_quantise_edges():
    x = np.zeros((4, 8), np.float32)
    x[1, 3] = -896.0
    x[2, 0] = np.inf
    x[3, 5] = np.float32(1e-44)
    c, s = oc.quantise(x)
    assert s[0] == np.float32(2.0 ** -126) and not c[0].any()
    assert s[1] == 2.0 and c[1, 3] == -448.0
    assert np.isnan(s[2]) and not c[2].any()
    assert s[3] == np.float32(2.0 ** -126)


def test_tree_mask_by_hand():
    parent = np.array([[-1, 0, 0, 1, 3, 2]], np.int32)
    pos, see = oc.tree_mask(parent, [6], [10])
    assert pos.tolist() == [[10, 11, 11, 12, 13, 12]]
    assert np.flatnonzero(see[0, 4]).tolist() == [0, 1, 3, 4]
    assert np.flatnonzero(see[0, 5]).tolist() == [0, 2, 5]
    _, near = oc.tree_mask(parent, [6], [10], window=2)
    assert np.flatnonzero(near[0, 4]).tolist() == [3, 4]
    assert oc.pack_bits(see)[0, 4, 0] == 0b011011
    pos, see = oc.tree_mask(np.array([[-1, 0, 2]], np.int32), [3], [0])  # its own parent
    assert (pos == -1).all() and not see.any()


def test_rotation_keeps_norms_and_relative_angles():
    g = np.random.default_rng(3)
    t = np.arange(40)[:, None] * 10.0 ** -(np.arange(8) / 4.0)[None, :]
    rope = np.stack([np.cos(t), np.sin(t)], -1)
    x, y = g.standard_normal((2, 1, 24))
    for inter in (False, True):
        a, b = (oc.norm_rotate(x, None, 0, rope, p, inter) for p in (5, 25))
        c, d = (oc.norm_rotate(y, None, 0, rope, p, inter) for p in (9, 29))
        assert np.allclose((a * a).sum(), (x * x).sum())
        assert np.allclose((a * c).sum(), (b * d).sum())   # scores go by the difference alone
        assert np.array_equal(a[:, 16:], x[:, 16:])
    z = oc.norm_rotate(x, np.ones(24), 0.0, None, 0, False)
    assert np.allclose((z * z).mean(), 1.0)


def test_attention_masks_and_empty_rows():
    g = np.random.default_rng(4)
    q, k, v = g.standard_normal((2, 4)), g.standard_normal((5, 4)), g.standard_normal((5, 4))
    k[2], v[2] = np.nan, np.inf
    see = np.array([[1, 0, 0, 1, 0], [0, 0, 0, 0, 0]], bool)
    o, lse, _, _ = oc.attention(q, k, v, see, 0.5)
    s = np.array([k[0] @ q[0], k[3] @ q[0]]) * 0.5
    w = np.exp(s) / np.exp(s).sum()
    assert np.allclose(o[0], w[0] * v[0] + w[1] * v[3]) and np.allclose(lse[0], np.log(np.exp(s).sum()))
    assert not o[1].any() and lse[1] == -np.inf
