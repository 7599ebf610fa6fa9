"""Attention of drafted tokens over the paged cache against the fp64 oracle."""
import numpy as np
import pytest
import torch

from cache_util import Cache, bf16, random_trees, reference_attention
from oracle import cache as oc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import lossless_verification_sampling_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


@pytest.fixture(scope="module")
def dev(sv):
    return torch.device("cuda:0")


def D(x, dev):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dev)


class Case:
    def __init__(self, seed, R, M, Hq, Hkv, Dh, page, kind, ctx, tree, window=0, n=None, qs=2.0):
        g = np.random.default_rng(seed)
        self.window, self.tree, self.dims = window, tree, (R, M, Hq, Dh)
        self.ctx = np.asarray(ctx, np.int32)
        self.n = np.array([M] * R if n is None else n, np.int32)
        self.c = Cache(g, R, int((self.ctx + self.n).max()), Hkv, Dh, page, kind)
        self.q = bf16(g.standard_normal((R, M, Hq, Dh)) * qs)
        self.parent = random_trees(g, R, M, self.n)
        self.pos, self.see = oc.tree_mask(self.parent, self.n, self.ctx, window)
        if not tree:
            self.pos = self.ctx[:, None] + np.arange(M)[None, :]
        self.scale = float(np.float32(Dh ** -0.5))

    def run(self, sv, dev, **kw):
        self.c.to(dev)
        out = torch.full(self.dims, 7.0, dtype=torch.bfloat16, device=dev)
        lse = torch.full(self.dims[:3], 7.0, dtype=torch.float32, device=dev)
        m = dict(mask=D(oc.pack_bits(self.see), dev), positions=D(self.pos, dev)) if self.tree else {}
        m.update(kw)
        sv.spec_tree_attention(self.q.to(dev), *self.c.args(), D(self.ctx, dev), D(self.n, dev),
                               scale=self.scale, window=self.window, out=out, out_lse=lse,
                               **self.c.kw(), **m)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), lse.double().cpu().numpy()

    def check(self, got, rows=None):
        out, lse = got
        q = self.q.double().numpy()
        ro, rl, to, tl = reference_attention(self.c, q, self.ctx, self.n, self.see, self.pos,
                                             self.scale, self.window, not self.tree)
        M = self.dims[1]
        for r in range(self.dims[0]):
            m = int(self.n[r])
            assert (out[r, m:] == 7.0).all() and (lse[r, m:] == 7.0).all()
            for v in range(m):
                a, b = out[r, v], ro[r, v]
                assert np.array_equal(np.isnan(a), np.isnan(b)), (r, v)
                f = np.isfinite(b)
                assert (np.abs(a - b) <= to[r, v])[f].all(), (r, v, float(
                    (np.abs(a - b) / to[r, v])[f].max()))
                a, b = lse[r, v], rl[r, v]
                f = np.isfinite(b)
                assert np.array_equal(a[~f], b[~f], equal_nan=True), (r, v)
                assert (np.abs(a - b) <= tl[r, v])[f].all(), (r, v, a, b)


SHAPES = [  # R, M, Hq, Hkv, D, page, ctx, tree, window, n
    (1, 1, 1, 1, 64, 16, [0], False, 0, None),                 # itself alone
    (1, 1, 4, 1, 128, 16, [1], False, 0, None),
    (1, 1, 32, 8, 128, 64, [1023], False, 0, None),
    (1, 9, 32, 8, 128, 64, [700], True, 0, None),
    (3, 8, 8, 2, 128, 32, [31, 0, 300], False, 0, [8, 3, 0]),  # an idle slot
    (2, 48, 8, 2, 128, 32, [129, 47], True, 0, [48, 31]),
    (2, 33, 7, 1, 64, 16, [65, 200], True, 0, None),           # seven heads a key head
    (2, 70, 2, 2, 256, 64, [90, 15], True, 0, [70, 1]),
    (1, 200, 5, 1, 128, 128, [77], True, 0, None),
    (2, 100, 3, 3, 64, 16, [16, 513], False, 0, None),
    (1, 300, 1, 1, 64, 32, [0], False, 0, None),               # a prompt
    (2, 20, 4, 2, 128, 16, [500, 3], False, 17, None),         # a window inside the chain
    (2, 40, 4, 2, 64, 32, [400, 90], True, 3, None),
    (2, 5, 16, 1, 256, 16, [260, 33], True, 100, None),
    (1, 1, 8, 8, 64, 1024, [5000], False, 1, None),            # a window of one
    (5, 3, 64, 1, 128, 16, [5, 17, 1000, 64, 0], False, 0, None),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_fp64(sv, dev, shape, kind):
    R, M, Hq, Hkv, Dh, page, ctx, tree, window, n = shape
    print(f"[attn] {shape} {kind}", flush=True)
    c = Case(sum(ctx) + M, R, M, Hq, Hkv, Dh, page, kind, ctx, tree, window, n)
    c.check(c.run(sv, dev))


def test_largest_tree(sv, dev):
    c = Case(11, 1, 1024, 2, 1, 64, 64, "bf16", [130], True)
    c.check(c.run(sv, dev))


def test_long_contexts_beside_short_ones(sv, dev):
    c = Case(12, 6, 2, 4, 2, 64, 64, "e4m3", [9001, 1, 0, 33, 4097, 2], False, 0, [2, 2, 1, 2, 0, 2])
    c.check(c.run(sv, dev))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_rows_that_see_nothing(sv, dev, kind):
    c = Case(13, 2, 6, 4, 2, 128, 16, kind, [0, 40], True)
    c.see[0, 3] = False                       # no context, no node
    c.see[1, 2] = False                       # context alone
    c.see[0, 5] = False
    c.see[0, 5, 1] = True                     # not even itself
    got = c.run(sv, dev)
    assert not got[0][0, 3].any() and (got[1][0, 3] == -np.inf).all()
    c.check(got)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf, float(np.finfo(np.float32).max)])
def test_unseen_tokens_have_no_part(sv, dev, tree, value):
    """A node's K and V rows hold NaN, infinities or the type's largest value:
    rows that do not see the node are as if it were not there."""
    M = 20
    c = Case(14, 1, M, 4, 2, 64, 16, "bf16", [37], tree)
    if tree:
        c.see[0, :, 7] = False                # nobody sees node 7
        c.see[0, 9] = False
        c.see[0, 9, :7] = True
    clean = Case(14, 1, M, 4, 2, 64, 16, "bf16", [37], tree)
    clean.see = c.see
    t = 37 + (7 if tree else M - 1)           # the chain's last token
    pg, off = int(c.c.table[0, t // 16]), t % 16
    for x in c.c.dev:
        x[pg, :, off] = value
    a, b = c.run(sv, dev), clean.run(sv, dev)
    seen = M if tree else M - 1
    np.testing.assert_array_equal(a[0][:, :seen], b[0][:, :seen])
    np.testing.assert_array_equal(a[1][:, :seen], b[1][:, :seen])
    assert np.isfinite(a[0][:, :seen]).all()


def test_seen_infinities_follow_the_formula(sv, dev):
    c = Case(15, 1, 8, 2, 1, 64, 16, "bf16", [50], True)
    k, v = c.c.dev
    at = lambda t: (int(c.c.table[0, t // 16]), 0, t % 16)  # noqa: E731
    v[at(50 + 3)][5] = np.inf                 # its descendants' d = 5 becomes inf
    v[at(20)][9] = np.nan                     # everybody's d = 9
    out, lse = c.run(sv, dev)
    below = c.see[0, :, 3]
    assert (out[0, below, :, 5] == np.inf).all() and np.isfinite(out[0, ~below][..., 5]).all()
    assert np.isnan(out[0, ..., 9]).all()
    rest = np.delete(out[0], [5, 9], -1)
    assert np.isfinite(rest).all() and np.isfinite(lse).all()


def test_garbage_behind_the_last_token(sv, dev):
    c = Case(16, 2, 5, 4, 1, 128, 32, "bf16", [40, 3], False)
    c.run(sv, dev)
    for r, L in ((0, 45), (1, 8)):
        pg = int(c.c.table[r, L // 32])
        for x in c.c.dev:
            x[pg, :, L % 32:] = float("nan")
    c.check(c.run(sv, dev))


def test_far_scores(sv, dev):
    """Scores in the thousands: one token takes all the weight."""
    c = Case(17, 1, 4, 4, 1, 128, 16, "bf16", [300], False, qs=300.0)
    c.check(c.run(sv, dev))


@pytest.mark.parametrize("fault", ["n_high", "n_negative", "ctx", "past", "page", "position"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_faults(sv, dev, fault, kind):
    c = Case(18, 3, 6, 4, 2, 64, 16, kind, [30, 40, 9], True)
    good = c.run(sv, dev)
    if fault == "n_high":
        c.n[1] = 7
    elif fault == "n_negative":
        c.n[1] = -1
    elif fault == "ctx":
        c.ctx[1] = -1
    elif fault == "past":
        c.ctx[1] = 43
    elif fault == "page":
        c.c.table[1, 2] = c.c.P               # tokens 32 .. 47
    else:
        c.pos[1, 4] = -1
    ws = sv.Workspace(dev, sv.spec_tree_attention_workspace_bytes(3, 6, 4, 2, 64))
    out, lse = c.run(sv, dev, workspace=ws)
    assert sv.spec_get_device_status(ws) == sv.SPEC_DEV_BAD_REQUEST
    rows = [4] if fault == "position" else list(range(6))
    assert np.isnan(out[1, rows]).all() and np.isnan(lse[1, rows]).all()
    rest = [i for i in range(6) if i not in rows]
    for a, b in ((out, good[0]), (lse, good[1])):
        np.testing.assert_allclose(a[[0, 2]], b[[0, 2]], rtol=2.0 ** -7, atol=1e-6)
        np.testing.assert_allclose(a[1, rest], b[1, rest], rtol=2.0 ** -7, atol=1e-6)
    assert sv.spec_get_device_status(ws) == 0


def test_same_call_same_bits(sv, dev):
    c = Case(19, 4, 12, 8, 2, 128, 16, "e4m3", [1000, 20, 300, 5], True)
    a, b = c.run(sv, dev), c.run(sv, dev)
    np.testing.assert_array_equal(a[0], b[0])
    np.testing.assert_array_equal(a[1], b[1])


# rows per key head: 8, 30 and 16 (waves divide the tokens), 96, 192 and 80 (waves divide the rows)
@pytest.mark.parametrize("M,G,Dh", [(8, 1, 64), (30, 1, 128), (8, 2, 256), (48, 2, 64), (64, 3, 128), (20, 4, 256)])
@pytest.mark.parametrize("what,value", [("k_scale", np.nan), ("k_scale", np.inf), ("v_scale", np.nan),
                                        ("v_scale", np.inf), ("codes", np.nan)])
def test_unseen_scales_and_codes(sv, dev, M, G, Dh, what, value):
    """e4m3: a token's scales or codes are no numbers.  Rows that do not see it
    are as if it were not there; what the others give is the formula's."""
    bad, dirty = 3, Case(20, 1, M, G, 1, Dh, 16, "e4m3", [37], True)
    clean = Case(20, 1, M, G, 1, Dh, 16, "e4m3", [37], True)
    at = int(dirty.c.table[0, (37 + bad) // 16]), 0, (37 + bad) % 16
    if what == "codes":
        for x in dirty.c.dev:
            x.view(torch.uint8)[at] = 0x7f
    else:
        dirty.c.scales[what == "v_scale"][at] = value
    got, good = dirty.run(sv, dev), clean.run(sv, dev)
    blind = ~dirty.see[0, :, bad]
    assert blind.any() and not blind.all()
    for a, b in zip(got, good):
        np.testing.assert_array_equal(a[0, blind], b[0, blind])
    seeing = got[0][0, ~blind]
    if what == "v_scale" and value == np.inf:  # inf times a code: its sign, or NaN for 0
        code = dirty.c.dev[1][at].float().cpu().numpy()
        with np.errstate(invalid="ignore"):
            assert np.array_equal(seeing, np.broadcast_to(code * np.inf, seeing.shape), equal_nan=True)
    elif what == "k_scale" and value == np.inf:
        assert not np.isnan(got[1][0, blind]).any()
    else:
        assert np.isnan(seeing).all()
    if what == "v_scale":                     # the scores have nothing of it
        np.testing.assert_array_equal(got[1], good[1])


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("M,G", [(6, 2), (40, 2)])
def test_largest_window_and_position(sv, dev, tree, M, G):
    """2^31 - 1 is as good as no window; a position of 2^31 - 1 is behind every
    token by more than a small window."""
    c = Case(21, 1, M, 2 * G, 2, 64, 16, "bf16", [100], tree)
    free = c.run(sv, dev)
    c.window = 2 ** 31 - 1
    for a, b in zip(c.run(sv, dev), free):
        np.testing.assert_array_equal(a, b)
    c.window = 5
    far = np.full(c.pos.shape, 2 ** 31 - 1, np.int32)
    got = c.run(sv, dev, positions=D(far, dev))
    c.pos = far.astype(np.int64)
    c.check(got)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", [
    (1, 30, 8, 2, 128, 32, [150], True, 0, None),               # 120 rows: two tiles a wave
    (2, 24, 8, 2, 128, 64, [9000, 5], True, 0, [24, 9]),        # an item in many parts, many rows
    (2, 24, 6, 1, 256, 128, [5000, 0], False, 900, None),
    (1, 70, 9, 3, 64, 16, [3001], True, 40, None),
    (4, 1, 8, 8, 64, 64, [9000, 8900, 9000, 8999], False, 0, None),  # units for two ranges a compute unit
    (3, 8, 4, 1, 128, 16, [2000, 1, 700], False, 0, [8, 8, 5]),  # 32 rows
])
def test_splits_and_joins(sv, dev, shape, kind):
    R, M, Hq, Hkv, Dh, page, ctx, tree, window, n = shape
    print(f"[attn] {shape} {kind}", flush=True)
    c = Case(sum(ctx) + M, R, M, Hq, Hkv, Dh, page, kind, ctx, tree, window, n)
    c.check(c.run(sv, dev))


def ragged(R, top, seed):
    g = np.random.default_rng(seed)
    return [int(x) for x in g.integers(0, top, R)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", [                             # batches of more than 12288 rows
    (33, 48, 16, 4, 128, 32, ragged(33, 300, 1), True, 0, ragged(33, 49, 2)),   # three tiles a wave
    (40, 64, 8, 2, 128, 16, ragged(40, 200, 3), True, 30, None),                # two
    (70, 100, 4, 2, 64, 64, ragged(70, 130, 4), False, 0, ragged(70, 101, 5)),  # three, D = 64
    (60, 33, 21, 3, 64, 32, ragged(60, 500, 6), False, 77, None),               # two, D = 64
    (30, 10, 128, 2, 256, 16, ragged(30, 90, 7), True, 0, None),                # one, D = 256
    (1, 1024, 16, 2, 64, 128, [1100], False, 0, None),                          # few items in many parts
])
def test_large_batches(sv, dev, shape, kind):
    R, M, Hq, Hkv, Dh, page, ctx, tree, window, n = shape
    print(f"[attn] {shape} {kind}", flush=True)
    c = Case(sum(ctx) + M, R, M, Hq, Hkv, Dh, page, kind, ctx, tree, window, n)
    c.check(c.run(sv, dev))


@pytest.mark.parametrize("what,value", [("none", 0.0), ("v_scale", np.nan), ("codes", np.nan)])
def test_unseen_in_large_batches(sv, dev, what, value):
    R, M, bad = 30, 48, 3
    a, b = [Case(22, R, M, 12, 3, 128, 16, "e4m3", [37] * R, True) for _ in range(2)]
    for r in range(R):
        at = int(a.c.table[r, (37 + bad) // 16]), 1, (37 + bad) % 16
        if what == "v_scale":
            a.c.scales[1][at] = value
        elif what == "codes":
            a.c.dev[1].view(torch.uint8)[at] = 0x7f
    got, good = a.run(sv, dev), b.run(sv, dev)
    for r in range(R):
        blind = ~a.see[r, :, bad]
        for x, y in zip(got, good):
            np.testing.assert_array_equal(x[r, blind], y[r, blind])
        if what != "none":
            assert np.isnan(got[0][r, ~blind, 4:8]).all()
            np.testing.assert_array_equal(got[0][r, ~blind, :4], good[0][r, ~blind, :4])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("ctx,window", [(20, 5), (40, 34), (64, 34), (70, 50), (93, 63)])
def test_a_far_position_beside_others(sv, dev, kind, ctx, window):
    """One node's position is 2^31 - 1, the others' are ordinary; the context's
    first tokens are out of everybody's window."""
    c = Case(23, 1, 40, 4, 2, 64, 16, kind, [ctx], True, window)
    c.pos = c.pos.copy()
    c.pos[0, 7] = 2 ** 31 - 1
    c.check(c.run(sv, dev))


@pytest.mark.parametrize("M,G", [(8, 2), (40, 2)])
@pytest.mark.parametrize("ctx", [0, 300, 5000])
def test_scores_of_minus_infinity(sv, dev, M, G, ctx):
    """Every score is -inf: the row is 0, whatever V holds."""
    c = Case(24, 1, M, G, 1, 64, 16, "bf16", [ctx], False)
    c.q[..., 5] = c.q[..., 5].abs() + 1
    c.c.dev[0][..., 5] = -float("inf")
    c.c.dev[1][..., 9] = float("inf")
    out, lse = c.run(sv, dev)
    assert not out.any() and (lse == -np.inf).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("M,G", [(8, 2), (40, 2)])
@pytest.mark.parametrize("ctx,window", [(69, 20), (79, 32), (500, 21)])
def test_pages_before_the_window_are_not_looked_at(sv, dev, kind, tree, M, G, ctx, window):
    """Pages of 16 tokens that lie before token ctx - window + 1 were given back."""
    c = Case(25, 1, M, G, 1, 64, 16, kind, [ctx], tree, window)
    c.c.table[0, :(ctx - window + 1) // 16] = -1
    ws = sv.Workspace(dev, sv.spec_tree_attention_workspace_bytes(1, M, G, 1, 64))
    got = c.run(sv, dev, workspace=ws)
    assert sv.spec_get_device_status(ws) == 0
    c.check(got)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,G,Dh", [(6, 2, 128), (1, 1, 64), (40, 2, 64), (30, 4, 256)])
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.5])
def test_scales_of_any_sign(sv, dev, kind, M, G, Dh, scale):
    c = Case(26, 2, M, 2 * G, 2, Dh, 32, kind, [90, 5], M > 1)
    c.scale = float(np.float32(scale))
    c.check(c.run(sv, dev))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,G,ctx", [(1, 4, 2003), (8, 2, 2003), (30, 4, 1990)])
def test_every_row_of_v_counts(sv, dev, kind, M, G, ctx):
    """Token t's V row has one positive value, in dimension t mod 64: a value of
    the output is the sum of some 31 weights, and nothing cancels, so a bound
    relative to the value itself (two bf16 roundings) shows one wrong row."""
    c = Case(27, 1, M, G, 1, 64, 16, kind, [ctx], False, qs=0.02)
    t = np.arange(ctx + M)
    v = np.zeros((ctx + M, 64), np.float32)
    v[t, t % 64] = 1 + (t * 37 % 101) / 101
    pg, off = c.c.table[0, t // 16], t % 16
    if kind == "bf16":
        c.c.dev[1][pg, 0, off] = bf16(v)
    else:
        codes, s = oc.quantise(v)
        c.c.dev[1].view(torch.uint8)[pg, 0, off] = torch.from_numpy(codes.astype(np.float32)).to(
            torch.float8_e4m3fn).view(torch.uint8)
        c.c.scales[1][pg, 0, off] = torch.from_numpy(s)
    c.check(c.run(sv, dev))                   # whose bound is |o| (2^-7 + less than 2^-9) here
    s = (c.c.rows(0, 0, 0, ctx + M)[:, 0] @ c.q[0, -1, 0].double().numpy()) * c.scale
    w = np.exp(s) * v.sum(-1)                 # the last node sees every token
    whole = np.array([w[t % 64 == d].sum() for d in range(64)])
    assert (w / whole[t % 64]).min() > 2.0 ** -7 + 2.0 ** -9


@pytest.mark.parametrize("M", [2, 20])
def test_many_idle_requests(sv, dev, M):
    """A padded batch: a few live requests among 30000."""
    R, live = 30000, [0, 1, 77, 15000, 29998]
    c = Case(28, len(live), M, 4, 2, 64, 16, "bf16", [100, 3, 0, 250, 40], False)
    c.c.to(dev)
    q = torch.zeros(R, M, 4, 64, dtype=torch.bfloat16, device=dev)
    table = torch.full((R, c.c.wide), -1, dtype=torch.int32, device=dev)
    n, ctx = torch.zeros(R, dtype=torch.int32, device=dev), torch.zeros(R, dtype=torch.int32, device=dev)
    at = torch.tensor(live, device=dev)
    q[at], table[at], n[at], ctx[at] = c.q.to(dev), c.c.t, M, D(c.ctx, dev)
    out = torch.full_like(q, 7.0)
    lse = torch.full((R, M, 4), 7.0, device=dev)
    ws = sv.Workspace(dev, sv.spec_tree_attention_workspace_bytes(R, M, 4, 2, 64))
    sv.spec_tree_attention(q, c.c.dev[0], c.c.dev[1], table, ctx, n, out=out, out_lse=lse, workspace=ws)
    assert sv.spec_get_device_status(ws) == 0
    c.check((out[at].double().cpu().numpy(), lse[at].double().cpu().numpy()))
    idle = torch.ones(R, dtype=torch.bool, device=dev)
    idle[at] = False
    assert (out[idle] == 7).all() and (lse[idle] == 7).all()
