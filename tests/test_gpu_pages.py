"""Key bounds of cache pages, page lists and attention over them against the
fp64 oracle."""
import numpy as np
import pytest
import torch

from cache_util import BF16_U, Cache, bf16, random_trees, reference_attention
from oracle import cache as oc
from oracle import pages as op

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import lossless_verification_sampling_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.spec_get_device_status(m.default_workspace("cuda:0"))     # what other files' faulty calls left
    return m


@pytest.fixture(scope="module")
def dev(sv):
    return torch.device("cuda:0")


def D(x, dev):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dev)


def status(sv):
    return sv.spec_get_device_status(sv.default_workspace("cuda:0"))


# ---------------------------------------------------------------------------
# bounds
# ---------------------------------------------------------------------------

def run_bounds(sv, dev, c, start, n, max_len, fill=7.0):
    c.to(dev)
    box = [torch.full((c.P, c.Hkv, c.D), fill, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    sv.spec_page_bounds(c.dev[0], c.t, D(np.int32(start), dev), D(np.int32(n), dev), max_len, *box,
                        k_scale=c.scales[0])
    torch.cuda.synchronize()
    return [b.double().cpu().numpy() for b in box]


def check_bounds(c, got, start, n, skip=(), fill=7.0):
    """bf16 values are exact; a code times its scale is rounded to fp32 (2^-24)
    and to bf16 (half a step)."""
    seen = set()
    for r in range(len(start)):
        if n[r] == 0 or r in skip:
            continue
        for i in range(start[r] // c.page, (start[r] + n[r] - 1) // c.page + 1):
            first = i * c.page
            count = min(c.page, start[r] + n[r] - first)
            want = op.bounds(c.rows(0, r, first, count))
            p = int(c.table[r, i])
            seen.add(p)
            for a, b in zip(got, want):
                f = np.isfinite(b)
                assert np.array_equal(a[p][~f], b[~f], equal_nan=True)
                tol = np.abs(b[f]) * (BF16_U + 2.0 ** -23) if c.kind == "e4m3" else 0.0
                assert (np.abs(a[p][f] - b[f]) <= tol).all()
    for p in set(range(c.P)) - seen:
        assert (got[0][p] == fill).all() and (got[1][p] == fill).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", [  # Hkv, D, page, starts, lengths
    (1, 64, 16, [0], [1]),
    (8, 128, 16, [15, 16, 3], [1, 17, 0]),
    (2, 128, 32, [31, 0, 100], [2, 200, 33]),
    (3, 256, 64, [5, 64], [60, 64]),
    (5, 64, 128, [0, 127, 300], [128, 2, 1]),
    (2, 128, 1024, [1000, 5], [1500, 700]),
    (1, 256, 1024, [0], [1024]),
])
def test_bounds_against_fp64(sv, dev, shape, kind):
    Hkv, Dh, page, start, n = shape
    print(f"[bounds] {shape} {kind}", flush=True)
    g = np.random.default_rng(sum(start) + Dh)
    c = Cache(g, len(start), int(max(s + m for s, m in zip(start, n))), Hkv, Dh, page, kind)
    check_bounds(c, run_bounds(sv, dev, c, start, n, max(n) + 3), start, n)
    assert status(sv) == 0


@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_bounds_of_nan_and_infinity(sv, dev, kind, page):
    g = np.random.default_rng(4)
    c = Cache(g, 1, 2 * page, 2, 64, page, kind)
    p = int(c.table[0, 0])
    if kind == "bf16":
        c.dev[0][p, 0, 3, 5] = float("nan")
        c.dev[0][p, 1, 2, 9] = float("inf")
        c.dev[0][p, 1, 7, 9] = float("-inf")
    else:
        c.scales[0][p, 0, 3] = float("nan")             # a row that held a NaN
        c.dev[0][p, 0, 3] = torch.zeros(64).to(torch.float8_e4m3fn)
    got = run_bounds(sv, dev, c, [0], [2 * page], 2 * page)
    check_bounds(c, got, [0], [2 * page])
    assert np.isnan(got[0][p, 0]).sum() == (1 if kind == "bf16" else 64)


def test_bounds_data_faults(sv, dev):
    g = np.random.default_rng(5)
    c = Cache(g, 6, 64, 2, 64, 16, "bf16")
    start, n = [0, -1, 60, 3, 0, 2147483647], [20, 5, 5, -1, 30, 3]
    c.table[0, 1] = 10 ** 6                             # passed over
    kept = c.table.copy()
    got = run_bounds(sv, dev, c, start, n, 20)
    assert status(sv) == sv.SPEC_DEV_BAD_REQUEST
    c.table = kept[:1, :1]
    check_bounds(c, got, [0], [16])
    c.table = kept


def test_bounds_of_a_pool_past_32_bits(sv, dev):
    """Pages whose byte offsets pass 2^32."""
    P, Hkv, page, Dh = 70000, 8, 64, 64
    k = torch.zeros(P, Hkv, page, Dh, dtype=torch.bfloat16, device=dev)
    k[P - 1, 7, 63, 11] = 5.0
    k[P - 1, 7, 62, 11] = -6.0
    box = [torch.zeros(P, Hkv, Dh, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    i32 = dict(dtype=torch.int32, device=dev)
    sv.spec_page_bounds(k, torch.tensor([[P - 1]], **i32), torch.tensor([0], **i32), torch.tensor([64], **i32), 64,
                        *box)
    assert box[0][P - 1, 7, 11] == -6.0 and box[1][P - 1, 7, 11] == 5.0
    assert box[0].abs().sum() == 6.0 and box[1].abs().sum() == 5.0


# ---------------------------------------------------------------------------
# lists
# ---------------------------------------------------------------------------

class Lists:
    """A step's queries, page tables and bounds."""

    def __init__(self, seed, R, M, Hq, Hkv, Dh, page, ctx, budget, first=0, last=0, n=None):
        g = np.random.default_rng(seed)
        self.ctx, self.page = np.asarray(ctx, np.int32), page
        self.n = np.array([M] * R if n is None else n, np.int32)
        wide = max(1, -(-int((self.ctx + self.n).max()) // page))
        self.P = R * wide + 2
        self.table = g.permutation(self.P)[:R * wide].reshape(R, wide).astype(np.int32)
        self.q = bf16(g.standard_normal((R, M, Hq, Dh)) * 2)
        mid = g.standard_normal((self.P, Hkv, Dh))
        self.lo, self.hi = bf16(mid - g.random(mid.shape)), bf16(mid + g.random(mid.shape))
        self.budget, self.first, self.last = budget, first, last

    def run(self, sv, dev, **kw):
        got = sv.spec_page_select(self.q.to(dev), self.lo.to(dev), self.hi.to(dev), D(self.table, dev),
                                  D(self.ctx, dev), D(self.n, dev), self.budget, self.page, first=self.first,
                                  last=self.last, **kw)
        torch.cuda.synchronize()
        return [x.cpu().numpy() for x in got]

    def want(self, width):
        return op.select(self.q.double().numpy(), self.lo.double().numpy(), self.hi.double().numpy(), self.table,
                         self.ctx, self.n, self.budget, self.page, self.first, self.last, width)

    def check(self, got):
        lists, length = self.want(got[0].shape[2])
        assert np.array_equal(got[1], length), (got[1], length)
        assert np.array_equal(got[0], lists), np.argwhere(got[0] != lists)[:5]


@pytest.mark.parametrize("shape", [  # R, M, Hq, Hkv, D, page, ctx, budget, first, last, n
    (1, 1, 1, 1, 64, 16, [0], 3, 0, 0, None),                       # nothing to choose
    (1, 1, 4, 1, 128, 16, [16], 1, 0, 0, None),
    (1, 1, 4, 1, 128, 16, [47], 1, 0, 0, None),
    (1, 1, 32, 8, 128, 16, [3001], 20, 1, 2, None),
    (3, 1, 8, 2, 64, 32, [1000, 63, 0], 5, 0, 1, None),
    (2, 1, 6, 2, 256, 16, [700, 333], 7, 3, 4, None),               # forced pages alone
    (2, 5, 8, 2, 128, 16, [900, 41], 6, 1, 0, [5, 0]),              # rows summed beforehand; an idle slot
    (2, 40, 8, 1, 256, 64, [2000, 1500], 4, 0, 0, [40, 33]),
    (1, 1, 8, 8, 64, 16, [1600], 0, 0, 0, None),                    # no full page at all
    (1, 3, 2, 2, 128, 1024, [5000], 2, 0, 0, None),
    (1, 1, 1, 1, 64, 16, [80000], 100, 1, 1, None),                 # more pages than shared memory holds
    (1, 1, 2, 1, 128, 16, [65551], 4096, 0, 0, None),               # one page fewer than there are
    (1, 1, 2, 1, 128, 16, [65536], 4095, 0, 0, None),
])
def test_lists_against_fp64(sv, dev, shape):
    R, M, Hq, Hkv, Dh, page, ctx, budget, first, last, n = shape
    print(f"[lists] {shape}", flush=True)
    s = Lists(sum(ctx) + Dh, R, M, Hq, Hkv, Dh, page, ctx, budget, first, last, n)
    s.check(s.run(sv, dev))
    assert status(sv) == 0


@pytest.mark.parametrize("budget", [1, 2, 5, 17, 31])
def test_equal_scores_take_the_lower_pages(sv, dev, budget):
    s = Lists(21, 2, 1, 4, 2, 64, 16, [16 * 40 + 3, 16 * 33], budget)
    same = s.table[:, 2:38:3][:, :11]                               # many alike, one a little better
    s.lo[torch.from_numpy(same).long()], s.hi[torch.from_numpy(same).long()] = -1.0, 1.0
    s.lo[int(s.table[0, 20])] = -1.0
    s.hi[int(s.table[0, 20])] = 1.0078125
    s.check(s.run(sv, dev))
    s.lo[:], s.hi[:] = -0.5, 0.25                                   # all alike
    s.check(s.run(sv, dev))
    s.q[:] = 0.0                                                    # zeros of either sign
    s.lo[::2], s.hi[::3] = 0.5, -0.25
    s.check(s.run(sv, dev))


@pytest.mark.parametrize("budget, first, last", [(1, 0, 0), (4, 1, 2), (30, 0, 1), (149, 0, 0)])
@pytest.mark.parametrize("F", [150, 4200])                          # keys in shared memory, and not
def test_scores_that_differ_in_their_last_bits(sv, dev, F, budget, first, last):
    """1 + i 2^-52, or far below: neighbours in fp64, whose keys differ in the lowest
    bits, in a range that has to be narrowed several times."""
    s = Lists(25, 1, 1, 1, 1, 64, 16, [16 * F], budget, first, last)
    i = np.random.default_rng(F).permutation(F) % 256
    s.q[:], s.lo[:], s.hi[:] = 0.0, 0.0, 0.0
    s.q[..., 3], s.q[..., 40] = 1.0, 2.0 ** -52
    at = torch.from_numpy(s.table[0, :F]).long()
    s.hi[at, 0, 3], s.hi[at, 0, 40] = 1.0, torch.from_numpy(i.astype(np.float32)).to(torch.bfloat16)
    s.check(s.run(sv, dev))
    s.hi[at[i < 200], 0, 3] = 0.5
    s.check(s.run(sv, dev))


def test_scores_that_are_no_numbers(sv, dev):
    s = Lists(22, 1, 1, 2, 1, 64, 16, [16 * 30], 4)
    t = s.table[0]
    s.hi[int(t[9]), 0, 3] = float("nan")
    s.hi[int(t[4]), 0, 3] = float("inf")
    s.lo[int(t[4]), 0, 3] = float("-inf")
    s.hi[int(t[2])], s.lo[int(t[2])] = float("-inf"), float("inf")
    got = s.run(sv, dev)
    assert {int(t[9]), int(t[4])} < set(got[0][0, 0].tolist())
    s.check(got)
    s.q[0, 0, 1, 5] = float("nan")                                  # every score: the lowest pages
    got = s.run(sv, dev)
    assert got[0][0, 0, :4].tolist() == t[:4].tolist()
    s.check(got)


@pytest.mark.parametrize("budget, first, last", [(1, 0, 0), (4, 0, 0), (4, 1, 1), (9, 2, 3), (12, 0, 0), (29, 0, 2)])
@pytest.mark.parametrize("F", [30, 4200])                           # keys in shared memory, and not
@pytest.mark.parametrize("kind", ["nan", "inf", "query"])
def test_more_infinite_scores_than_places(sv, dev, kind, F, budget, first, last):
    """Beside negative scores and -infinity the keys' range is wider than 2^63."""
    s = Lists(26, 2, 2, 4, 2, 64, 16, [16 * F, 16 * F - 5], budget, first, last)
    g = np.random.default_rng(F + budget)
    t = torch.from_numpy(s.table[:, g.permutation(F)]).long()
    many, some = t[:, :10 if F < 100 else 2000].flatten(), t[:, -7:].flatten()
    print(f"[infinite] {kind} {F} {budget} {first} {last}", flush=True)
    if kind != "query":                                             # scores by the largest values' sign
        s.q = s.q.abs()
        s.hi[::3] = -s.hi[::3].abs()
    if kind == "nan":
        s.lo[many, :, 9] = float("nan")
    elif kind == "inf":
        s.hi[many, :, 9] = float("inf")
        s.hi[some, :, 9] = float("-inf")
    else:                                                           # by the sign of the bound
        s.q[:, 0, ::2, 11] = float("inf")
        s.hi[..., 11] = -s.hi[..., 11].abs()
        s.hi[many, :, 11] = s.hi[many, :, 11].abs()
        s.lo[..., 11] = -2.0
    s.check(s.run(sv, dev))
    assert status(sv) == 0


def test_list_data_faults(sv, dev):
    s = Lists(23, 7, 3, 4, 2, 64, 16, [200, 200, 200, 200, 200, 200, 200], 5)
    s.ctx[1], s.ctx[2] = -1, 210                                    # past the table with its nodes
    s.n[3], s.n[4] = -1, 4
    s.table[5, 3], s.table[6, 12] = -1, s.P                         # a full page; the end's
    s.check(s.run(sv, dev))
    assert status(sv) == sv.SPEC_DEV_BAD_REQUEST


def test_list_outputs_of_another_width(sv, dev):
    s = Lists(24, 2, 2, 4, 2, 64, 16, [300, 20], 50, 1, 1)
    wide = torch.full((2, 2, 70), 7, dtype=torch.int32, device=dev)
    got = s.run(sv, dev, out_lists=wide, out_len=torch.full((2,), 7, dtype=torch.int32, device=dev))
    assert (got[0][:, :, 55:] == -1).all()
    s.check(got)


# ---------------------------------------------------------------------------
# attention over lists
# ---------------------------------------------------------------------------

class Attend:
    def __init__(self, seed, R, M, Hq, Hkv, Dh, page, kind, ctx, budget, tree, n=None):
        g = np.random.default_rng(seed)
        self.dims, self.tree = (R, M, Hq, Dh), tree
        self.n = np.array([M] * R if n is None else n, np.int32)
        ctx = np.asarray(ctx, np.int32)
        self.c = Cache(g, R, int((ctx + self.n).max()), Hkv, Dh, page, kind)
        self.q = bf16(g.standard_normal(self.dims) * 2)
        self.parent = random_trees(g, R, M, self.n)
        self.see = oc.tree_mask(self.parent, self.n, ctx, 0)[1]
        width = budget + (M + page - 2) // page + 2
        self.lists = np.full((R, Hkv, width), -1, np.int32)
        self.length = np.zeros(R, np.int32)
        for r in range(R):
            F = int(ctx[r]) // page
            tail = self.c.table[r, F:-(-int(ctx[r] + self.n[r]) // page)]
            take = min(F, budget)
            for h in range(Hkv):
                own = np.sort(g.choice(F, take, replace=False)) if take else []
                row = np.concatenate([self.c.table[r, own].astype(np.int32) if take else [], tail])
                self.lists[r, h, :len(row)] = row
            self.length[r] = take * page + ctx[r] % page
        self.scale = float(np.float32(Dh ** -0.5))

    def run(self, sv, dev, **kw):
        self.c.to(dev)
        out = torch.full(self.dims, 7.0, dtype=torch.bfloat16, device=dev)
        lse = torch.full(self.dims[:3], 7.0, dtype=torch.float32, device=dev)
        if self.tree:
            kw.update(mask=D(oc.pack_bits(self.see), dev))
        sv.spec_page_attention(self.q.to(dev), self.c.dev[0], self.c.dev[1], D(self.lists, dev), D(self.length, dev),
                               D(self.n, dev), scale=self.scale, out=out, out_lse=lse, **self.c.kw(), **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, got):
        out, lse = (x.double().cpu().numpy() for x in got)
        R, M, Hq, Dh = self.dims
        G = Hq // self.c.Hkv
        for h in range(self.c.Hkv):                                 # a head's cache by its list
            one = Cache.__new__(Cache)
            one.page, one.kind, one.P, one.Hkv, one.D = self.c.page, self.c.kind, self.c.P, 1, Dh
            one.table = self.lists[:, h]
            one.dev = [x[:, h:h + 1].cpu() for x in self.c.dev]
            one.scales = [None if x is None else x[:, h:h + 1].cpu() for x in self.c.scales]
            sl = slice(h * G, (h + 1) * G)
            pos = self.length[:, None] + np.arange(M)[None, :]
            ro, rl, to, tl = reference_attention(one, self.q.double().numpy()[:, :, sl], self.length, self.n, self.see,
                                                 pos, self.scale, 0, not self.tree)
            for r in range(R):
                m = int(self.n[r])
                assert (out[r, m:] == 7.0).all() and (lse[r, m:] == 7.0).all()
                assert (np.abs(out[r, :m, sl] - ro[r, :m]) <= to[r, :m]).all(), (h, r)
                assert (np.abs(lse[r, :m, sl] - rl[r, :m]) <= tl[r, :m]).all(), (h, r)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", [  # R, M, Hq, Hkv, D, page, ctx, budget, tree, n
    (1, 1, 1, 1, 64, 16, [0], 2, False, None),
    (1, 1, 8, 2, 128, 16, [1000], 9, False, None),
    (3, 1, 32, 8, 128, 32, [500, 31, 64], 4, False, [1, 1, 0]),
    (2, 6, 12, 4, 64, 16, [333, 200], 11, True, [6, 3]),
    (2, 20, 10, 2, 128, 16, [450, 90], 7, True, None),
    (1, 60, 4, 2, 256, 64, [700], 3, False, None),
    (2, 30, 24, 3, 64, 32, [900, 257], 8, True, None),
    (1, 2, 128, 2, 128, 1024, [3000], 1, False, None),
])
def test_attention_against_fp64(sv, dev, shape, kind):
    R, M, Hq, Hkv, Dh, page, ctx, budget, tree, n = shape
    print(f"[page attn] {shape} {kind}", flush=True)
    a = Attend(sum(ctx) + M, R, M, Hq, Hkv, Dh, page, kind, ctx, budget, tree, n)
    a.check(a.run(sv, dev))
    assert status(sv) == 0


@pytest.mark.parametrize("M", [1, 12, 80])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_lists_of_every_page_are_the_tree_attention(sv, dev, kind, M):
    """Bit for bit."""
    a = Attend(31, 2, M, 8, 2, 128, 16, kind, [300, 77], 100, True)
    got = a.run(sv, dev)
    pos = D((np.array([300, 77], np.int32)[:, None] + np.zeros((1, M), np.int32)).astype(np.int32), dev)
    want = sv.spec_tree_attention(a.q.to(dev), a.c.dev[0], a.c.dev[1], a.c.t,
                                  D(np.array([300, 77], np.int32), dev), D(a.n, dev),
                                  mask=D(oc.pack_bits(a.see), dev), positions=pos, scale=a.scale, want_lse=True,
                                  **a.c.kw())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_data_faults(sv, dev):
    a = Attend(32, 4, 2, 4, 2, 64, 16, "bf16", [100, 100, 100, 100], 3, False)
    a.length[1] = -1                                                # as a faulty request's
    a.lists[2, 1, 1] = a.c.P                                        # one key head's page
    a.length[3] = a.lists.shape[2] * 16                             # past its list
    out, lse = a.run(sv, dev)
    assert status(sv) == sv.SPEC_DEV_BAD_REQUEST
    bad = torch.isnan(lse).cpu().numpy()
    want = np.zeros((4, 2, 4), bool)
    want[1], want[3], want[2, :, 2:] = True, True, True
    assert np.array_equal(bad, want) and np.array_equal(torch.isnan(out).all(-1).cpu().numpy(), want)


# ---------------------------------------------------------------------------
# a drafting step
# ---------------------------------------------------------------------------

class Step:
    """qkv write, bounds, lists and attention of one layer, on buffers that
    stay."""

    def __init__(self, sv, dev, seed, kind):
        g = np.random.default_rng(seed)
        self.sv, self.R, self.M, self.Hq, self.Hkv, self.Dh, self.page = sv, 3, 2, 4, 2, 64, 16
        self.ctx = np.array([400, 95, 16], np.int32)
        self.c = Cache(g, self.R, 500, self.Hkv, self.Dh, self.page, kind).to(dev)
        self.box = [torch.zeros(self.c.P, self.Hkv, self.Dh, dtype=torch.bfloat16, device=dev) for _ in range(2)]
        self.x = torch.zeros(self.R, self.M, self.Hq + 2 * self.Hkv, self.Dh, dtype=torch.bfloat16, device=dev)
        self.at, self.n = D(self.ctx, dev), D(np.array([2, 2, 1], np.int32), dev)
        self.ws = sv.Workspace(dev, 1 << 22)
        sv.spec_page_bounds(self.c.dev[0], self.c.t, torch.zeros_like(self.at), self.at, 400, *self.box,
                            k_scale=self.c.scales[0], workspace=self.ws)

    def inputs(self, seed):
        return bf16(np.random.default_rng(seed).standard_normal(self.x.shape)).to(self.x.device)

    def run(self, stream=None):
        sv, h, k = self.sv, self.Hq, self.Hkv
        how = dict(workspace=self.ws, stream=stream)
        q = sv.spec_qkv_write(self.x[:, :, h:h + k], self.x[:, :, h + k:], *self.c.dev, self.c.t, self.at, self.n,
                              q=self.x[:, :, :h], **self.c.kw(), **how)
        sv.spec_page_bounds(self.c.dev[0], self.c.t, self.at, self.n, self.M, *self.box, k_scale=self.c.scales[0],
                            **how)
        lists, length = sv.spec_page_select(q, *self.box, self.c.t, self.at, self.n, 6, self.page, first=1, last=1,
                                            **how)
        out, lse = sv.spec_page_attention(q, *self.c.dev, lists, length, self.n, want_lse=True, **self.c.kw(), **how)
        return q, lists, length, out, lse


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_drafting_step(sv, dev, kind):
    s = Step(sv, dev, 41, kind)
    s.x.copy_(s.inputs(1))
    q, lists, length, out, lse = s.run()
    torch.cuda.synchronize()
    n = s.n.cpu().numpy()
    for r in range(s.R):                                            # every page's bounds are up to date
        c = s.c
        for i in range(-(-int(s.ctx[r] + n[r]) // s.page)):
            want = op.bounds(c.rows(0, r, i * s.page, min(s.page, int(s.ctx[r] + n[r]) - i * s.page)))
            for a, b in zip(s.box, want):
                got = a[int(c.table[r, i])].double().cpu().numpy()
                assert (np.abs(got - b) <= np.abs(b) * (BF16_U + 2.0 ** -23)).all()
    qd = q.double().cpu().numpy()
    wl, wn = op.select(qd, *(b.double().cpu().numpy() for b in s.box), s.c.table, s.ctx, n, 6, s.page, 1, 1,
                       lists.shape[2])
    assert np.array_equal(lists.cpu().numpy(), wl) and np.array_equal(length.cpu().numpy(), wn)
    a = Attend.__new__(Attend)
    a.dims, a.tree, a.n, a.c, a.lists, a.length = (s.R, s.M, s.Hq, s.Dh), False, n, s.c, wl, wn
    a.q, a.scale, a.see = q.cpu(), float(np.float32(s.Dh ** -0.5)), np.zeros((s.R, s.M, s.M), bool)
    live = (np.arange(s.M)[None, :] < n[:, None])
    out, lse = out.clone(), lse.clone()
    out[D(~live, dev)], lse[D(~live, dev)] = 7.0, 7.0
    a.check((out, lse))
    assert sv.spec_get_device_status(s.ws) == 0


def test_captured_steps_replay(sv, dev):
    """Two graphs that share a workspace, with eager steps between the replays."""
    s, t = Step(sv, dev, 42, "bf16"), Step(sv, dev, 43, "e4m3")
    t.ws = s.ws
    graphs, kept = [], []
    side = torch.cuda.Stream()
    for k in (s, t):
        k.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept.append(k.run())
        graphs.append(graph)
    for seed in range(3):
        for k, graph, res in zip((s, t), graphs, kept):
            k.x.copy_(k.inputs(100 + seed))
            graph.replay()
            torch.cuda.synchronize()
            got = [x.clone() for x in res]
            want = k.run()
            live = torch.arange(k.M, device=dev)[None, :] < k.n[:, None]
            torch.cuda.synchronize()
            assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
            for i in (0, 3, 4):
                assert torch.equal(got[i][live], want[i][live])
    assert sv.spec_get_device_status(s.ws) == 0


def test_a_step_on_another_stream(sv, dev):
    s = Step(sv, dev, 44, "bf16")
    s.x.copy_(s.inputs(5))
    want = s.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = s.run(stream=side)
    side.synchronize()
    live = torch.arange(s.M, device=dev)[None, :] < s.n[:, None]
    assert torch.equal(got[1], want[1]) and torch.equal(got[3][live], want[3][live])


def test_a_step_repeated_gives_the_same_bits(sv, dev):
    s = Lists(51, 4, 1, 8, 2, 128, 16, [9000, 4000, 8000, 12000], 64, 1, 1)
    a, b = s.run(sv, dev), s.run(sv, dev)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_empty_calls(sv, dev):
    i32 = dict(dtype=torch.int32, device=dev)
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16, device=dev)
    box = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev)
    none, table = torch.zeros(0, **i32), torch.zeros(0, 4, **i32)
    q = torch.zeros(0, 2, 4, 64, dtype=torch.bfloat16, device=dev)
    sv.spec_page_bounds(k, table, none, none, 5, box, box.clone())
    lists, length = sv.spec_page_select(q, box, box, table, none, none, 2, 16)
    out, _ = sv.spec_page_attention(q, k, k, lists, length, none)
    assert tuple(lists.shape) == (0, 2, 4) and out.numel() == 0
    # a batch without tables: idle slots are no fault, tokens are
    table, n = torch.zeros(2, 0, **i32), torch.tensor([0, 1], **i32)
    q = torch.zeros(2, 2, 4, 64, dtype=torch.bfloat16, device=dev)
    lists, length = sv.spec_page_select(q, box, box, table, torch.zeros(2, **i32), n, 2, 16)
    assert length.tolist() == [0, -1] and (lists == -1).all()
    sv.spec_page_bounds(k, table, torch.zeros(2, **i32), n, 5, box, box.clone())
    assert status(sv) == sv.SPEC_DEV_BAD_REQUEST
