"""Truncated draws and rows against the fp64 oracle."""
import numpy as np
import pytest
import torch

import oracle
from oracle import sample as osm

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    import lossless_verification_sampling_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.spec_get_device_status(m.default_workspace("cuda:0"))     # what other files' faulty calls left
    return m


@pytest.fixture(scope="module")
def dev(sv):
    return torch.device("cuda:0")


def D(x, dev, dtype=None):
    t = torch.from_numpy(np.array(x)).to(dev)
    return t if dtype is None else t.to(dtype)


def status(sv):
    return sv.spec_get_device_status(sv.default_workspace("cuda:0"))


class Rows:
    """Requests' rows x [R, J, V] (values of dtype) and settings."""

    def __init__(self, x, dtype, t=1.0, k=0, p=1.0, mp=0.0, u=0.5, rows=None):
        self.x = torch.as_tensor(x, dtype=torch.float64).to(dtype)
        R, J, _ = self.x.shape

        def per(v, shape, kind):
                return np.array(np.broadcast_to(np.asarray(v, kind), shape))
        self.t, self.p, self.mp = (per(v, (R,), np.float32) for v in (t, p, mp))
        self.k, self.u = per(k, (R,), np.int32), per(u, (R, J), np.float32)
        self.rows = per(J if rows is None else rows, (R,), np.int32)

    def kw(self, dev):
        return dict(temperature=D(self.t, dev), top_k=D(self.k, dev), top_p=D(self.p, dev), min_p=D(self.mp, dev),
                    rows=D(self.rows, dev))

    def place(self, dev, ld=None, shift=0):
        """The rows on the GPU, ld elements apart from element `shift` on, in
        memory that holds NaN elsewhere."""
        R, J, V = self.x.shape
        ld = V if ld is None else ld
        room = torch.full((shift + R * J * ld + 8,), float("nan"), dtype=self.x.dtype, device=dev)
        t = room[shift:shift + R * J * ld].view(R, J, ld)[:, :, :V]
        t.copy_(self.x)
        return t

    def check(self, sv, dev, ld=None, shift=0, in_place=False):
        x = self.place(dev, ld, shift)
        R, J, V = self.x.shape
        out = dict(tokens=torch.full((R, J), 77, dtype=torch.int32, device=dev),
                   logq=torch.full((R, J), 77.0, device=dev),
                   kept=torch.full((R, J), 77, dtype=torch.int32, device=dev))
        sv.spec_sample(x, D(self.u, dev), **self.kw(dev), out=out)
        whole = x if in_place else torch.full((R, J, V), 77.0, dtype=x.dtype, device=dev)
        before = whole.clone()
        kept2 = out["kept"].clone()
        sv.spec_truncate_logits(x, **self.kw(dev), out=whole, out_kept=kept2)
        torch.cuda.synchronize()
        tok, lq, kept, kept2 = (v.cpu().numpy() for v in (out["tokens"], out["logq"], out["kept"], kept2))
        rows, before = whole.double().cpu(), before.double().cpu()
        for r in range(R):
            for j in range(J):
                if j >= self.rows[r]:
                    assert tok[r, j] == 77 and lq[r, j] == 77.0 and kept[r, j] == 77
                    assert torch.equal(rows[r, j], before[r, j])
                    continue
                x = self.x[r, j].double().numpy()
                how = (int(self.k[r]), float(self.p[r]), float(self.mp[r]))
                wt, wl, wn = osm.draw(x, float(self.t[r]), float(self.u[r, j]), *how)
                mask, _ = osm.kept(x, float(self.t[r]), *how)
                assert kept[r, j] == wn == mask.sum() and kept2[r, j] == wn, (r, j, kept[r, j], wn)
                got = rows[r, j].numpy()
                assert np.array_equal(got, np.where(mask, x, -np.inf)), (r, j, np.flatnonzero((got > -np.inf) != mask)[:9])
                assert tok[r, j] == wt, (r, j, tok[r, j], wt)
                # fp64 up to the one rounding to fp32; a weight is off by a unit at most
                assert abs(lq[r, j] - wl) <= abs(wl) * 2.0 ** -24 + 1e-9, (r, j, lq[r, j], wl)
        assert status(sv) == 0


SETTINGS = dict(t=[1.0, 0.7, 1.3, 0.0, 1.0, 0.9, 2.0], k=[0, 50, 7, 3, 0, 1, 300], p=[1.0, 1.0, 0.9, 0.5, 0.95, 1.0, 0.7],
                mp=[0.0, 0.0, 0.0, 0.2, 0.0, 0.3, 0.01])


def uniforms(g, *shape):
    return np.floor(g.random(shape) * 2 ** 24).astype(np.float32) / np.float32(2 ** 24)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1, 2, 7, 63, 512, 1000, 4097, 32003, 151936, 262144])
def test_against_fp64(sv, dev, V, dtype):
    print(f"[sample] V={V} {dtype}", flush=True)
    g = np.random.default_rng(V)
    R, J = 7, 2
    x = g.standard_normal((R, J, V)) * 3
    x[:, :, :: max(1, V // 20)] += 8 * g.random((R, J, len(range(0, V, max(1, V // 20)))))
    Rows(x, dtype, u=uniforms(g, R, J), rows=[2, 2, 1, 2, 0, 2, 2], **SETTINGS).check(sv, dev)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ld, shift", [(1001, 0), (1003, 1), (1024, 3), (1008, 8), (1000, 5)])
def test_rows_apart_and_off_their_alignment(sv, dev, ld, shift, dtype):
    g = np.random.default_rng(ld)
    x = g.standard_normal((7, 3, 1000)) * 4
    s = Rows(x, dtype, u=uniforms(g, 7, 3), **SETTINGS)
    s.check(sv, dev, ld, shift)
    s.check(sv, dev, ld, shift, in_place=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_equal_logits(sv, dev, dtype):
    V = 50001
    g = np.random.default_rng(2)
    x = np.zeros((9, 1, V))
    x[1] = 1.0 * (np.arange(V) % 7 == 3)
    x[2] = np.where(np.arange(V) % 5 == 0, 0.0, -0.0)
    x[3] = -1e30
    x[4] = np.where(np.arange(V) % 1000 == 999, 2.0, -np.inf)
    x[5] = np.where(np.arange(V) == 40000, 2.0, -np.inf)
    x[6] = g.integers(0, 3, V)
    x[7] = g.integers(0, 3, V)
    x[8] = -0.0
    for k, p in ((0, 1.0), (33, 1.0), (30000, 1.0), (0, 0.3), (20000, 0.5), (0, 0.999), (49999, 0.99)):
        Rows(x, dtype, t=0.8, k=k, p=p, u=uniforms(g, 9, 1)).check(sv, dev)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_close_logits(sv, dev, dtype):
    """Neighbouring values, in one part of the first histogram: the cut is
    found by further ones, from a list and from the row."""
    g = np.random.default_rng(3)
    for V in (1500, 9000):
        step = 2.0 ** (-23 if dtype is F32 else -7)
        x = np.stack([1 + step * g.integers(0, 1 << 11, V), 1e-3 * g.random(V), g.permutation(V) * 1e-38,
                      np.where(np.arange(V) < 5, 1.0, 1 + step), 1e-40 * g.standard_normal(V)])[:, None]
        for k, p in ((700, 1.0), (0, 0.4), (1200, 0.77), (3, 1.0), (V - 1, 0.999)):
            Rows(x, dtype, t=40.0, k=k, p=p, u=uniforms(g, 5, 1)).check(sv, dev)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_wide_logits(sv, dev, dtype):
    g = np.random.default_rng(4)
    big = float(torch.finfo(dtype).max)
    V = 3000
    x = np.stack([g.standard_normal(V) * 1e30, g.choice([-big, 0.0, big], V), g.standard_normal(V) * 100,
                  np.where(g.random(V) < 0.5, -np.inf, g.standard_normal(V) * 50),
                  -big + big / 256 * g.integers(0, 3, V), g.standard_normal(V) * 1e-30])[:, None]
    for t in (1.0, 1e-30, 1e30, 0.0, 1e-3):
        for k, p, mp in ((0, 1.0, 0.0), (1700, 0.9, 0.0), (5, 1.0, 1e-40), (0, 1e-40, 0.0), (0, float(1 - 2.0 ** -24), 1.0)):
            Rows(x, dtype, t=t, k=k, p=p, mp=mp, u=uniforms(g, 6, 1)).check(sv, dev)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("off", [300.0, -300.0, 4e4, -4e4, 3e5])
def test_logits_far_from_zero(sv, dev, off, dtype):
    """top_p's estimated tail where x / T is far larger than the differences."""
    g = np.random.default_rng(11)
    V = 20000
    x = g.standard_normal((4, 1, V)) * 2 * max(1.0, abs(off) / 300)
    x[:, :, ::500] += 9 * max(1.0, abs(off) / 300)
    for t, p in ((1.0, 0.9), (0.3, 0.99), (1.0, 0.99), (0.02, 0.7)):
        Rows(x + off, dtype, t=t * max(1.0, abs(off) / 300), p=p, u=uniforms(g, 4, 1)).check(sv, dev)
    if dtype is F32:                                                # steps of 2^-5 at 3e5, x / T past 2^20
        x = g.standard_normal((4, 1, V)) * 2 + off
        for t, p in ((0.2, 0.9), (0.7, 0.95), (0.7, 0.6)):
            Rows(x, dtype, t=t, p=p, u=uniforms(g, 4, 1)).check(sv, dev)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_truncation_into_rows_between(sv, dev, dtype):
    """The output's rows lie between the logits' own."""
    g = np.random.default_rng(12)
    s = Rows(g.standard_normal((7, 2, 1001)) * 4, dtype, **SETTINGS)
    both = torch.full((7, 2, 2100), 5.0, dtype=dtype, device=dev)
    x, out = both[:, :, :1001], both[:, :, 1050:2051]
    x.copy_(s.x)
    want, _ = sv.spec_truncate_logits(x.contiguous(), **s.kw(dev))
    sv.spec_truncate_logits(x, **s.kw(dev), out=out)
    assert torch.equal(out, want) and torch.equal(x.cpu(), s.x)
    assert (both[:, :, 1001:1050] == 5.0).all() and (both[:, :, 2051:] == 5.0).all()
    with pytest.raises(sv.SpecError):
        sv.spec_truncate_logits(x, **s.kw(dev), out=both[:, :, 1000:2001])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V, shift", [(8186, 5), (8192, 0), (8192, 1), (8193, 0), (8240, 3), (16384 + 1100, 0), (24575, 2)])
def test_rows_that_end_inside_a_part(sv, dev, V, shift, dtype):
    """Lengths around a multiple of the 8192 ids that a workgroup reads; the
    likely ids spread, or all at one end of the row, or the rest masked out."""
    print(f"[sample] V={V} {dtype}", flush=True)
    g = np.random.default_rng(V)
    R = 6
    x = g.standard_normal((R, 1, V)) * 2
    ids = [np.arange(0, V, V // 60), np.arange(300), V - 1 - np.arange(300), g.choice(V, 900, False), np.arange(0), [V - 1]]
    for r, at in enumerate(ids):
        x[r, 0, at] += 6 + 3 * g.random(len(at))
    x[3, 0, : V // 2] = -np.inf
    x[4, 0, 7000:] = -np.inf
    x[5, 0, : V - 500] = -np.inf
    for k, p, mp in ((1, 0.5, 0.0), (20, 1.0, 0.0), (140, 0.9, 0.0), (200, 1.0, 1e-4), (256, 0.97, 0.0), (257, 0.97, 0.0),
                     (0, 0.99, 1e-3), (0, 0.6, 0.0), (2000, 1.0, 0.0)):
        Rows(x, dtype, t=1.1, k=k, p=p, mp=mp, u=uniforms(g, R, 1)).check(sv, dev, V + shift, shift)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("u", [0.0, float(1 - 2.0 ** -24), 0.5, 1e-45])
def test_the_ends_of_the_uniforms(sv, dev, u, dtype):
    g = np.random.default_rng(5)
    x = g.standard_normal((7, 1, 5000)) * 2
    Rows(x, dtype, u=u, **SETTINGS).check(sv, dev)
    x[:, :, :4990] = -np.inf
    Rows(x, dtype, u=u, **SETTINGS).check(sv, dev)
    x[:, :, 10:] = -80.0                                            # weights of 0 behind the last drawn id
    x[:, :, 3] = 0.0
    Rows(x, dtype, u=u, t=1.0, k=[0, 5, 100, 0, 0, 0, 0], mp=[0, 0, 0, .5, 0, 0, 0]).check(sv, dev)


def test_min_p_at_its_edge(sv, dev):
    x = np.full((4, 1, 900), -9.0)
    x[:, 0, 5], x[:, 0, 6] = 1.0, 0.0
    x[:, 0, 7] = 1.0
    e = np.float32(np.exp(-1.0))
    mp = [np.nextafter(e, np.float32(0)), np.nextafter(e, np.float32(1)), 1.0, np.float32(1 - 2.0 ** -24)]
    s = Rows(x, F32, mp=mp)
    s.check(sv, dev)
    kept = sv.spec_sample(s.place(dev), D(s.u, dev), **s.kw(dev))["kept"]
    assert kept[:, 0].tolist() == [3, 2, 2, 2]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_many_kinds(sv, dev, dtype):
    """Peaked rows, whose cuts lie among few candidates, and flat ones, whose
    cuts lie deep; several chunks a row, equal logits and masked ids among
    them; settings alone and together."""
    g = np.random.default_rng(6)
    V = 40007
    x = np.empty((8, 1, V))
    x[0] = g.standard_normal(V) * 2
    x[0, 0, g.integers(0, V, 40)] = 12 + 2.5 * g.standard_normal(40)
    x[1] = g.standard_normal(V) * 0.3                               # flat
    x[2] = np.where(g.random(V) < 0.001, 9.0, g.standard_normal(V))  # equal likely ids
    x[3] = np.where(g.random(V) < 0.995, -np.inf, 2 * g.standard_normal(V))
    x[4] = -np.arange(V) / 50.0                                     # all in the first chunk
    x[5] = np.arange(V) / 500.0 - 3                                 # in the last
    x[6] = np.where(np.arange(V) // 8192 == 2, 3.0 * g.standard_normal(V), -np.inf)
    x[7] = np.round(g.standard_normal(V) * 4) / 2
    for k in (0, 1, 2, 40, 256, 257, 5000):
        for p in (1.0, 0.9, 0.9999, 0.05):
            for mp in (0.0, 0.05, 0.9, 1e-6):
                Rows(x, dtype, t=0.9, k=k, p=p, mp=mp, u=uniforms(g, 8, 1)).check(sv, dev)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_data_faults(sv, dev, dtype):
    V = 700
    x = torch.zeros(12, 2, V, dtype=dtype)
    x[0, 1, 699], x[1, 0, 3], x[2, 0] = float("nan"), float("inf"), float("-inf")
    x[10, 1, 5] = float("nan")                                      # a row that is not in use
    t = np.ones(12, np.float32)
    k, p, mp, rows = np.zeros(12, np.int32), np.ones(12, np.float32), np.zeros(12, np.float32), np.full(12, 2, np.int32)
    t[3], p[4], p[5], mp[6], rows[7], rows[8] = np.nan, 0.0, np.nan, 1.5, 3, -1
    rows[10] = 1
    u = np.full((12, 2), 0.3, np.float32)
    u[9, 1], u[11, 0] = 1.0, -0.1
    kw = dict(temperature=D(t, dev), top_k=D(k, dev), top_p=D(p, dev), min_p=D(mp, dev), rows=D(rows, dev))
    bad = np.zeros((12, 2), bool)
    bad[0, 1] = bad[1, 0] = bad[2, 0] = True
    bad[3:9] = True
    badu = bad.copy()
    badu[9, 1] = badu[11, 0] = True
    got = sv.spec_sample(x.to(dev), D(u, dev), **kw)
    assert status(sv) == sv.SPEC_DEV_BAD_REQUEST
    used = np.arange(2)[None, :] < np.where((rows < 0) | (rows > 2), 2, rows)[:, None]
    tok, lq, kept = (got[n].cpu().numpy() for n in ("tokens", "logq", "kept"))
    assert (tok[badu] == -1).all() and np.isnan(lq[badu]).all() and (kept[badu] == -1).all()
    good = used & ~badu
    assert (tok[good] == int(0.3 * V)).all() and (kept[good] == V).all()
    out, kept = sv.spec_truncate_logits(x.to(dev), **kw)
    assert status(sv) == sv.SPEC_DEV_BAD_REQUEST
    assert np.array_equal(torch.isnan(out).all(-1).cpu().numpy()[used], bad[used])
    assert (kept.cpu().numpy()[bad] == -1).all()
    t[:] = 1.0
    t[0], t[1], t[2] = -1.0, 1e-31, 2e30
    t[3] = np.inf
    got = sv.spec_sample(torch.zeros(12, 2, V, dtype=dtype, device=dev), D(np.full((12, 2), 0.3, np.float32), dev),
                         temperature=D(t, dev))
    assert (got["tokens"][:4] == -1).all() and (got["tokens"][4:] == int(0.3 * V)).all()
    assert status(sv) == sv.SPEC_DEV_BAD_REQUEST


def test_greedy_rows_read_no_uniform(sv, dev):
    x = torch.randn(3, 2, 4000, device=dev)
    got = sv.spec_sample(x, torch.full((3, 2), float("nan"), device=dev), temperature=torch.zeros(3, device=dev))
    assert torch.equal(got["tokens"].long(), x.argmax(-1)) and (got["logq"] == 0).all() and (got["kept"] == 1).all()
    assert status(sv) == 0


def test_empty_calls(sv, dev):
    z = torch.zeros(0, device=dev)
    got = sv.spec_sample(torch.zeros(0, 3, 10, device=dev), torch.zeros(0, 3, device=dev), temperature=z)
    assert got["tokens"].shape == (0, 3)
    out, kept = sv.spec_truncate_logits(torch.zeros(2, 0, 10, device=dev), temperature=torch.ones(2, device=dev))
    assert out.shape == (2, 0, 10) and kept.shape == (2, 0)


def test_optional_outputs(sv, dev):
    x, u, t = torch.randn(2, 2, 500, device=dev), torch.rand(2, 2, device=dev), torch.ones(2, device=dev)
    a = sv.spec_sample(x, u, temperature=t)
    b = sv.spec_sample(x, u, temperature=t, want_logq=False, want_kept=False)
    assert torch.equal(a["tokens"], b["tokens"]) and b["logq"] is None and b["kept"] is None
    out, kept = sv.spec_truncate_logits(x, temperature=t, want_kept=False)
    assert torch.equal(out, x) and kept is None


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_verification_of_truncated_rows(sv, dev, dtype):
    """Drafts drawn under truncation, both sides' rows truncated alike: the
    verification agrees with the CPU oracle on the truncated rows, and only
    ids that the target keeps are committed."""
    g = np.random.default_rng(7)
    R, gamma, V = 16, 4, 3001
    target = Rows(g.standard_normal((R, gamma + 1, V)) * 2, dtype, t=0.8, k=40, p=0.95, mp=0.02)
    draft = Rows(target.x[:, :gamma].double().numpy() + 0.5 * g.standard_normal((R, gamma, V)), dtype, t=0.8, k=40, p=0.95,
                 mp=0.02)
    x = draft.place(dev)
    tok = sv.spec_sample(x, D(uniforms(g, R, gamma), dev), **draft.kw(dev))["tokens"]
    p, _ = sv.spec_truncate_logits(x, **draft.kw(dev), out=x)
    q, _ = sv.spec_truncate_logits(target.place(dev), **target.kw(dev))
    ln = g.integers(0, gamma + 1, R).astype(np.int32)
    ua, us = uniforms(g, R, gamma), uniforms(g, R, gamma + 1)
    got = sv.spec_verify_batch(q, p, tok, D(ln, dev), D(target.t, dev), D(ua, dev), D(us, dev))
    torch.cuda.synchronize()

    def host(t):
        return t.float().cpu().numpy() if dtype is F32 else t.cpu().view(torch.int16).numpy().view(np.uint16)
    ref = oracle.verify_batch(host(q), host(p), tok.cpu().numpy(), ln, target.t, ua, us)
    tie = ref["first_tie"] >= 0
    n, out = got["num_accepted"].cpu().numpy(), got["tokens"].cpu().numpy()
    assert tie.sum() <= 1 and (n >= 0).all()
    assert np.array_equal(n[~tie], ref["num_accepted"][~tie]) and np.array_equal(out[~tie], ref["tokens"][~tie])
    for r in range(R):
        for i in range(int(n[r]) + 1):
            assert q[r, i, int(out[r, i])] > -float("inf")


def test_more_rows_than_one_slice(sv, dev):
    """A call takes 16384 chunks at a time."""
    g = np.random.default_rng(10)
    x = D(g.standard_normal((4100, 2, 9000)), dev, BF16)            # two chunks a row
    u, t = D(uniforms(g, 4100, 2), dev), torch.full((4100,), 0.8, device=dev)
    how = dict(temperature=t, top_k=torch.full((4100,), 30, dtype=torch.int32, device=dev))
    got = sv.spec_sample(x, u, **how)
    out, kept = sv.spec_truncate_logits(x, **how)
    assert (kept == 30).all() and torch.equal(got["kept"], kept) and ((out > -float("inf")).sum(-1) == 30).all()
    for r in (0, 4094, 4095, 4096, 4099):
        for j in range(2):
            want = osm.draw(x[r, j].double().cpu().numpy(), float(t[0]), float(u[r, j]), 30)
            assert int(got["tokens"][r, j]) == want[0]
    parts = sv.spec_sample(x[4000:].contiguous(), u[4000:].contiguous(), temperature=t[4000:],
                           top_k=how["top_k"][4000:])
    assert all(torch.equal(parts[n], got[n][4000:]) for n in parts)


def test_captured_calls_replay(sv, dev):
    g = np.random.default_rng(8)
    ws = sv.Workspace(dev, 1 << 20)
    s = Rows(g.standard_normal((7, 2, 20011)) * 3, BF16, **SETTINGS)
    x, u, kw = s.place(dev), D(s.u, dev), s.kw(dev)
    small = Rows(g.standard_normal((3, 1, 900)), F32, k=5)
    y, v, kw2 = small.place(dev), D(small.u, dev), small.kw(dev)

    def both():
        a = sv.spec_sample(x, u, **kw, workspace=ws)
        return [a["tokens"], a["logq"], a["kept"], *sv.spec_truncate_logits(x, **kw, workspace=ws)]

    def other():
        return list(sv.spec_sample(y, v, **kw2, workspace=ws).values())
    graphs, kept = [], []
    side = torch.cuda.Stream()
    for f in (both, other):
        f()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept.append(f())
        graphs.append(graph)
    for seed in range(4):
        x.copy_(D(g.standard_normal((7, 2, 20011)) * 3, dev, BF16))
        y.copy_(D(g.standard_normal((3, 1, 900)), dev, F32))
        u.copy_(D(uniforms(g, 7, 2), dev))
        for f, graph, res in zip((both, other), graphs, kept):
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in res]
            want = f()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert sv.spec_get_device_status(ws) == 0


def test_calls_on_other_streams(sv, dev):
    g = np.random.default_rng(9)
    s = Rows(g.standard_normal((7, 3, 30000)) * 3, F32, u=uniforms(g, 7, 3), **SETTINGS)
    x, u, kw = s.place(dev), D(s.u, dev), s.kw(dev)
    want = sv.spec_sample(x, u, **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [sv.spec_sample(x, u, **kw, stream=st, workspace=sv.Workspace(dev)) for st in streams]
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(o[n], want[n]) for n in want)
