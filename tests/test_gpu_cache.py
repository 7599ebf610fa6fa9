"""The paged cache on the GPU: tree masks, normalised and rotated writes,
reads and path commits against the fp64 oracle."""
import numpy as np
import pytest
import torch

from cache_util import BF16_U, Cache, bf16, random_trees
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


# ---------------------------------------------------------------- tree masks

@pytest.mark.parametrize("R,M,window,chain", [(1, 1, 0, False), (3, 9, 0, False), (2, 32, 2, False),
                                              (2, 33, 0, True), (5, 130, 3, False),
                                              (2, 1024, 0, False), (1, 1024, 40, True)])
def test_tree_mask(sv, dev, R, M, window, chain):
    g = np.random.default_rng([M, window])
    n = np.array([M] + [int(g.integers(0, M + 1)) for _ in range(R - 1)], np.int32)
    ctx = g.integers(0, 5000, R).astype(np.int32)
    parent = random_trees(g, R, M, n, chain)
    pos, mask = sv.spec_tree_mask(D(parent, dev), D(n, dev), D(ctx, dev), window=window)
    rp, rs = oc.tree_mask(parent, n, ctx, window)
    np.testing.assert_array_equal(pos.cpu().numpy(), rp)
    np.testing.assert_array_equal(mask.cpu().numpy(), oc.pack_bits(rs))


@pytest.mark.parametrize("fault", ["parent_self", "parent_negative", "n_high", "n_negative",
                                   "ctx_negative", "ctx_overflow"])
def test_tree_mask_faults(sv, dev, fault):
    g = np.random.default_rng(7)
    n, ctx = np.array([20, 20, 7], np.int32), np.array([5, 6, 7], np.int32)
    parent = random_trees(g, 3, 20, n)
    if fault == "parent_self":
        parent[1, 11] = 11
    elif fault == "parent_negative":
        parent[1, 3] = -1
    elif fault == "n_high":
        n[1] = 21
    elif fault == "n_negative":
        n[1] = -2
    elif fault == "ctx_negative":
        ctx[1] = -1
    else:
        ctx[1] = 2 ** 31 - 10
    ws = sv.Workspace(dev, 256)
    pos, mask = sv.spec_tree_mask(D(parent, dev), D(n, dev), D(ctx, dev), workspace=ws)
    assert sv.spec_get_device_status(ws) == sv.SPEC_DEV_BAD_REQUEST
    assert (pos[1] == -1).all() and not mask[1].any()
    rp, rs = oc.tree_mask(parent, n, ctx)
    np.testing.assert_array_equal(pos.cpu().numpy(), rp)
    np.testing.assert_array_equal(mask.cpu().numpy(), oc.pack_bits(rs))


# -------------------------------------------------------------------- writes

def check_write(c, before, after, r, tok, got_rows, exact, slack):
    """Cache rows of tokens `tok` of request r (values, fp64) against the fp64
    rows `exact` with fp32 slack `slack`."""
    if c.kind == "bf16":
        tol = np.abs(exact) * BF16_U + slack
    else:
        s = np.abs(exact).max(-1, keepdims=True) / 448.0
        tol = np.maximum(np.abs(exact) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 1e-5) + 2 * slack
    assert (np.abs(got_rows - exact) <= tol).all(), float((np.abs(got_rows - exact) / tol).max())


WRITES = [  # R, M, Hq, Hkv, D, page, kind, dtype, norm, rot, interleaved, positions
    (1, 1, 1, 1, 64, 16, "bf16", "bf16", True, 64, False, False),
    (2, 9, 32, 8, 128, 64, "bf16", "bf16", True, 128, False, True),
    (3, 33, 6, 2, 128, 16, "e4m3", "bf16", True, 128, True, True),
    (2, 17, 5, 5, 256, 32, "e4m3", "f32", True, 64, False, False),
    (2, 20, 7, 1, 64, 128, "e4m3", "f32", False, 32, True, True),
    (2, 40, 3, 1, 256, 16, "bf16", "f32", True, 256, False, True),
    (1, 70, 4, 4, 64, 16, "bf16", "bf16", False, 16, False, False),
    (2, 21, 0, 3, 128, 32, "e4m3", "bf16", True, 48, False, True),
    (2, 19, 0, 2, 128, 32, "bf16", "bf16", False, 0, False, False),
]


@pytest.mark.parametrize("case", WRITES)
@pytest.mark.parametrize("fused", [False, True])
def test_qkv_write(sv, dev, case, fused):
    R, M, Hq, Hkv, Dh, page, kind, dt, norm, rot, inter, with_pos = case
    g = np.random.default_rng(M)
    ctx = g.integers(0, 60, R).astype(np.int32)
    n = np.array([M] + [M // 2] * (R - 1), np.int32)
    c = Cache(g, R, int(ctx.max()) + M, Hkv, Dh, page, kind).to(dev)
    H = Hq + 2 * Hkv
    x = bf16(g.standard_normal((R, M, H, Dh)) * 2)
    x = x if dt == "bf16" else x.float() + torch.from_numpy(
        (g.standard_normal((R, M, H, Dh)) * 1e-3).astype(np.float32))
    xd = x.to(dev)
    parts = [xd[:, :, :Hq], xd[:, :, Hq:Hq + Hkv], xd[:, :, Hq + Hkv:]]
    if not fused:
        parts = [p.contiguous() for p in parts]
    q, k, v = parts
    w = [None, None]
    if norm:
        w = [(bf16(1 + 0.3 * g.standard_normal(Dh))).to(x.dtype) for _ in range(2)]
    rope = None
    max_pos = int(ctx.max()) + M
    if rot:
        t = np.arange(max_pos)[:, None] * 100.0 ** -(np.arange(rot // 2) * 2 / rot)[None, :]
        rope = np.stack([np.cos(t), np.sin(t)], -1).astype(np.float32)
    pos = ctx[:, None] + np.arange(M)[None, :]
    if with_pos:
        pos = np.where(np.arange(M)[None, :] < n[:, None], g.integers(0, max_pos, (R, M)), -1)
    before = [t.clone() for t in c.dev] + [None if t is None else t.clone() for t in c.scales]
    out = torch.full((R, M, Hq, Dh), 7.0, dtype=torch.bfloat16, device=dev) if Hq else None
    ws = sv.Workspace(dev, 256)
    got = sv.spec_qkv_write(k, v, *c.args(), D(ctx, dev), D(n, dev), q=q if Hq else None,
                            q_weight=w[0].to(dev) if norm and Hq else None,
                            k_weight=w[1].to(dev) if norm else None, eps=1e-5,
                            rope=None if rope is None else D(rope, dev), interleaved=inter,
                            positions=D(pos.astype(np.int32), dev) if with_pos else None,
                            out_q=out, workspace=ws, **c.kw())
    torch.cuda.synchronize()
    assert sv.spec_get_device_status(ws) == 0
    assert got is out
    xf = x.double().numpy()
    wf = [None if t is None else t.double().numpy() for t in w]
    touched = np.zeros((c.P, page), bool)
    for r in range(R):
        for i in range(M):
            if i >= n[r]:
                assert not Hq or (out[r, i] == 7.0).all()
                continue
            t = int(ctx[r]) + i
            pg, off = c.table[r, t // page], t % page
            touched[pg, off] = True
            rows = xf[r, i]
            for part, lo, hi, wt in (("q", 0, Hq, wf[0]), ("k", Hq, Hq + Hkv, wf[1])):
                if lo == hi:
                    continue
                y = oc.norm_rotate(rows[lo:hi], wt, 1e-5, rope, pos[r, i], inter)
                plain = oc.norm_rotate(rows[lo:hi], wt, 1e-5, None, 0, inter)
                # fp32: D/64 + 10 roundings in the mean (halved by the root),
                # three in the products, three in the rotation, of terms no
                # larger than the row's largest before it (two of them)
                slack = 2.0 ** -19 * np.abs(plain).max(-1, keepdims=True)
                if part == "q":
                    gq = out[r, i].double().cpu().numpy()
                    assert (np.abs(gq - y) <= np.abs(y) * BF16_U + slack).all()
                else:
                    check_write(c, before, None, r, t, c.rows(0, r, t, 1)[0], y, slack)
            val = rows[Hq + Hkv:].astype(np.float32)
            if kind == "bf16":
                want = bf16(val).double().numpy()
            else:
                codes, s = oc.quantise(val)
                want = codes * s.astype(np.float64)[:, None]
            np.testing.assert_array_equal(c.rows(1, r, t, 1)[0], want)
    # nothing else in the pools changed
    keep = torch.from_numpy(~touched).to(dev)
    for now, old in zip(c.dev + c.scales, before):
        if now is None:
            continue
        b = torch.uint8 if now.element_size() == 1 else torch.int16 if now.element_size() == 2 else torch.int32
        a, o = now.view(b).transpose(1, 2)[keep], old.view(b).transpose(1, 2)[keep]
        assert torch.equal(a, o)


def test_write_of_non_finite_and_zero_rows(sv, dev):
    g = np.random.default_rng(5)
    c = Cache(g, 1, 16, 1, 64, 16, "e4m3").to(dev)
    x = torch.zeros(1, 5, 1, 64)
    x[0, 1, 0, 5] = float("nan")
    x[0, 2, 0, 6] = float("-inf")
    x[0, 3, 0, 7] = 3e38
    x[0, 4, 0, 8] = 1e-40
    x = x.to(dev)
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device=dev)  # noqa: E731
    sv.spec_qkv_write(x, x, *c.args(), i32(0), i32(5), **c.kw())
    for which in (0, 1):
        rows = c.rows(which, 0, 0, 5)[:, 0]
        assert not rows[0].any()
        assert np.isnan(rows[1]).all() and np.isnan(rows[2]).all()
        assert abs(rows[3, 7] / 3e38 - 1) < 2.0 ** -22 and not np.delete(rows[3], 7).any()
        assert rows[4, 8] == oc.quantise(x[0, 4].cpu().numpy())[0][0, 8] * 2.0 ** -126


@pytest.mark.parametrize("fault", ["n_high", "ctx_negative", "past_table", "bad_page", "position"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_write_faults(sv, dev, fault, kind):
    g = np.random.default_rng(9)
    R, M, Hq, Hkv, Dh, page = 3, 6, 4, 2, 64, 16
    ctx, n = np.array([3, 14, 20], np.int32), np.array([6, 6, 4], np.int32)
    c = Cache(g, R, 32, Hkv, Dh, page, kind)
    pos = (ctx[:, None] + np.arange(M)[None, :]).astype(np.int32)
    if fault == "n_high":
        n[1] = 7
    elif fault == "ctx_negative":
        ctx[1] = -3
    elif fault == "past_table":
        ctx[1] = 27
    elif fault == "bad_page":
        c.table[1, 1] = c.P                     # tokens 16 .. 19 of the request
    else:
        pos[1, 4] = 40
    c.to(dev)
    before = [t.clone().cpu() for t in c.dev]
    x = bf16(g.standard_normal((R, M, Hq + 2 * Hkv, Dh))).to(dev)
    rope = np.zeros((40, 16, 2), np.float32)
    rope[:, :, 0] = 1.0                         # no turn
    ws = sv.Workspace(dev, 256)
    out = torch.full((R, M, Hq, Dh), 7.0, dtype=torch.bfloat16, device=dev)
    sv.spec_qkv_write(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], *c.args(), D(ctx, dev), D(n, dev),
                      q=x[:, :, :Hq], rope=D(rope, dev), positions=D(pos, dev), out_q=out,
                      workspace=ws, **c.kw())
    torch.cuda.synchronize()
    assert sv.spec_get_device_status(ws) == sv.SPEC_DEV_BAD_REQUEST
    assert torch.equal(out[0], x[0, :, :Hq]) and torch.equal(out[2, :4], x[2, :4, :Hq])
    if fault in ("n_high", "ctx_negative", "past_table"):
        assert torch.isnan(out[1]).all()
        mine = c.table[1]
        for now, old in zip(c.dev, before):
            b = torch.uint8 if kind == "e4m3" else torch.int16
            assert torch.equal(now.cpu().view(b)[mine], old.view(b)[mine])
    elif fault == "bad_page":
        assert torch.equal(out[1], x[1, :, :Hq])
        if kind == "bf16":
            np.testing.assert_array_equal(c.rows(1, 1, 14, 2), x[1, :2, Hq + Hkv:].double().cpu().numpy())
    else:
        bad = torch.isnan(out[1]).all(-1).all(-1).cpu()
        assert bad.tolist() == [False] * 4 + [True, False]
        assert np.isnan(c.rows(0, 1, 18, 1)).all() and not np.isnan(c.rows(1, 1, 14, 6)).any()


# --------------------------------------------------------------------- reads

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,L,Hkv,Dh,page", [(1, 1, 1, 64, 16), (3, 77, 3, 128, 32),
                                             (2, 130, 2, 256, 64), (2, 257, 8, 64, 128)])
def test_kv_read(sv, dev, kind, dt, R, L, Hkv, Dh, page):
    g = np.random.default_rng(L)
    start = g.integers(0, 40, R).astype(np.int32)
    ln = np.array([L] + [int(g.integers(0, L)) for _ in range(R - 1)], np.int32)
    c = Cache(g, R, int((start + ln).max()), Hkv, Dh, page, kind).to(dev)
    ok = torch.full((R, L, Hkv, Dh), 7.0, dtype=dt, device=dev)
    ov = torch.full_like(ok, 7.0)
    sv.spec_kv_read(*c.args(), D(start, dev), D(ln, dev), L, out_k=ok, out_v=ov, **c.kw())
    for which, got in ((0, ok), (1, ov)):
        for r in range(R):
            m = int(ln[r])
            want = torch.from_numpy(c.rows(which, r, int(start[r]), m))
            # an e4m3 code has 4 significant bits and its scale 24: the fp32
            # product rounds once, and bf16 may round it a second time
            x = got[r, :m].double().cpu()
            u = (2.0 ** -24 if kind == "e4m3" else 0.0) + (
                BF16_U if dt == torch.bfloat16 and kind == "e4m3" else 0.0)
            assert ((x - want).abs() <= want.abs() * u).all()
            assert (got[r, m:] == 7.0).all()


@pytest.mark.parametrize("fault", ["start", "len", "past", "page"])
def test_kv_read_faults(sv, dev, fault):
    g = np.random.default_rng(2)
    c = Cache(g, 2, 48, 2, 64, 16, "bf16")
    start, ln, L = np.array([0, 4], np.int32), np.array([30, 30], np.int32), 32
    if fault == "start":
        start[1] = -1
    elif fault == "len":
        ln[1] = 33
    elif fault == "past":
        start[1] = 19
    else:
        c.table[1, 1] = -5
    c.to(dev)
    ws = sv.Workspace(dev, 256)
    k, v = sv.spec_kv_read(*c.args(), D(start, dev), D(ln, dev), L, workspace=ws)
    assert sv.spec_get_device_status(ws) == sv.SPEC_DEV_BAD_REQUEST
    np.testing.assert_array_equal(k[0, :30].double().cpu().numpy(), c.rows(0, 0, 0, 30))
    nan = torch.isnan(v[1]).all(-1).all(-1).cpu().numpy()
    if fault == "page":
        np.testing.assert_array_equal(nan[:30], (np.arange(30) >= 12) & (np.arange(30) < 28))
    else:
        assert nan.all()


# ------------------------------------------------------------------- commits

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("R,M,Hkv,Dh,page", [(4, 9, 2, 64, 16), (6, 48, 8, 128, 32),
                                             (3, 200, 1, 256, 16)])
def test_kv_commit(sv, dev, kind, R, M, Hkv, Dh, page):
    g = np.random.default_rng(M)
    ctx = g.integers(0, 50, R).astype(np.int32)
    A = np.array([M - 1, 0, -1] + [int(g.integers(1, min(M, 40))) for _ in range(R - 3)], np.int32)
    path = np.full((R, M), -1, np.int32)
    for r in range(R):
        if A[r] > 0:
            path[r, :A[r]] = np.sort(g.choice(np.arange(1, M), A[r], replace=False))
    if A[-1] > 1:
        path[-1, :A[-1]] = np.arange(2, A[-1] + 2)       # every row moves by one
    c = Cache(g, R, 50 + M, Hkv, Dh, page, kind).to(dev)
    want = [[c.rows(w, r, 0, 50 + M) for r in range(R)] for w in (0, 1)]
    for w in (0, 1):
        for r in range(R):
            for i in range(max(A[r], 0)):
                want[w][r][ctx[r] + 1 + i] = want[w][r][ctx[r] + path[r, i]]
    ws = sv.Workspace(dev, 256)
    new = sv.spec_kv_commit(*c.args(), D(ctx, dev), D(A, dev), D(path, dev), workspace=ws, **c.kw())
    assert sv.spec_get_device_status(ws) == 0
    np.testing.assert_array_equal(new.cpu().numpy(), np.where(A < 0, ctx, ctx + 1 + A))
    for w in (0, 1):
        for r in range(R):
            np.testing.assert_array_equal(c.rows(w, r, 0, 50 + M), want[w][r])


@pytest.mark.parametrize("fault", ["accepted_high", "accepted_low", "not_rising", "path_high",
                                   "past", "page"])
def test_kv_commit_faults(sv, dev, fault):
    g = np.random.default_rng(3)
    R, M = 2, 12
    c = Cache(g, R, 32, 2, 64, 16, "e4m3")
    ctx, A = np.array([2, 10], np.int32), np.array([2, 3], np.int32)
    path = np.full((R, M), -1, np.int32)
    path[0, :2], path[1, :3] = [3, 7], [2, 5, 9]
    if fault == "accepted_high":
        A[1] = 12
    elif fault == "accepted_low":
        A[1] = -2
    elif fault == "not_rising":
        path[1, 2] = 5
    elif fault == "path_high":
        path[1, 2] = 12
    elif fault == "past":
        ctx[1] = 25
    else:
        c.table[1, 1] = c.P + 3
    c.to(dev)
    before = [t.view(torch.uint8).clone() for t in c.dev]
    keep = c.table[1][:1] if fault == "page" else c.table[1]
    ws = sv.Workspace(dev, 256)
    new = sv.spec_kv_commit(*c.args(), D(ctx, dev), D(A, dev), D(path, dev), workspace=ws, **c.kw())
    assert sv.spec_get_device_status(ws) == sv.SPEC_DEV_BAD_REQUEST
    assert new.tolist() == [5, -1]
    for now, old in zip(c.dev, before):
        assert torch.equal(now.view(torch.uint8)[keep], old[keep])


def test_the_largest_launches(sv, dev):
    """One token of 2^24 - 1 (and the same beyond: refused before the launch)."""
    most = (1 << 24) - 1
    x = torch.empty(1, most + 1, 1, 64, dtype=torch.bfloat16, device=dev)
    x[0, :1] = 2.0
    k, v = (torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    one = torch.ones(1, dtype=torch.int32, device=dev)
    table, zero = torch.zeros(1, 1, dtype=torch.int32, device=dev), torch.zeros_like(one)
    sv.spec_qkv_write(x[:, :most], x[:, :most], k, v, table, zero, one)
    assert (k[0, 0, 0] == 2).all() and (v[0, 0, 0] == 2).all() and not k[0, 0, 1:].any()
    with pytest.raises(sv.SpecError) as e:
        sv.spec_qkv_write(x, x, k, v, table, zero, one)
    assert e.value.status == -5
    del x
    got = [torch.full((1, 4 * most, 1, 64), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    sv.spec_kv_read(k, v, table, zero, one, 4 * most, out_k=got[0], out_v=got[1])
    for x in got:
        assert (x[0, 0] == 2).all() and (x[0, 1:1000] == 7).all() and (x[0, -1000:] == 7).all()


PROMPTS = [  # R, M, Hq, Hkv, D, page, norm, rot, interleaved
    (7, 73, 5, 1, 64, 16, True, 64, False),        # 511 tokens: a head row a thread
    (4, 128, 5, 1, 64, 16, True, 64, False),       # 512: a workgroup a token
    (3, 171, 32, 8, 128, 64, True, 128, False),
    (4, 131, 7, 7, 128, 32, True, 48, True),
    (5, 110, 60, 4, 128, 16, True, 64, False),     # more rows than one pass holds
    (4, 129, 128, 8, 64, 32, False, 16, False),
    (3, 200, 2, 1, 256, 16, True, 256, True),
    (4, 140, 16, 8, 256, 128, True, 64, False),
    (4, 128, 33, 3, 256, 16, True, 0, False),
    (2, 300, 0, 5, 128, 64, True, 128, False),     # no queries
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", PROMPTS)
def test_qkv_write_prompts(sv, dev, case, dt, kind):
    R, M, Hq, Hkv, Dh, page, norm, rot, inter = case
    print(f"[write] {case} {dt} {kind}", flush=True)
    g = np.random.default_rng([R, M])
    ctx = g.integers(0, 60, R).astype(np.int32)
    n = np.array([M, 0] + [int(x) for x in g.integers(1, M + 1, R - 2)], np.int32)
    c = Cache(g, R, int(ctx.max()) + M, Hkv, Dh, page, kind).to(dev)
    H = Hq + 2 * Hkv
    x = bf16(g.standard_normal((R, M, H, Dh), np.float32) * 2)
    if dt == "f32":
        x = x.float() + torch.from_numpy(g.standard_normal((R, M, H, Dh), np.float32) * 1e-3)
    w = [None, None]
    if norm:
        w = [bf16(1 + 0.3 * g.standard_normal(Dh)).to(x.dtype) for _ in range(2)]
    rope, max_pos = None, int(ctx.max()) + M
    if rot:
        a = np.arange(max_pos)[:, None] * 100.0 ** -(np.arange(rot // 2) * 2 / rot)[None, :]
        rope = np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)
    before = [t.clone() for t in c.dev] + [None if t is None else t.clone() for t in c.scales]
    out = torch.full((R, M, Hq, Dh), 7.0, dtype=torch.bfloat16, device=dev) if Hq else None
    ws = sv.Workspace(dev, 256)
    xd = x.to(dev)
    sv.spec_qkv_write(xd[:, :, Hq:Hq + Hkv], xd[:, :, Hq + Hkv:], *c.args(), D(ctx, dev), D(n, dev),
                      q=xd[:, :, :Hq] if Hq else None, q_weight=w[0].to(dev) if norm and Hq else None,
                      k_weight=w[1].to(dev) if norm else None, eps=1e-5,
                      rope=None if rope is None else D(rope, dev), interleaved=inter, out_q=out,
                      workspace=ws, **c.kw())
    torch.cuda.synchronize()
    assert sv.spec_get_device_status(ws) == 0
    live = np.arange(M)[None, :] < n[:, None]
    r, i = np.nonzero(live)
    t = ctx[r] + i
    pg, off = c.table[r, t // page], t % page
    rows = x.double().numpy()[live]                # [tokens, H, Dh]

    def rotated(part, wt):
        """(rows, those before the rotation), fp64"""
        p = part
        if wt is not None:
            p = p / np.sqrt((p * p).mean(-1, keepdims=True) + 1e-5) * wt.double().numpy()
        if not rot:
            return p, p
        z, y = rope[t].astype(np.float64)[:, None], p.copy()
        h = rot // 2
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, h), slice(h, rot))
        y[..., a] = p[..., a] * z[..., 0] - p[..., b] * z[..., 1]
        y[..., b] = p[..., b] * z[..., 0] + p[..., a] * z[..., 1]
        return y, p

    def held(which):
        """values of the cache rows that were written, fp64 [tokens, Hkv, Dh]"""
        v = c.dev[which][torch.from_numpy(pg).long().to(dev), :, torch.from_numpy(off).long().to(dev)]
        v = v.float().cpu().numpy().astype(np.float64)
        if c.scales[which] is not None:
            v = v * c.scales[which].cpu().numpy().astype(np.float64)[pg, :, off][..., None]
        return v
    # fp32: 13 roundings in the mean's sum (halved by the root), three to the
    # factor, two products, three in the rotation of two terms: below 32 half
    # steps of the row's largest value before it
    if Hq:
        y, p = rotated(rows[:, :Hq], w[0])
        slack = 2.0 ** -19 * np.abs(p).max(-1, keepdims=True)
        got = out.double().cpu().numpy()
        assert (got[~live] == 7.0).all()
        assert (np.abs(got[live] - y) <= np.abs(y) * BF16_U + slack).all()
    y, p = rotated(rows[:, Hq:Hq + Hkv], w[1])
    check_write(c, None, None, None, None, held(0), y, 2.0 ** -19 * np.abs(p).max(-1, keepdims=True))
    val = rows[:, Hq + Hkv:].astype(np.float32)
    if kind == "bf16":
        want = bf16(val).double().numpy()
    else:
        codes, s = oc.quantise(val)
        want = codes * s.astype(np.float64)[..., None]
    np.testing.assert_array_equal(held(1), want)
    touched = np.zeros((c.P, page), bool)
    touched[pg, off] = True
    keep = torch.from_numpy(~touched).to(dev)
    for now, old in zip(c.dev + c.scales, before):
        if now is None:
            continue
        b = torch.uint8 if now.element_size() == 1 else torch.int16 if now.element_size() == 2 else torch.int32
        assert torch.equal(now.view(b).transpose(1, 2)[keep], old.view(b).transpose(1, 2)[keep])
