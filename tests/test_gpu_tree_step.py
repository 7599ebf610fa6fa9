"""The cache operators as a decoding step uses them: tree mask, cache write,
attention, verification of the tree's logits and the path's commit, two steps
in a row, against the same step in fp64; and the same calls on other streams,
captured into graphs and with shared workspaces."""
import numpy as np
import pytest
import torch

from cache_util import BF16_U, Cache, bf16, random_trees
from oracle import cache as oc
from oracle import tree as otree
from test_gpu_graph import capture, replay_and_compare

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


class Step:
    """One layer and an output projection over small trees."""

    def __init__(self, seed, kind, dev, R=3, M=12, Hq=4, Hkv=2, Dh=64, page=16, V=300):
        g = np.random.default_rng(seed)
        self.dims = R, M, Hq, Hkv, Dh, V
        self.ctx = g.integers(5, 40, R).astype(np.int32)
        self.c = Cache(g, R, 40 + 4 * M, Hkv, Dh, page, kind).to(dev)
        self.w = bf16(1 + 0.2 * g.standard_normal((2, Dh)))
        t = np.arange(200)[:, None] * 50.0 ** -(np.arange(Dh // 2) * 2 / Dh)[None, :]
        self.rope = np.stack([np.cos(t), np.sin(t)], -1).astype(np.float32)
        self.head = g.standard_normal((Hq * Dh, V)).astype(np.float32)
        self.g, self.dev = g, dev

    def draft(self):
        R, M, Hq, Hkv, Dh, V = self.dims
        n = np.array([M, M - 3, 1], np.int32)
        return n, random_trees(self.g, R, M, n), bf16(self.g.standard_normal((R, M, Hq + 2 * Hkv, Dh)))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_two_steps(sv, dev, kind):
    s = Step(31, kind, dev)
    R, M, Hq, Hkv, Dh, V = s.dims
    ctx = D(s.ctx, dev)
    for step in range(2):
        n, parent, qkv = s.draft()
        x = qkv.to(dev)
        nd, pd = D(n, dev), D(parent, dev)
        pos, mask = sv.spec_tree_mask(pd, nd, ctx)
        q = sv.spec_qkv_write(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], *s.c.args(), ctx, nd,
                              q=x[:, :, :Hq], q_weight=s.w[0].to(dev), k_weight=s.w[1].to(dev),
                              rope=D(s.rope, dev), positions=pos, **s.c.kw())
        o, _ = sv.spec_tree_attention(q, *s.c.args(), ctx, nd, mask=mask, positions=pos, **s.c.kw())
        logits = (o.float().reshape(R, M, -1) @ D(s.head, dev)).contiguous()
        # drafted tokens: half of the nodes get what their parent's row prefers
        best = logits.argmax(-1).cpu().numpy()
        tok = s.g.integers(0, V, (R, M)).astype(np.int32)
        for r in range(R):
            for v in range(1, n[r]):
                if s.g.random() < 0.5:
                    tok[r, v] = best[r, parent[r, v]]
        acc, path, _ = sv.spec_tree_verify(logits, pd, D(tok, dev), nd, M - 1)
        # ---- the same in fp64, on the cache as it now stands
        c0 = ctx.cpu().numpy()
        rp, see = oc.tree_mask(parent, n, c0)
        np.testing.assert_array_equal(pos.cpu().numpy(), rp)
        xf = qkv.double().numpy()
        for r in range(R):
            m, c = int(n[r]), int(c0[r])
            k, v = s.c.rows(0, r, 0, c + m), s.c.rows(1, r, 0, c + m)
            for i in range(m):
                y = oc.norm_rotate(xf[r, i, :Hq], s.w[0].double().numpy(), 1e-6, s.rope, rp[r, i], False)
                gq = q[r, i].double().cpu().numpy()
                assert (np.abs(gq - y) <= np.abs(y) * BF16_U + 2.0 ** -16).all()
                for h in range(Hq):
                    ok = np.concatenate([np.ones(c, bool), see[r, i, :m]])[None]
                    a, _, w, ds = oc.attention(gq[h:h + 1], k[:, h // 2], v[:, h // 2], ok, Dh ** -0.5)
                    tol = np.abs(a) * BF16_U + w * (BF16_U + 4 * (Dh + 4) * 2.0 ** -24 * ds[:, None]
                                                    + 2.0 ** -16) + 1e-30
                    assert (np.abs(o[r, i, h].double().cpu().numpy() - a[0]) <= tol[0]).all()
        ref = otree.tree_verify(logits.cpu().numpy(), parent, tok, n)
        np.testing.assert_array_equal(acc.cpu().numpy(), ref["accepted"])
        A, pth = ref["accepted"], ref["path"]
        want = [[s.c.rows(w, r, 0, int(c0[r]) + M) for r in range(R)] for w in (0, 1)]
        new = sv.spec_kv_commit(*s.c.args(), ctx, acc, path, **s.c.kw())
        np.testing.assert_array_equal(new.cpu().numpy(), c0 + 1 + A)
        assert step or A.max() > 0
        for w in (0, 1):
            for r in range(R):
                keep = [want[w][r][:c0[r] + 1]] + [want[w][r][c0[r] + u][None] for u in pth[r, :A[r]]]
                np.testing.assert_array_equal(s.c.rows(w, r, 0, int(c0[r]) + 1 + A[r]), np.concatenate(keep))
        ctx = new


def calls(sv, s, dev, seed, ws):
    """Inputs of one step and a function that runs it into fixed outputs."""
    R, M, Hq, Hkv, Dh, V = s.dims
    n, parent, qkv = s.draft()
    x, nd, pd, ctx = qkv.to(dev), D(n, dev), D(parent, dev), D(s.ctx, dev)
    rope, w = D(s.rope, dev), s.w.to(dev)
    acc = torch.tensor([1, 0, 0], dtype=torch.int32, device=dev)
    path = torch.full((R, M), -1, dtype=torch.int32, device=dev)
    path[0, 0] = 5

    def run():
        pos, mask = sv.spec_tree_mask(pd, nd, ctx, workspace=ws)
        q = sv.spec_qkv_write(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], *s.c.args(), ctx, nd,
                              q=x[:, :, :Hq], q_weight=w[0], k_weight=w[1], rope=rope, positions=pos,
                              workspace=ws, **s.c.kw())
        o = torch.zeros_like(q)
        l = torch.zeros(q.shape[:3], device=dev)
        sv.spec_tree_attention(q, *s.c.args(), ctx, nd, mask=mask, positions=pos, out=o, out_lse=l,
                               workspace=ws, **s.c.kw())
        new = sv.spec_kv_commit(*s.c.args(), ctx, acc, path, workspace=ws, **s.c.kw())
        live = torch.arange(M, device=dev)[None] < nd[:, None]
        k, v = sv.spec_kv_read(*s.c.args(), torch.zeros_like(ctx), new, 60, workspace=ws,
                               out_k=torch.zeros(R, 60, Hkv, Dh, device=dev),
                               out_v=torch.zeros(R, 60, Hkv, Dh, device=dev), **s.c.kw())
        return pos, mask, torch.where(live[..., None, None], q.float(), 0.0), o.float(), l, new, k, v

    def fill(_):
        nn, pp, xx = s.draft()
        x.copy_(xx.to(dev))
        pd.copy_(D(pp, dev))
    return run, fill


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_step_graph(sv, dev, kind):
    """A captured step, replayed with new inputs and eager calls (of this step
    and of another operator, on the same workspace) between the replays."""
    s = Step(32, kind, dev)
    need = max(sv.spec_tree_attention_workspace_bytes(3, 12, 4, 2, 64), sv.spec_tv_workspace_bytes(4, 5000))
    ws = sv.Workspace(dev, need)
    run, fill = calls(sv, s, dev, 1, ws)
    g, out = capture(run)
    t = torch.randn(4, 5000, device=dev)

    def eager():
        sv.spec_tv_accept_rate(t, t + 1, torch.ones(4, device=dev), workspace=ws)
        return run()
    replay_and_compare(g, out, fill, eager, rounds=4)
    assert sv.spec_get_device_status(ws) == 0


def test_two_graphs_share_a_workspace(sv, dev):
    a, b = Step(33, "bf16", dev), Step(34, "e4m3", dev, M=40, Hq=8, Hkv=1, Dh=128)
    ws = sv.Workspace(dev, max(sv.spec_tree_attention_workspace_bytes(3, 12, 4, 2, 64),
                               sv.spec_tree_attention_workspace_bytes(3, 40, 8, 1, 128)))
    (ra, fa), (rb, fb) = calls(sv, a, dev, 1, ws), calls(sv, b, dev, 2, ws)
    (ga, oa), (gb, ob) = capture(ra), capture(rb)
    for k in range(3):
        fa(k)
        fb(k)
        wa, wb = [x.clone() for x in ra()], [x.clone() for x in rb()]
        for t in oa + ob:
            t.zero_()
        ga.replay()
        gb.replay()
        torch.cuda.synchronize()
        for x, y in zip(oa + ob, wa + wb):
            assert torch.equal(x, y)


def test_a_graph_keeps_a_workspace_that_was_outgrown(sv, dev):
    """A larger call after the capture takes a new buffer; the replay still
    writes to the old one, which nobody else may have got meanwhile."""
    s = Step(39, "bf16", dev)
    need = sv.spec_tree_attention_workspace_bytes(3, 12, 4, 2, 64)
    ws = sv.Workspace(dev, need)
    run, fill = calls(sv, s, dev, 1, ws)
    g, out = capture(run)
    size = ws.nbytes
    ws.ensure(2 * size)
    others = [torch.full((size,), 77, dtype=torch.uint8, device=dev) for _ in range(3)]
    fill(1)
    want = [x.clone() for x in run()]
    for t in out:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip(out, want):
        assert torch.equal(x, y)
    assert all((o == 77).all() for o in others)


def test_two_streams_with_workspaces_of_their_own(sv, dev):
    steps = [Step(35 + i, "e4m3", dev, M=20) for i in range(2)]
    spaces = [sv.Workspace(dev, sv.spec_tree_attention_workspace_bytes(3, 20, 4, 2, 64)) for _ in steps]
    runs = [calls(sv, s, dev, 1, w)[0] for s, w in zip(steps, spaces)]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = runs[i]()
    torch.cuda.synchronize()
    for x, y in zip(sum(map(list, got), []), sum(want, [])):
        assert torch.equal(x, y)


def test_given_stream(sv, dev):
    s = Step(41, "bf16", dev)
    R, M, Hq, Hkv, Dh, V = s.dims
    q = torch.randn(R, M, Hq, Dh, device=dev).to(torch.bfloat16)
    n, ctx = torch.full((R,), M, dtype=torch.int32, device=dev), D(s.ctx, dev)
    want, _ = sv.spec_tree_attention(q, *s.c.args(), ctx, n)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got, _ = sv.spec_tree_attention(q, *s.c.args(), ctx, n, stream=st,
                                    workspace=sv.Workspace(dev, sv.spec_tree_attention_workspace_bytes(
                                        R, M, Hq, Hkv, Dh)))
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_empty_calls(sv, dev):
    e = lambda *s, t=torch.int32: torch.empty(s, dtype=t, device=dev)  # noqa: E731
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device=dev)
    pos, mask = sv.spec_tree_mask(e(0, 5), e(0), e(0))
    assert pos.shape == (0, 5) and mask.shape == (0, 5, 1)
    o, l = sv.spec_tree_attention(e(0, 5, 2, 64, t=torch.bfloat16), k, k, e(0, 3), e(0), e(0), want_lse=True)
    assert o.shape == (0, 5, 2, 64) and l.shape == (0, 5, 2)
    assert sv.spec_kv_commit(k, k, e(0, 3), e(0), e(0), e(0, 5)).shape == (0,)
    x = e(2, 0, 1, 64, t=torch.bfloat16)
    sv.spec_qkv_write(x, x, k, k, e(2, 3), e(2), e(2))
    z = torch.zeros(2, dtype=torch.int32, device=dev)
    a, b = sv.spec_kv_read(k, k, torch.zeros(2, 1, dtype=torch.int32, device=dev), z, z, 0)
    assert a.shape == b.shape == (2, 0, 1, 64)
    # idle slots only
    q = torch.ones(2, 3, 2, 64, dtype=torch.bfloat16, device=dev)
    out = torch.full_like(q, 7.0)
    sv.spec_tree_attention(q, k, k, torch.zeros(2, 1, dtype=torch.int32, device=dev), z, z, out=out)
    assert (out == 7.0).all()


def test_refusals(sv, dev):
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device=dev)
    z = torch.zeros(2, dtype=torch.int32, device=dev)
    tb = torch.zeros(2, 1, dtype=torch.int32, device=dev)
    q = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16, device=dev)
    with pytest.raises(TypeError):
        sv.spec_tree_attention(q.float(), k, k, tb, z, z)
    with pytest.raises(TypeError):
        sv.spec_tree_attention(q, k.float(), k, tb, z, z)
    with pytest.raises(ValueError):
        sv.spec_tree_attention(q, k, k, tb, z[:1], z)
    with pytest.raises(ValueError):
        sv.spec_tree_attention(q, k, k.cpu(), tb, z, z)
    with pytest.raises(ValueError):
        sv.spec_tree_attention(q.transpose(1, 2), k, k, tb, z, z)
    with pytest.raises(ValueError):                     # e4m3 without scales
        k8 = k.to(torch.float8_e4m3fn)
        sv.spec_tree_attention(q, k8, k8, tb, z, z)
    with pytest.raises(sv.SpecError):                   # 3 query heads over 2
        sv.spec_tree_attention(q[:, :, :1].expand(2, 3, 3, 64).contiguous(), torch.cat([k, k], 1),
                               torch.cat([k, k], 1), tb, z, z)
    x = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError):                     # tokens not evenly spaced
        sv.spec_qkv_write(x[:, :, :1].transpose(0, 1), x[:, :, :1].transpose(0, 1), k, k,
                          torch.zeros(3, 1, dtype=torch.int32, device=dev), z, z)
    with pytest.raises(ValueError):                     # a head apart
        sv.spec_qkv_write(x[:, :, ::2][:, :, :1], x[..., ::2][:, :, :1], k, k, tb, z, z)
    with pytest.raises(ValueError):
        sv.spec_qkv_write(x[:, :, :1], x[:, :, :1], k, k, tb, z, z, q_weight=torch.ones(64, device=dev))
    with pytest.raises(ValueError):
        sv.spec_kv_read(k, k, tb, z, z, -1)
    with pytest.raises(sv.SpecError):
        sv.spec_kv_commit(k, k, tb, z, z, torch.zeros(2, 3, dtype=torch.int32, device=dev), out_ctx_len=z)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("M", [3, 24])
def test_pages_past_32_bits(sv, dev, kind, M):
    """The same step over pages whose byte offsets pass 2^32: the same bits."""
    s = Step(40, kind, dev, M=M + 3, Dh=128, page=64)
    near, far = s.c, Step(40, kind, dev, M=M + 3, Dh=128, page=64).c
    shape = near.dev[0].shape
    gap = (1 << 32) // (shape[1] * shape[2] * shape[3] * near.dev[0].element_size())
    for w in (0, 1):
        big = torch.empty((gap + shape[0],) + shape[1:], dtype=near.dev[w].dtype, device=dev)
        big[gap:].copy_(near.dev[w])
        far.dev[w] = big
        if kind == "e4m3":
            sc = torch.empty((gap + shape[0],) + shape[1:3], device=dev)
            sc[gap:].copy_(near.scales[w])
            far.scales[w] = sc
    far.P, far.t = gap + shape[0], near.t + gap
    outs = []
    n, parent, qkv = s.draft()
    for c in (near, far):
        s.c = c
        R, M1, Hq, Hkv, Dh, V = s.dims
        x, nd, ctx = qkv.to(dev), D(n, dev), D(s.ctx, dev)
        pos, mask = sv.spec_tree_mask(D(parent, dev), nd, ctx)
        q = sv.spec_qkv_write(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], *c.args(), ctx, nd,
                              q=x[:, :, :Hq], rope=D(s.rope, dev), positions=pos, **c.kw())
        o = torch.zeros_like(q)
        _, lse = sv.spec_tree_attention(q, *c.args(), ctx, nd, mask=mask, positions=pos, out=o,
                                        out_lse=torch.zeros(R, M1, Hq, device=dev), **c.kw())
        path = torch.full((R, M1), -1, dtype=torch.int32, device=dev)
        path[0, :2] = torch.tensor([2, M1 - 1])
        acc = torch.tensor([2, 0, 0], dtype=torch.int32, device=dev)
        new = sv.spec_kv_commit(*c.args(), ctx, acc, path, **c.kw())
        kv = sv.spec_kv_read(*c.args(), torch.zeros_like(ctx), ctx + nd, 60 + M1,
                             out_k=torch.zeros(R, 60 + M1, Hkv, Dh, device=dev),
                             out_v=torch.zeros(R, 60 + M1, Hkv, Dh, device=dev), **c.kw())
        outs.append((o, lse, new, *kv))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert outs[0][0].abs().sum() > 0 and outs[0][3].abs().sum() > 0


def test_a_workspace_elsewhere_is_refused(sv, dev):
    ws = sv.Workspace(dev, 256)
    ws.buf = torch.zeros(1 << 26, dtype=torch.uint8)
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device=dev)
    z = torch.zeros(2, dtype=torch.int32, device=dev)
    tb = torch.zeros(2, 1, dtype=torch.int32, device=dev)
    q = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16, device=dev)
    for call in (lambda: sv.spec_tree_mask(tb, z, z, workspace=ws),
                 lambda: sv.spec_tree_attention(q, k, k, tb, z, z, workspace=ws),
                 lambda: sv.spec_qkv_write(q[:, :, :1], q[:, :, 1:], k, k, tb, z, z, workspace=ws),
                 lambda: sv.spec_kv_read(k, k, tb, z, z, 3, workspace=ws),
                 lambda: sv.spec_kv_commit(k, k, tb, z, z, tb, workspace=ws)):
        with pytest.raises(ValueError):
            call()


def test_token_numbers_past_31_bits_are_faults(sv, dev):
    """A table wide enough for more than 2^31 tokens (its pages repeat)."""
    k = torch.zeros(1, 1, 1024, 64, dtype=torch.bfloat16, device=dev)
    tb = torch.zeros(1, (1 << 21) + 8, dtype=torch.int32, device=dev)
    ctx = torch.tensor([2 ** 31 - 1000], dtype=torch.int32, device=dev)
    n = torch.tensor([1010], dtype=torch.int32, device=dev)
    few = torch.tensor([3], dtype=torch.int32, device=dev)
    q = torch.ones(1, 1024, 1, 64, dtype=torch.bfloat16, device=dev)
    ws = sv.Workspace(dev, sv.spec_tree_attention_workspace_bytes(1, 1024, 1, 1, 64))

    def bad():
        return sv.spec_get_device_status(ws) == sv.SPEC_DEV_BAD_REQUEST
    for m in (n, few):
        x = q[:, :int(m)].contiguous()
        out, _ = sv.spec_tree_attention(x, k, k, tb, ctx, m, workspace=ws)
        assert bad() and torch.isnan(out).all()
        out = sv.spec_qkv_write(x, x, k, k, tb, ctx, m, q=x, workspace=ws)
        assert bad() and torch.isnan(out).all() and not k.any()
        out, _ = sv.spec_kv_read(k, k, tb, ctx, m, int(m), workspace=ws)
        assert bad() and torch.isnan(out).all()
    path = torch.tensor([[2, 3, -1, -1]], dtype=torch.int32, device=dev)
    new = sv.spec_kv_commit(k, k, tb, ctx, few - 1, path, workspace=ws)
    assert bad() and int(new) == -1


@pytest.mark.parametrize("R,M", [(0, 3), (2, 0), (0, 0)])
def test_empty_writes_with_queries(sv, dev, R, M):
    e = lambda *s, t=torch.int32: torch.empty(s, dtype=t, device=dev)  # noqa: E731
    c = torch.ones(2, 1, 16, 64, dtype=torch.bfloat16, device=dev)
    x = e(R, M, 4, 64, t=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16, device=dev)
    out = e(R, M, 2, 64, t=torch.bfloat16)
    for given in (None, out):
        got = sv.spec_qkv_write(x[:, :, 2:3], x[:, :, 3:], c, c.clone(), e(R, 3), e(R), e(R), q=x[:, :, :2],
                                q_weight=w, k_weight=w, out_q=given)
        assert got.shape == (R, M, 2, 64) and (given is None or got is given)
    assert (c == 1).all()


def test_a_given_stream_takes_no_memory_of_the_current_one(sv, dev):
    """Blocks that the current stream has just freed, each of an output's size,
    may still be in use there."""
    s = Step(42, "bf16", dev)
    R, M, Hq, Hkv, Dh, V = s.dims
    n, parent, qkv = s.draft()
    x, nd, pd, ctx = qkv.to(dev), D(n, dev), D(parent, dev), D(s.ctx, dev)
    q = x[:, :, :Hq].contiguous()
    st = torch.cuda.Stream()
    ws = sv.Workspace(dev, sv.spec_tree_attention_workspace_bytes(R, M, Hq, Hkv, Dh))
    acc, path = torch.zeros_like(ctx), torch.full((R, M), -1, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()

    def run(**kw):
        pos, mask = sv.spec_tree_mask(pd, nd, ctx, workspace=ws, **kw)
        qo = sv.spec_qkv_write(x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], *s.c.args(), ctx, nd, q=q,
                               workspace=ws, **kw)
        o, l = sv.spec_tree_attention(q, *s.c.args(), ctx, nd, mask=mask, positions=pos, want_lse=True,
                                      workspace=ws, **kw)
        k, v = sv.spec_kv_read(*s.c.args(), torch.zeros_like(ctx), ctx, 40, workspace=ws, **kw)
        return pos, mask, qo, o, l, k, v, sv.spec_kv_commit(*s.c.args(), ctx, acc, path, workspace=ws, **kw)
    want = run()
    free = [torch.empty_like(t) for t in want for _ in range(2)]
    taken = {t.data_ptr() for t in free}
    torch.cuda.synchronize()
    del free
    got = run(stream=st)
    st.synchronize()
    assert not taken & {t.data_ptr() for t in got}
    for r in range(R):
        m = int(n[r])
        for a, b in zip(got[:5], want[:5]):
            assert torch.equal(a[r, :m], b[r, :m])


def test_faults_in_an_outgrown_buffer_are_seen(sv, dev):
    """A fault raised before the workspace grew, and one by a replay after it."""
    s = Step(43, "bf16", dev)
    R, M, Hq, Hkv, Dh, V = s.dims
    n, parent, qkv = s.draft()
    q, ctx = qkv.to(dev)[:, :, :Hq].contiguous(), D(s.ctx, dev)
    good, bad = D(n, dev), D(np.array([M + 1, M, M], np.int32), dev)
    nd = good.clone()
    ws = sv.Workspace(dev, sv.spec_tree_attention_workspace_bytes(R, M, Hq, Hkv, Dh))
    g, out = capture(lambda: sv.spec_tree_attention(q, *s.c.args(), ctx, nd, workspace=ws)[:1])
    assert sv.spec_get_device_status(ws) == 0
    nd.copy_(bad)
    sv.spec_tree_attention(q, *s.c.args(), ctx, nd, workspace=ws)
    nd.copy_(good)
    ws.ensure(ws.nbytes + 1)
    assert sv.spec_get_device_status(ws) == sv.SPEC_DEV_BAD_REQUEST
    for k in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert sv.spec_get_device_status(ws) == 0
        nd.copy_(bad)
        g.replay()
        torch.cuda.synchronize()
        assert torch.isnan(out[0][0]).all()
        assert sv.spec_get_device_status(ws) == sv.SPEC_DEV_BAD_REQUEST
        nd.copy_(good)


def test_a_workspace_taken_inside_a_capture(sv, dev):
    """Its clearing is recorded, not done."""
    s = Step(44, "bf16", dev)
    calls(sv, s, dev, 1, sv.Workspace(dev))[0]()    # all code is loaded
    ws = sv.Workspace(dev)
    run, fill = calls(sv, s, dev, 1, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    ws.buf.fill_(255)                           # what the memory may have held
    assert sv.spec_get_device_status(ws) == 0
    ws.buf.fill_(255)
    run()
    assert sv.spec_get_device_status(ws) == 0
    replay_and_compare(g, out, fill, run)
    assert sv.spec_get_device_status(ws) == 0
