"""A model that drafts for itself over a budget of its cache's pages, the
operators together as a server runs them: per drafted token the cache write,
the page's bounds, the page lists, attention over them and a truncated draw;
then one pass over the whole context, both sides' rows truncated, verified,
and the path committed.  Two rounds, eager and as one captured graph."""
import numpy as np
import pytest
import torch

import oracle
from cache_util import BF16_U, Cache, bf16
from oracle import pages as op
from oracle import sample as osm
from test_gpu_sample import uniforms

pytestmark = pytest.mark.gpu
GAMMA, V, FIRST, LAST, BUDGET = 3, 517, 1, 1, 4


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


class Model:
    """One attention layer between an embedding and a head, R requests."""

    def __init__(self, sv, dev, seed, kind):
        g = np.random.default_rng(seed)
        self.sv, self.dev, self.g = sv, dev, g
        self.R, self.Hq, self.Hkv, self.Dh, self.page = 4, 4, 2, 64, 16
        self.c = Cache(g, self.R, 330, self.Hkv, self.Dh, self.page, kind).to(dev)
        width = self.Hq + 2 * self.Hkv
        self.embed = bf16(g.standard_normal((V, width, self.Dh))).to(dev)
        self.head = D((0.4 * g.standard_normal((self.Hq * self.Dh, V))).astype(np.float32), dev)
        self.box = [torch.zeros(self.c.P, self.Hkv, self.Dh, dtype=torch.bfloat16, device=dev) for _ in range(2)]
        t = np.arange(400)[:, None] * 50.0 ** -(np.arange(self.Dh // 2) * 2 / self.Dh)[None, :]
        self.rope = D(np.stack([np.cos(t), np.sin(t)], -1).astype(np.float32), dev)
        self.ctx = D(np.array([300, 129, 15, 0], np.int32), dev)
        self.anchor = D(g.integers(0, V, self.R).astype(np.int32), dev)
        self.t = np.array([0.7, 1.0, 0.0, 1.2], np.float32)
        self.k, self.p = np.array([40, 0, 0, 200], np.int32), np.array([0.95, 0.8, 1.0, 1.0], np.float32)
        self.mp = np.array([0.0, 0.05, 0.0, 0.0], np.float32)
        self.how = dict(temperature=D(self.t, dev), top_k=D(self.k, dev), top_p=D(self.p, dev), min_p=D(self.mp, dev))
        self.ws = sv.Workspace(dev, 1 << 22)
        sv.spec_page_bounds(self.c.dev[0], self.c.t, torch.zeros_like(self.ctx), self.ctx, 300, *self.box,
                            k_scale=self.c.scales[0], workspace=self.ws)
        self.one = torch.ones(self.R, dtype=torch.int32, device=dev)
        self.all = torch.full((self.R,), GAMMA + 1, dtype=torch.int32, device=dev)
        # the drafts are a chain of nodes behind the anchor
        self.path = (torch.arange(GAMMA + 1, dtype=torch.int32, device=dev) + 1).expand(self.R, -1).contiguous()
        # a round's uniforms, which a captured round reads anew
        self.ud, self.ua = torch.zeros(self.R, GAMMA, device=dev), torch.zeros(self.R, GAMMA, device=dev)
        self.us = torch.zeros(self.R, GAMMA + 1, device=dev)

    def uniforms(self, seed):
        g = np.random.default_rng(seed)
        for t in (self.ud, self.ua, self.us):
            t.copy_(D(uniforms(g, *t.shape), self.dev))

    def write(self, tokens, at, n):
        x, h, k = self.embed[tokens.long()], self.Hq, self.Hkv
        return self.sv.spec_qkv_write(x[:, :, h:h + k], x[:, :, h + k:], *self.c.args(), at, n, q=x[:, :, :h],
                                      rope=self.rope, workspace=self.ws, **self.c.kw())

    def logits(self, o):
        return (o.float().flatten(2) @ self.head).to(torch.bfloat16)

    def round(self):
        """Every tensor of a round that a check wants to see."""
        sv, ws, c = self.sv, self.ws, self.c
        tok, seen, drafted, rows = self.anchor[:, None], [], [], []
        for j in range(GAMMA):
            at = self.ctx + j
            q = self.write(tok, at, self.one)
            sv.spec_page_bounds(c.dev[0], c.t, at, self.one, 1, *self.box, k_scale=c.scales[0], workspace=ws)
            lists, length = sv.spec_page_select(q, *self.box, c.t, at, self.one, BUDGET, self.page, first=FIRST,
                                                last=LAST, workspace=ws)
            o, _ = sv.spec_page_attention(q, *c.dev, lists, length, self.one, workspace=ws, **c.kw())
            z = self.logits(o)
            d = sv.spec_sample(z, self.ud[:, j:j + 1].contiguous(), **self.how, workspace=ws)
            tok = d["tokens"]
            seen += [q, lists, length, z, tok, d["kept"], *(b.clone() for b in self.box)]
            drafted.append(tok)
            rows.append(z)
        drafted = torch.cat(drafted, 1)
        q = self.write(torch.cat([self.anchor[:, None], drafted], 1), self.ctx, self.all)
        o, _ = sv.spec_tree_attention(q, *c.args(), self.ctx, self.all, workspace=ws, **c.kw())
        target = self.logits(o)
        tt, _ = sv.spec_truncate_logits(target, **self.how, workspace=ws)
        draft = torch.cat(rows, 1)
        td, _ = sv.spec_truncate_logits(draft, **self.how, out=draft, workspace=ws)
        got = sv.spec_verify_batch(tt, td, drafted, self.all - 1, self.how["temperature"], self.ua, self.us, workspace=ws)
        n = got["num_accepted"]
        ctx = sv.spec_kv_commit(*c.args(), self.ctx, n, self.path, workspace=ws, **c.kw())
        # rejected tokens leave the bounds of the pages they were in
        sv.spec_page_bounds(c.dev[0], c.t, self.ctx, n + 1, GAMMA + 1, *self.box, k_scale=c.scales[0], workspace=ws)
        return seen, target, tt, td, drafted, got["tokens"], n, ctx

    def go_on(self, tokens, n, ctx):
        self.anchor.copy_(tokens.gather(1, n.long()[:, None])[:, 0])
        self.ctx.copy_(ctx)


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_rounds(sv, dev, kind):
    m = Model(sv, dev, 61, kind)
    R, moved = m.R, 0
    for turn in range(2):
        print(f"[drafting] {kind} round {turn}", flush=True)
        m.uniforms(70 + turn)
        c0 = m.ctx.cpu().numpy()
        seen, target, tt, td, drafted, tokens, n, ctx = m.round()
        torch.cuda.synchronize()
        # ---- drafts: lists by the bounds as they were, tokens by the rows
        for j in range(GAMMA):
            q, lists, length, z, tok, kept, lo, hi = seen[8 * j:8 * j + 8]
            wl, wn = op.select(q.double().cpu().numpy(), lo.double().cpu().numpy(), hi.double().cpu().numpy(), m.c.table,
                               c0 + j, np.ones(R, int), BUDGET, m.page, FIRST, LAST, lists.shape[2])
            assert np.array_equal(lists.cpu().numpy(), wl) and np.array_equal(length.cpu().numpy(), wn)
            for r in range(R):
                want = osm.draw(z[r, 0].double().cpu().numpy(), float(m.t[r]), float(m.ud[r, j]), int(m.k[r]),
                                float(m.p[r]), float(m.mp[r]))
                assert (int(tok[r, 0]), int(kept[r, 0])) == (want[0], want[2])
        # ---- truncated rows and their verification
        for full, cut in ((target, tt), (torch.cat([seen[8 * j + 3] for j in range(GAMMA)], 1), td)):
            for r in range(R):
                for j in range(full.shape[1]):
                    x = full[r, j].double().cpu().numpy()
                    keep, _ = osm.kept(x, float(m.t[r]), int(m.k[r]), float(m.p[r]), float(m.mp[r]))
                    assert np.array_equal(cut[r, j].double().cpu().numpy(), np.where(keep, x, -np.inf))
        ref = oracle.verify_batch(bits(tt), bits(td), drafted.cpu().numpy(), np.full(R, GAMMA, np.int32), m.t,
                                  m.ua.cpu().numpy(), m.us.cpu().numpy())
        na, out = n.cpu().numpy(), tokens.cpu().numpy()
        sure = ref["first_tie"] < 0
        assert np.array_equal(na[sure], ref["num_accepted"][sure]) and np.array_equal(out[sure], ref["tokens"][sure])
        for r in range(R):
            for i in range(int(na[r]) + 1):
                assert tt[r, i, int(out[r, i])] > -float("inf")
        # ---- what is committed, and its bounds
        assert np.array_equal(ctx.cpu().numpy(), c0 + 1 + na)
        moved += int(na.sum())
        for r in range(R):
            last = int(c0[r] + na[r])
            for i in range(last // m.page + 1):
                want = op.bounds(m.c.rows(0, r, i * m.page, min(m.page, last + 1 - i * m.page)))
                for a, b in zip(m.box, want):
                    got = a[int(m.c.table[r, i])].double().cpu().numpy()
                    assert (np.abs(got - b) <= np.abs(b) * (BF16_U + 2.0 ** -23)).all()
        m.go_on(tokens, n, ctx)
    assert moved > 0
    assert sv.spec_get_device_status(m.ws) == 0


def test_captured_rounds_replay(sv, dev):
    """A round in one graph: replays, with an eager round of another model on
    the same workspace between them, give what eager rounds give."""
    eager, other = Model(sv, dev, 62, "bf16"), Model(sv, dev, 63, "e4m3")
    held = Model(sv, dev, 62, "bf16")
    other.ws = held.ws
    state = [x.clone() for x in (*held.c.dev, *held.box)]
    held.round()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        kept = held.round()
    for a, b in zip((*held.c.dev, *held.box), state):   # as before the first round
        a.copy_(b)
    for turn in range(3):
        for m in (eager, held, other):
            m.uniforms(80 + turn)
        want = eager.round()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*want[0], *want[1:]), (*kept[0], *kept[1:])):
            assert torch.equal(a, b)
        eager.go_on(*want[5:])
        held.go_on(*kept[5:])
        x = other.round()
        other.go_on(*x[5:])
        torch.cuda.synchronize()
    assert sv.spec_get_device_status(held.ws) == 0
