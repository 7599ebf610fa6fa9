"""Timed cases of drafting with the target's own cache and of truncated draws.

A drafting step that attends to a budget of pages instead of the whole context
keeps, for every page and key head, the least and the largest value of each key
dimension; scores the full pages of the context against the step's queries;
lists the best ones; and attends over the lists.  The logits' rows are drawn
from under temperature, top-k, top-p and min-p with given uniforms, and
lossless verification gets the target's and the draft's rows with the ids that
these leave out at -inf.

`own` False: plain torch; `own` True: the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
UNIT = 2.0 ** 44  # weights of ids are whole numbers, UNIT for the row's largest


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one user's next draft token: latency only
        dict(name="sample_user", op="sample", R=1, J=1, V=151936, dtype="bf16", mix="kp"),
        # the draft head's fp32 rows of 64 users, every request its own settings
        dict(name="sample_draft", op="sample", R=64, J=1, V=129280, dtype="f32", mix="mixed"),
        # a server's step without drafts, nucleus sampling
        dict(name="sample_server", op="sample", R=256, J=1, V=151936, dtype="bf16", mix="p"),
        # one user's draft of eight tokens and the bonus row, before verification
        dict(name="truncate_user", op="truncate", R=1, J=9, V=151936, dtype="f32", mix="kp"),
        # the target rows of a batched verification, ragged verify lengths
        dict(name="truncate_verify", op="truncate", R=64, J=8, V=151936, dtype="bf16", mix="mixed"),
        # after a step of up to eight new tokens: latency
        dict(name="bounds_step", op="bounds", R=16, L=8, hkv=8, d=128, page=16, cache="bf16", ctx=4000),
        # after ragged prompts into an e4m3 cache
        dict(name="bounds_prompt", op="bounds", R=8, L=12001, hkv=8, d=128, page=32, cache="e4m3", ctx=77),
        # one user's long context in small pages
        dict(name="select_user", op="select", R=1, M=1, hq=32, hkv=8, d=128, page=16, ctx=30011,
             budget=128),
        # 64 users' ragged contexts
        dict(name="select_batch", op="select", R=64, M=1, hq=32, hkv=8, d=128, page=16, ctx=16000,
             budget=128),
        # one user, one token over 2 k chosen tokens of each key head
        dict(name="sparse_user", op="sparse", R=1, M=1, hq=32, hkv=8, d=128, page=16, budget=128,
             ctx=30011, cache="bf16", tree=False),
        # 64 users, one token, a quantised cache
        dict(name="sparse_batch", op="sparse", R=64, M=1, hq=32, hkv=8, d=128, page=16, budget=128,
             ctx=8000, cache="e4m3", tree=False),
        # a level of drafted trees over wider pages
        dict(name="sparse_tree", op="sparse", R=64, M=20, hq=40, hkv=8, d=128, page=32, budget=64,
             ctx=8000, cache="bf16", tree=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["sample", "sample", "truncate", "bounds", "select", "sparse", "sparse"])
    if op in ("sample", "truncate"):
        c = dict(op=op, R=log(1, 256), J=log(1, 9), V=log(1000, 151936),
                 dtype=rng.choice(["bf16", "f32"]), mix=rng.choice(["k", "p", "m", "kp", "none", "mixed"]))
        most = 256 * 151936 if op == "sample" else 64 * 8 * 151936
        while c["R"] * c["J"] * c["V"] * (2 if c["dtype"] == "f32" else 1) > most:
            c["R"] = max(1, c["R"] * 2 // 3)
            c["V"] = c["V"] if c["R"] > 1 else c["V"] * 2 // 3
        return c
    hkv = rng.choice([1, 2, 4, 5, 8])
    c = dict(op=op, R=log(1, 64), hkv=hkv, d=rng.choice([64, 128, 128, 256]), page=rng.choice([16, 32, 64]),
             ctx=log(100, 30000))
    if op == "bounds":
        c.update(L=log(1, 12000), cache=rng.choice(["bf16", "e4m3"]), ctx=log(1, 4000))
        while c["R"] * (c["L"] + c["ctx"]) * hkv * c["d"] > 8 * 12000 * 8 * 128:
            c["L"], c["ctx"] = max(1, c["L"] * 2 // 3), max(1, c["ctx"] * 2 // 3)
        return c
    c.update(hq=hkv * rng.choice([1, 3, 4, 5, 8]), budget=max(4, log(64, 4096) // c["page"]))
    if op == "select":
        c.update(M=rng.choice([1, 1, 1, log(2, 32)]))
    else:
        c.update(M=rng.choice([1, 1, log(2, 40)]), cache=rng.choice(["bf16", "e4m3"]), tree=rng.random() < 0.5)
    most = 64 * 8000 * 8 * 128
    while c["R"] * c["ctx"] * hkv * c["d"] > most or \
            (op == "sparse" and c["R"] * c["M"] * c["hq"] * c["d"] * c["budget"] * c["page"]
             > 64 * 20 * 40 * 128 * 2048):
        k = "R" if c["R"] > 1 and rng.random() < 0.6 else "ctx" if c["ctx"] > 200 else "M"
        c[k] = max(1, c[k] * 2 // 3)
    return c


def lengths(case):
    """Context lengths per request, spread over the range, and node counts."""
    R, M = case["R"], case.get("M", 1)
    i = np.arange(R)
    frac = (i * 0.6180339887498949) % 1.0
    ctx = np.maximum(1, np.round(case["ctx"] * (1.0 - 0.7 * frac))).astype(np.int32)
    n = np.maximum(1, M - (i * 7) % (M // 4 + 1)).astype(np.int32)
    return ctx, n


def spans(case):
    """First new token and number of new tokens per request."""
    ctx = lengths(case)[0]
    i = np.arange(case["R"])
    return ctx, np.maximum(1, case["L"] - (i * 131) % (case["L"] // 2 + 1)).astype(np.int32)


def live_rows(case):
    """Rows of every request that are in use (a verify length and the bonus row)."""
    J = case["J"]
    return np.maximum(1, J - (np.arange(case["R"]) * 5) % (J // 2 + 1)).astype(np.int32)


def listed_tokens(case):
    """Per request: full context pages listed, tokens listed, node counts."""
    ctx, n = lengths(case)
    full = np.minimum(ctx // case["page"], case["budget"])
    return full, full * case["page"] + ctx % case["page"], n


def work(case):
    op, R = case["op"], case["R"]
    if op in ("sample", "truncate"):
        rows = int(live_rows(case).sum())
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * (case["V"] * e * (1 if op == "sample" else 2) + 16) + 16 * R,
                "flops": rows * case["V"] * 4}
    if op == "bounds":
        start, n = spans(case)
        page, hkv, d = case["page"], case["hkv"], case["d"]
        first, last = start // page, (start + n - 1) // page
        tokens = int((start + n - first * page).sum())
        row = hkv * (d * 2 if case["cache"] == "bf16" else d + 4)
        return {"bytes": tokens * row + int((last - first + 1).sum()) * (4 * hkv * d + 4),
                "flops": 2 * tokens * hkv * d}
    if op == "select":
        ctx, n = lengths(case)
        full = int((ctx // case["page"]).sum())
        return {"bytes": full * case["hkv"] * case["d"] * 4 + full * 4 + 2 * int(n.sum()) * case["hq"] * case["d"]
                + 4 * R * case["hkv"] * case["budget"], "flops": 4 * full * case["hkv"] * case["d"]}
    full, tok, n = (x.astype(np.int64) for x in listed_tokens(case))
    row = case["hkv"] * (case["d"] * 2 if case["cache"] == "bf16" else case["d"] + 4)
    pairs = int((n * tok + (n if case["tree"] else n * (n + 1) // 2)).sum())
    return {"bytes": 2 * int((tok + n).sum()) * row + 4 * int(n.sum()) * case["hq"] * case["d"],
            "flops": 4 * case["d"] * case["hq"] * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def host(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def settings(case, seed):
    """Temperature, top-k, top-p and min-p of every request."""
    R, mix = case["R"], case["mix"]
    g = np.random.default_rng([seed, 3])
    kind = (np.array(["k", "p", "m", "kp", "zero", "none"])[(np.arange(R) + seed) % 6] if mix == "mixed"
            else np.array([mix] * R))
    has = {c: np.array([c in k and k not in ("none", "zero") for k in kind]) for c in "kpm"}
    t = np.where(kind == "zero", 0.0, g.uniform(0.6, 1.2, R))
    return dict(temperature=host(t.astype(np.float32)),
                top_k=host(np.where(has["k"], g.integers(20, 200, R), 0).astype(np.int32)),
                top_p=host(np.where(has["p"], g.uniform(0.8, 0.98, R), 1.0).astype(np.float32)),
                min_p=host(np.where(has["m"], g.uniform(0.02, 0.1, R), 0.0).astype(np.float32)))


def trees(case, seed, n):
    """Ancestor-or-self matrices [R, M, M] of random trees in topological order."""
    R, M = case["R"], case["M"]
    g = np.random.default_rng([seed, 1])
    see = np.zeros((R, M, M), bool)
    rows = np.arange(R)
    for v in range(M):
        if v:
            lo = max(0, v // 3 - 2)
            parent = np.minimum(lo + (g.random(R) * 4).astype(np.int64), v - 1)
            see[:, v] = see[rows, parent]
        see[:, v, v] = True
    return see & (np.arange(M)[None, :] < n[:, None])[:, :, None]


def pack(see):
    """Bits of the last axis as int32 words."""
    R, M, N = see.shape
    W = (N + 31) // 32
    out = np.zeros((R, M, W * 32), bool)
    out[:, :, :N] = see
    return np.packbits(out.reshape(R, M, W, 32), axis=-1, bitorder="little").view(np.int32).reshape(R, M, W)


def table_of(case, seed, tokens):
    """Shuffled page tables for `tokens` tokens a request, and the pool's pages."""
    wide = -(-int(tokens) // case["page"])
    P = case["R"] * wide + 3
    g = torch.Generator(device=DEV).manual_seed(seed)
    table = torch.randperm(P, generator=g, device=DEV)[:case["R"] * wide].reshape(case["R"], wide)
    return table.to(torch.int32).contiguous(), P, g


def pages(case, P, g, names):
    s = {}
    for k in names:
        x = torch.randn(P, case["hkv"], case["page"], case["d"], generator=g, device=DEV)
        s[k + "_scale"] = None
        if case["cache"] == "e4m3":
            s[k + "_scale"] = sc = (x.abs().amax(-1) / E4M3_MAX).clamp_min(2.0 ** -126)
            s[k + "_cache"] = (x / sc[..., None]).to(torch.float8_e4m3fn)
        else:
            s[k + "_cache"] = x.to(torch.bfloat16)
    return s


def prepare(case, seed):
    op, R = case["op"], case["R"]
    if op in ("sample", "truncate"):
        J, V = case["J"], case["V"]
        g = torch.Generator(device=DEV).manual_seed(seed)
        # a broad floor of logits and a few dozen likely ids a row
        x = 2.0 * torch.randn(R, J, V, generator=g, device=DEV)
        at = torch.randint(V, (R, J, 40), generator=g, device=DEV)
        x.scatter_(2, at, 12.0 + 2.5 * torch.randn(R, J, 40, generator=g, device=DEV))
        x = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        u = torch.floor(torch.rand(R, J, generator=g, device=DEV, dtype=torch.float64) * 2 ** 24) / 2 ** 24
        s = dict(op=op, logits=x, u=u.float(), rows=host(live_rows(case)), **settings(case, seed))
        if op == "truncate":
            s["out"] = torch.zeros_like(x)
        else:
            s["tokens"] = torch.full((R, J), -1, device=DEV, dtype=torch.int32)
            s["logq"] = torch.zeros(R, J, device=DEV)
        s["kept"] = torch.full((R, J), -1, device=DEV, dtype=torch.int32)
        return s
    if op == "bounds":
        start, n = spans(case)
        table, P, g = table_of(case, seed, (start + n).max())
        s = dict(op=op, page_table=table, start=host(start), length=host(n), L=case["L"],
                 **pages(case, P, g, ["k"]))
        for k in ("k_min", "k_max"):
            s[k] = torch.zeros(P, case["hkv"], case["d"], device=DEV, dtype=torch.bfloat16)
        return s
    ctx, n = lengths(case)
    M, hq, hkv, d, page = (case[k] for k in ("M", "hq", "hkv", "d", "page"))
    table, P, g = table_of(case, seed, ctx.max() + M)
    s = dict(op=op, n_nodes=host(n), budget=case["budget"],
             q=(2.0 * torch.randn(R, M, hq, d, generator=g, device=DEV)).to(torch.bfloat16))
    if op == "select":
        a = torch.randn(P, hkv, d, generator=g, device=DEV)
        s.update(page_table=table, ctx_len=host(ctx), page=page,
                 k_min=(a - 1.5 - torch.rand(P, hkv, d, generator=g, device=DEV)).to(torch.bfloat16),
                 k_max=(a + 1.5 + torch.rand(P, hkv, d, generator=g, device=DEV)).to(torch.bfloat16),
                 first=min(1, case["budget"]), last=min(2, case["budget"] - 1),
                 lists=torch.zeros(R, hkv, case["budget"] + (M + page - 2) // page + 1, device=DEV,
                                   dtype=torch.int32),
                 listed=torch.zeros(R, device=DEV, dtype=torch.int32))
        return s
    # page lists as a selection leaves them: `budget` full pages of the
    # context in their order, and the pages of its end and of the nodes
    full, tok, _ = listed_tokens(case)
    wide = case["budget"] + (M + page - 2) // page + 1
    r = np.random.default_rng([seed, 2])
    lists = np.full((R, hkv, wide), -1, np.int32)
    own_table = table.cpu().numpy()
    for i in range(R):
        F, f = int(ctx[i]) // page, int(full[i])
        tail = own_table[i, F:(int(ctx[i]) + int(n[i]) - 1) // page + 1]
        order = np.sort(np.argsort(r.random((hkv, F)), 1)[:, :f], 1)
        lists[i, :, :f] = own_table[i][order]
        lists[i, :, f:f + len(tail)] = tail
    s.update(lists=host(lists), listed=host(tok.astype(np.int32)), mask=None, scale=d ** -0.5, page=page,
             out=torch.zeros(R, M, hq, d, device=DEV, dtype=torch.bfloat16),
             lse=torch.zeros(R, M, hq, device=DEV), **pages(case, P, g, ["k", "v"]))
    if case["tree"]:
        s["mask"] = host(pack(trees(case, seed, n)))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return run_own(s)
    return {"sample": plain_sample, "truncate": plain_truncate, "bounds": plain_bounds,
            "select": plain_select, "sparse": plain_sparse}[s["op"]](s)


def run_own(s):
    import lossless_verification_sampling_amd as sv
    op = s["op"]
    if op in ("sample", "truncate"):
        how = dict(temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                   rows=s["rows"])
        if op == "sample":
            return sv.spec_sample(s["logits"], s["u"], **how,
                                  out={k: s[k] for k in ("tokens", "logq", "kept")})
        out, kept = sv.spec_truncate_logits(s["logits"], **how, out=s["out"], out_kept=s["kept"])
        return {"out": out, "kept": kept}
    if op == "bounds":
        sv.spec_page_bounds(s["k_cache"], s["page_table"], s["start"], s["length"], s["L"], s["k_min"],
                            s["k_max"], k_scale=s["k_scale"])
        return {"k_min": s["k_min"], "k_max": s["k_max"]}
    if op == "select":
        lists, listed_len = sv.spec_page_select(s["q"], s["k_min"], s["k_max"], s["page_table"], s["ctx_len"],
                                                s["n_nodes"], s["budget"], s["page"], first=s["first"],
                                                last=s["last"], out_lists=s["lists"], out_len=s["listed"])
        return {"lists": lists, "listed": listed_len}
    out, lse = sv.spec_page_attention(s["q"], s["k_cache"], s["v_cache"], s["lists"], s["listed"],
                                      s["n_nodes"], mask=s["mask"], scale=s["scale"], k_scale=s["k_scale"],
                                      v_scale=s["v_scale"], out=s["out"], out_lse=s["lse"])
    return {"out": out, "lse": lse}


def plain_kept(s):
    """Live rows [N, V] with their weights and which ids are kept.  (64 bits:
    a cumulative sum next to a border decides on a whole token.)"""
    R, J, V = s["logits"].shape
    live = torch.arange(J, device=DEV)[None, :] < s["rows"][:, None]
    x = s["logits"][live].double()

    def per_row(t):
        return t[:, None].expand(R, J)[live][:, None]

    t, k, p, mp = (per_row(s[n]).double() for n in ("temperature", "top_k", "top_p", "min_p"))
    top = x.amax(1, keepdim=True)
    part = torch.exp((x - top) / torch.where(t == 0, 1.0, t))
    w = torch.round(part * UNIT).long()
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    rank = torch.arange(V, device=DEV)[None, :]
    left = torch.gather(x, 1, order) > float("-inf")
    left &= (k <= 0) | (rank < k)
    left &= (t > 0) | (rank < 1)
    ws = torch.gather(w, 1, order) * left
    total = ws.sum(1, keepdim=True)
    before = torch.cumsum(ws, 1) - ws
    left &= (p >= 1) | (before < torch.ceil(p * total.double()).long())
    left &= torch.gather(part, 1, order) >= mp
    keep = torch.zeros_like(left).scatter_(1, order, left)
    return live, x, top, t, w * keep, keep


def plain_sample(s):
    live, x, top, t, w, keep = plain_kept(s)
    u = s["u"][live][:, None].double()
    sums = torch.cumsum(w, 1)
    total = sums[:, -1:]
    # (a greedy row keeps one id)
    token = (sums > torch.floor(u * total.double()).long()).int().argmax(1, keepdim=True)
    logq = (torch.gather(x, 1, token) - top) / torch.where(t == 0, 1.0, t) - torch.log(total.double() / UNIT)
    got = {"tokens": s["tokens"].clone(), "logq": s["logq"].clone(), "kept": s["kept"].clone()}
    got["tokens"][live] = token[:, 0].int()
    got["logq"][live] = logq[:, 0].float()
    got["kept"][live] = keep.sum(1).int()
    return got


def plain_truncate(s):
    live, _, _, _, _, keep = plain_kept(s)
    got = {"out": s["out"].clone(), "kept": s["kept"].clone()}
    got["out"][live] = torch.where(keep, s["logits"][live], float("-inf"))
    got["kept"][live] = keep.sum(1).int()
    return got


def values(s, name, index):
    """fp32 values of the pages that `index` names."""
    x = s[name + "_cache"][index].float()
    return x if s[name + "_scale"] is None else x * s[name + "_scale"][index][..., None]


def plain_bounds(s):
    page = s["k_cache"].shape[2]
    end = s["start"] + s["length"]
    index = torch.arange(s["page_table"].shape[1], device=DEV)[None, :]
    due = (index >= s["start"][:, None] // page) & (index * page < end[:, None])
    where = s["page_table"][due].long()
    filled = (end[:, None] - index * page)[due]
    x = values(s, "k", where)
    there = (torch.arange(page, device=DEV)[None, :] < filled[:, None])[:, None, :, None]
    s["k_min"][where] = torch.where(there, x, float("inf")).amin(2).to(torch.bfloat16)
    s["k_max"][where] = torch.where(there, x, float("-inf")).amax(2).to(torch.bfloat16)
    return {"k_min": s["k_min"], "k_max": s["k_max"]}


def plain_select(s):
    R, M, hq, d = s["q"].shape
    page, hkv, budget = s["page"], s["k_min"].shape[1], s["budget"]
    n, ctx, table = s["n_nodes"][:, None], s["ctx_len"][:, None], s["page_table"].long()
    live = (torch.arange(M, device=DEV)[None, :] < n)[:, :, None, None]
    q = torch.where(live, s["q"], 0).double().reshape(R, M, hkv, hq // hkv, d)
    up, down = q.clamp_min(0).sum((1, 3)), q.clamp_max(0).sum((1, 3))              # [R, hkv, d]
    lo, hi = (s[k][table].double().permute(0, 2, 1, 3) for k in ("k_min", "k_max"))  # [R, hkv, wide, d]
    score = (hi * up[:, :, None]).sum(-1) + (lo * down[:, :, None]).sum(-1)
    full = ctx // page
    index = torch.arange(table.shape[1], device=DEV)[None, :]
    always = (index < s["first"]) | ((index >= full - s["last"]) & (index < full))
    score = torch.where(always[:, None], float("inf"), score)
    score = torch.where((index < full)[:, None], score, float("-inf"))
    order = torch.sort(score, dim=2, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, index[None].expand_as(order).contiguous())
    take = full.clamp_max(budget)
    chosen = (rank < take[:, None]) | ((index >= full) & (index * page < ctx + n))[:, None]
    place = torch.cumsum(chosen.long(), 2) - 1
    lists = torch.full((R, hkv, s["lists"].shape[2] + 1), -1, device=DEV, dtype=torch.int32)
    place = torch.where(chosen, place, s["lists"].shape[2])
    lists.scatter_(2, place, s["page_table"][:, None].expand(R, hkv, -1).contiguous())
    return {"lists": lists[:, :, :-1].contiguous(), "listed": (take * page + ctx % page)[:, 0].int()}


def plain_sparse(s):
    R, M, hq, d = s["q"].shape
    hkv, page = s["lists"].shape[1], s["page"]
    G, L = hq // hkv, s["lists"].shape[2] * page
    where = s["lists"].clamp_min(0).long()
    head = torch.arange(hkv, device=DEV)[None, :, None]
    k, v = (values(s, name, (where, head)).reshape(R, hkv, L, d) for name in ("k", "v"))
    at, node = torch.arange(L, device=DEV)[None, None, :], torch.arange(M, device=DEV)
    u = at - s["listed"][:, None, None]
    if s["mask"] is None:
        tree = u <= node[None, :, None]
    else:
        slot = u.clamp(0, M - 1).expand(R, M, L)
        tree = (u < 0) | ((s["mask"].gather(2, (slot >> 5).long()) >> (slot & 31)) & 1 == 1)
    see = tree & (u < s["n_nodes"][:, None, None])
    q = s["q"].float().reshape(R, M, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(R, hkv, M * G, d)
    x = torch.matmul(q.contiguous(), k.transpose(2, 3).contiguous()) * s["scale"]
    x = torch.where(see[:, None, :, None], x.reshape(R, hkv, M, G, L), float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(R, M, hq)
    o = torch.matmul((x / total.clamp_min(1e-38)).reshape(R, hkv, M * G, L), v)
    o = o.reshape(R, hkv, M, G, d).permute(0, 2, 1, 3, 4).reshape(R, M, hq, d).to(torch.bfloat16)
    live = (node[None, :] < s["n_nodes"][:, None])[:, :, None]
    return {"out": torch.where(live[..., None], o, s["out"]), "lse": torch.where(live, lse, s["lse"])}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact_row(x, t, k, p, mp):
    """(which ids are kept, their whole-number weights, the largest logit) of
    one row: from the row's distinct values and how often each occurs."""
    x = x.double()
    val, inverse, count = torch.unique(x, return_inverse=True, return_counts=True)
    val, count = val.flip(0), count.flip(0)
    count = torch.where(val > float("-inf"), count, 0)
    place = len(val) - 1 - inverse
    if t == 0:
        k, p, mp, t = 1, 1.0, 0.0, 1.0
    part = torch.exp((val - val[0]) / t)
    unit = torch.round(part * UNIT).long()
    behind = torch.cumsum(count, 0)
    if k > 0:
        count = torch.clamp(torch.clamp(k - (behind - count), min=0), max=count)
    if p < 1:
        mass = count * unit
        need = math.ceil(p * float(mass.sum()))
        missing = torch.clamp(need - (torch.cumsum(mass, 0) - mass), min=0)
        taken = (missing + unit - 1) // unit.clamp_min(1)
        count = torch.minimum(count, torch.where(unit > 0, taken, 0))
    count = torch.where(part >= mp, count, 0)
    # of equal values the lowest ids
    keep = (count > 0)[place]
    whole = torch.bincount(place, minlength=len(val))
    for i in torch.nonzero((count > 0) & (count < whole))[:, 0].tolist():
        ids = torch.nonzero(place == i)[:, 0]
        keep[ids[int(count[i]):]] = False
    return keep, torch.where(keep, unit[place], 0), val[0]


def exact(case, seed):
    s = prepare(case, seed)
    op, R = case["op"], case["R"]
    if op in ("sample", "truncate"):
        rows, kept = live_rows(case), s["kept"].clone()
        t, k, p, mp = (s[n].cpu().numpy().tolist() for n in ("temperature", "top_k", "top_p", "min_p"))
        u = s["u"].double().cpu().numpy()
        got = {"out": s["out"].double()} if op == "truncate" else \
            {"tokens": s["tokens"].clone(), "logq": s["logq"].double()}
        for r in range(R):
            for j in range(int(rows[r])):
                x = s["logits"][r, j]
                keep, w, top = exact_row(x, t[r], k[r], p[r], mp[r])
                kept[r, j] = keep.sum()
                if op == "truncate":
                    got["out"][r, j] = torch.where(keep, x.double(), float("-inf"))
                    continue
                sums = torch.cumsum(w, 0)
                total = float(sums[-1])
                i = int(torch.searchsorted(sums, math.floor(u[r, j] * total), right=True))
                got["tokens"][r, j] = i
                got["logq"][r, j] = float((x[i].double() - top) / (t[r] or 1.0)) - math.log(total / UNIT)
        return {**got, "kept": kept}
    if op == "bounds":
        start, n = spans(case)
        table, page = s["page_table"].cpu().numpy(), case["page"]
        got = {"k_min": s["k_min"].double(), "k_max": s["k_max"].double()}
        for r in range(R):
            first, end = int(start[r]) // page, int(start[r] + n[r])
            where = host(table[r, first:-(-end // page)].astype(np.int64))
            x = s["k_cache"][where].double()
            if s["k_scale"] is not None:
                x = x * s["k_scale"][where].double()[..., None]
            got["k_min"][where], got["k_max"][where] = x.amin(2), x.amax(2)
            last = x[-1, :, :end - (end - 1) // page * page]
            got["k_min"][where[-1]], got["k_max"][where[-1]] = last.amin(1), last.amax(1)
        return got
    ctx, n = lengths(case)
    M, hq, hkv, d, page = (case[k] for k in ("M", "hq", "hkv", "d", "page"))
    G = hq // hkv
    if op == "select":
        lists, table = np.full(tuple(s["lists"].shape), -1, np.int32), s["page_table"].cpu().numpy()
        listed_len = np.zeros(R, np.int32)
        for r in range(R):
            F = int(ctx[r]) // page
            tail = table[r, F:(int(ctx[r]) + int(n[r]) - 1) // page + 1]
            where = host(table[r, :F].astype(np.int64))
            lo, hi = s["k_min"][where].double(), s["k_max"][where].double()
            take = min(F, case["budget"])
            for h in range(hkv):
                q = s["q"][r, :int(n[r]), h * G:(h + 1) * G].double().reshape(-1, d)
                bound = torch.zeros(F, device=DEV, dtype=torch.float64)
                for row in q:  # every dimension's larger product
                    bound += torch.maximum(lo[:, h] * row, hi[:, h] * row).sum(1)
                bound[:s["first"]] = float("inf")
                bound[max(0, F - s["last"]):] = float("inf")
                best = np.sort(np.argsort(-bound.cpu().numpy(), kind="stable")[:take])
                lists[r, h, :take] = table[r][best]
                lists[r, h, take:take + len(tail)] = tail
            listed_len[r] = take * page + int(ctx[r]) % page
        return {"lists": host(lists), "listed": host(listed_len)}
    full, tok, _ = listed_tokens(case)
    see = trees(case, seed, n) if case["tree"] else np.tril(np.ones((M, M), bool))[None].repeat(R, 0)
    out, lse = s["out"].double(), s["lse"].double()
    lists = s["lists"].cpu().numpy()
    for r in range(R):
        c, m = int(tok[r]), int(n[r])
        t = np.arange(c + m)
        off = host(t % page)
        ok = host(np.concatenate([np.ones((m, c), bool), see[r, :m, :m]], 1))
        for h in range(hkv):
            where = host(lists[r, h, t // page].astype(np.int64))
            k, v = (s[name + "_cache"][where, h, off].double() for name in ("k", "v"))
            if s["k_scale"] is not None:
                k = k * s["k_scale"][where, h, off].double()[:, None]
                v = v * s["v_scale"][where, h, off].double()[:, None]
            q = s["q"][r, :m, h * G:(h + 1) * G].double().reshape(m * G, d)
            x = (q @ k.T.contiguous()) * s["scale"]
            x = x.reshape(m, G, -1).masked_fill(~ok[:, None, :], float("-inf"))
            lse[r, :m, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            out[r, :m, h * G:(h + 1) * G] = (torch.softmax(x, -1).reshape(m * G, -1) @ v).reshape(m, G, -1)
    return {"out": out, "lse": lse}
