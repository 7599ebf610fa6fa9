"""Seeded inputs of the paged-cache tests and the fp64 reference over whole
batches."""
from __future__ import annotations

import numpy as np
import torch

from oracle import cache as oc

BF16_U = 2.0 ** -8      # half a step of bf16, relative


def bf16(x):
    """fp32 values rounded to bf16."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def random_trees(g, R, M, n, chain=False):
    p = np.full((R, M), -1, np.int32)
    for r in range(R):
        for v in range(1, int(n[r])):
            p[r, v] = v - 1 if chain else g.integers(max(0, v // 3 - 2), v)
    return p


class Cache:
    """Pages filled with random rows, page tables of distinct shuffled pages."""

    def __init__(self, g, R, tokens, Hkv, D, page, kind, spare=2):
        self.wide = -(-tokens // page)
        P = R * self.wide + spare
        self.page, self.kind, self.P, self.Hkv, self.D = page, kind, P, Hkv, D
        self.table = g.permutation(P)[:R * self.wide].reshape(R, self.wide).astype(np.int32)
        x = [g.standard_normal((P, Hkv, page, D)).astype(np.float32) for _ in range(2)]
        self.scales = [None, None]
        if kind == "bf16":
            self.dev = [bf16(t) for t in x]
        else:
            qs = [oc.quantise(t * np.float32(3.0)) for t in x]
            self.dev = [torch.from_numpy(c.astype(np.float32)).to(torch.float8_e4m3fn) for c, _ in qs]
            self.scales = [torch.from_numpy(s) for _, s in qs]

    def to(self, dev):
        self.dev = [t.to(dev) for t in self.dev]
        self.scales = [None if t is None else t.to(dev) for t in self.scales]
        self.t = torch.from_numpy(self.table).to(dev)
        return self

    def args(self):
        return self.dev[0], self.dev[1], self.t

    def kw(self):
        return dict(k_scale=self.scales[0], v_scale=self.scales[1])

    def rows(self, which, r, first, count):
        """fp64 values [count, Hkv, D] the request's tokens stand for."""
        t = np.arange(first, first + count)
        pg, off = self.table[r, t // self.page], t % self.page
        x = self.dev[which].float().cpu().numpy().astype(np.float64)[pg, :, off]
        if self.scales[which] is not None:
            x = x * self.scales[which].cpu().numpy().astype(np.float64)[pg, :, off][..., None]
        return x


def reference_attention(cache, q, ctx, n, see, pos, scale, window, chain):
    """fp64 out [R, M, Hq, D], lse and their tolerances; rows v >= n are NaN."""
    R, M, Hq, D = q.shape
    G = Hq // cache.Hkv
    out, lse = np.full(q.shape, np.nan), np.full(q.shape[:3], np.nan)
    to, tl = np.zeros(q.shape), np.zeros(q.shape[:3])
    for r in range(R):
        c, m = int(ctx[r]), int(n[r])
        k, v = cache.rows(0, r, 0, c + m), cache.rows(1, r, 0, c + m)
        ok = np.zeros((m, c + m), bool)
        for i in range(m):
            j = np.arange(c + m)
            ok[i] = (j < c) & ((j > pos[r, i] - window) if window else True)
            if chain:
                ok[i] |= (j >= c) & (j - c <= i) & ((i - (j - c) < window) if window else True)
            else:
                ok[i, c:] |= see[r, i, :m]
        for h in range(Hq):
            o, l, a, s = oc.attention(q[r, :m, h], k[:, h // G], v[:, h // G], ok, scale)
            out[r, :m, h], lse[r, :m, h] = o, l
            # scores: D + 4 roundings of fp32 sums of |q k|, and the same again
            # for the exponent's argument; output and weights: one bf16
            # rounding each
            ds = 2 * (D + 4) * 2.0 ** -24 * s
            to[r, :m, h] = np.abs(o) * BF16_U + a * (BF16_U + 2 * ds[:, None] + (c + m) * 2.0 ** -24
                                                     + 2.0 ** -20) + 1e-37
            with np.errstate(invalid="ignore"):
                tl[r, :m, h] = ds + 2.0 ** -20 + (c + m) * 2.0 ** -24 + np.abs(l) * 2.0 ** -22
    return out, lse, to, tl
