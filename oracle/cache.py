"""Plain CPU oracle of the paged-cache operators, in fp64.

TEST INFRASTRUCTURE ONLY: the tests, the smoke check and the benchmark may
call this; the product library never does.  It shares no code with the HIP
library.

Definitions (the C ABI header states them in full): node v of request r is
cache token ctx_len[r] + v; a tree node sees the context and its ancestors; a
chain node sees the context and every earlier node.  fp32 / fp64 arrays are
used throughout; e4m3 pages are arrays of code values (fp64) beside their
scales.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126


def e4m3_round(x):
    """Nearest e4m3 value, ties to the even code (|x| <= 448; 3 mantissa bits,
    smallest normal 2^-6, subnormal step 2^-9)."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(np.where(x == 0, 1.0, np.abs(x)))
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(x / step) * step


def quantise(x32):
    """(code values, fp32 scale) of fp32 rows [..., D]."""
    x32 = np.asarray(x32, np.float32)
    fin = np.isfinite(x32).all(-1)
    amax = np.where(fin, np.abs(np.where(np.isfinite(x32), x32, 0)).max(-1), 0).astype(np.float32)
    s = np.maximum(amax / np.float32(E4M3_MAX), np.float32(MIN_SCALE)).astype(np.float32)
    with np.errstate(invalid="ignore"):
        y = (x32 / s[..., None]).astype(np.float32)
    codes = e4m3_round(np.where(fin[..., None], y, 0))
    return codes, np.where(fin, s, np.float32(np.nan))


def tree_mask(parent, n_nodes, ctx_len, window=0):
    """(positions [R, M], see [R, M, M] bool); a faulty request gets -1 and
    nothing."""
    R, M = parent.shape
    pos = np.full((R, M), -1, np.int32)
    see = np.zeros((R, M, M), bool)
    for r in range(R):
        n, c = int(n_nodes[r]), int(ctx_len[r])
        if not 0 <= n <= M or c < 0 or c + M > 2 ** 31 - 1:
            continue
        if any(not 0 <= parent[r, v] < v for v in range(1, n)):
            continue
        for v in range(n):
            path, u = [v], v
            while u:
                u = int(parent[r, u])
                path.append(u)
            pos[r, v] = c + len(path) - 1
            see[r, v, path[:window] if window else path] = True
    return pos, see


def pack_bits(see):
    """[R, M, M] bool as [R, M, W] int32 words."""
    R, M, N = see.shape
    W = (N + 31) // 32
    out = np.zeros((R, M, W), np.uint32)
    for u in range(N):
        out[:, :, u // 32] |= see[:, :, u].astype(np.uint32) << np.uint32(u % 32)
    return out.view(np.int32)


def norm_rotate(x, weight, eps, rope, pos, interleaved):
    """fp64 norm and rotation of one token's head rows [H, D]."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if rope is None:
        return x
    cs = np.asarray(rope[pos], np.float64)
    h = cs.shape[0]
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    y = x.copy()
    y[..., a] = x[..., a] * cs[:, 0] - x[..., b] * cs[:, 1]
    y[..., b] = x[..., b] * cs[:, 0] + x[..., a] * cs[:, 1]
    return y


def attention(q, k, v, see, scale):
    """One head group in fp64: q [N, D], k, v [L, D], see [N, L].  Returns
    (o [N, D], lse [N], a [N, D] = sum p |v|, ds [N] = the largest sum of
    |q_i k_i| * scale over the seen tokens).  Unseen tokens have no part."""
    N, L = see.shape
    o, lse = np.zeros((N, q.shape[1])), np.full(N, -np.inf)
    a, ds = np.zeros_like(o), np.zeros(N)
    for i in range(N):
        j = np.flatnonzero(see[i])
        if not len(j):
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            s = (k[j] @ q[i]) * scale
            m = s.max()
            p = np.exp(s - m)
            t = p.sum()
            p = p / t
            o[i], a[i], lse[i] = p @ v[j], p @ np.abs(v[j]), m + np.log(t)
            ds[i] = (np.abs(k[j]) @ np.abs(q[i])).max() * abs(scale)
    return o, lse, a, ds
