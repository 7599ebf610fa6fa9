"""The narrowing of the page scores' key range (csrc/page_cut.h) on the host, with plain
counts, against a sort."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lossless_verification_sampling_amd", "csrc")

SOURCE = r"""
#include <vector>
#include "page_cut.h"
// the chosen of n keys (flags), by the cut behind the `want` largest; returns the levels it
// took, or -1 if a level found no part
extern "C" int choose(const uint64_t *keys, int n, uint32_t want, unsigned char *in) {
    uint64_t lo = ~0ull, hi = 0;
    for (int i = 0; i < n; ++i) {
        if (keys[i] < lo) lo = keys[i];
        if (keys[i] > hi) hi = keys[i];
    }
    int levels = 0;
    bool lost = false;
    const sv::KeyCut cut = sv::key_cut(lo, hi, want, [&](uint64_t lo, uint64_t hi, int shift, uint32_t want) {
        std::vector<uint32_t> count(sv::kParts);
        for (int i = 0; i < n; ++i)
            if (keys[i] >= lo && keys[i] <= hi) ++count.at((keys[i] - lo) >> shift);
        ++levels;
        uint32_t before = 0;
        for (int p = sv::kParts - 1; p >= 0; --p) {
            if (before < want && before + count[p] >= want)
                return sv::CutPart{(uint64_t)p, count[p], want - before};
            before += count[p];
        }
        lost = true;
        return sv::CutPart{0, 1, 1};
    });
    uint32_t tie = 0;
    for (int i = 0; i < n; ++i) {
        in[i] = keys[i] > cut.key || (keys[i] == cut.key && tie < cut.ties);
        tie += keys[i] == cut.key;
    }
    return lost ? -1 : levels;
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    d = tmp_path_factory.mktemp("page_cut")
    (d / "cut.cpp").write_text(SOURCE)
    so = str(d / "cut.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-I" + CSRC, "-o", so,
                           str(d / "cut.cpp")])
    lib = ctypes.CDLL(so)

    def run(keys, want):
        keys = np.ascontiguousarray(keys, np.uint64)
        out = np.zeros(len(keys), np.uint8)
        levels = lib.choose(keys.ctypes.data_as(ctypes.c_void_p), len(keys), ctypes.c_uint32(want),
                            out.ctypes.data_as(ctypes.c_void_p))
        assert 1 <= levels <= 6
        return np.flatnonzero(out).tolist()
    return run


def keys_of(scores):
    """Whole numbers in the order of the scores; NaN stands with +infinity."""
    s = np.asarray(scores, np.float64)
    b = (np.where(np.isnan(s), np.inf, s) + 0.0).view(np.uint64)
    return np.where(b >> np.uint64(63), ~b, b | np.uint64(1 << 63))


def best(keys, want):
    order = sorted(range(len(keys)), key=lambda i: (-int(keys[i]), i))
    return sorted(order[:want])


@pytest.mark.parametrize("scores, want", [
    ([-1.0, 5.0, math.nan, math.nan], 1),
    ([-100.0, 5.0] + [math.inf] * 10, 4),
    ([math.inf] * 3 + [-math.inf] * 3, 2),
    ([-math.inf, 0.0, math.inf, math.inf], 1),
    ([-math.inf] * 4, 2),
    ([-1.0] + [1.7976931348623157e308] * 3 + [math.inf] * 2, 4),
])
def test_more_infinite_scores_than_places(choose, scores, want):
    keys = keys_of(scores)
    assert choose(keys, want) == best(keys, want)


@pytest.mark.parametrize("seed", range(8))
def test_random_scores(choose, seed):
    g = np.random.default_rng(seed)
    special = np.array([np.inf, -np.inf, np.nan, 0.0, -0.0, 5e-324, -5e-324, 1.7976931348623157e308,
                        -1.7976931348623157e308])
    for _ in range(400):
        n = int(g.integers(2, 80))
        s = g.standard_normal(n) * 10.0 ** g.integers(-300, 300)
        at = g.random(n) < g.random()
        s[at] = g.choice(special[:int(g.integers(1, 10))], at.sum())
        keys = keys_of(s)
        want = int(g.integers(1, n + 1))
        assert choose(keys, want) == best(keys, want), (s.tolist(), want)


@pytest.mark.parametrize("seed", range(4))
def test_random_keys(choose, seed):
    """Keys of the whole range, in knots of neighbours."""
    g = np.random.default_rng(100 + seed)
    for _ in range(300):
        n = int(g.integers(2, 60))
        knots = g.integers(1, 2 ** 64, 3, dtype=np.uint64, endpoint=False)
        knots[g.random(3) < 0.3] = np.uint64(2 ** 64 - 1)
        near = g.integers(0, 2 ** int(g.integers(1, 54)), n, dtype=np.uint64)
        base = g.choice(knots, n)
        keys = np.maximum(np.where(base > near, base - near, base), np.uint64(1))
        want = int(g.integers(1, n + 1))
        assert choose(keys, want) == best(keys, want), (keys.tolist(), want)
