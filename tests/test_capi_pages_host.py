"""Host checks of the page entry points (no GPU needed): bad arguments are
refused before anything is enqueued."""
import pytest
import torch

import fake_gpu
from test_capi_cache_host import (A, BF16, E4M3, EDTYPE, EINVAL, EUNSUPPORTED, EWORKSPACE, F32, OK, P, I, F, S,
                                  CACHE, TAIL, caller, lib)  # noqa: F401


@pytest.fixture(scope="module")
def bounds(lib):  # noqa: F811
    d = dict(k_cache=A, cache_dtype=BF16, k_scale=None, num_pages=9, page_size=64, table=A, max_pages=4,
             start=A, len=A, R=2, max_len=9, Hkv=8, D=128, lo=A, hi=A, **TAIL)
    return caller(lib.spec_page_bounds, [P, I, P, I, I, P, I, P, P, I, I, I, I, P, P, P, S, P], d)


@pytest.fixture(scope="module")
def select(lib):  # noqa: F811
    d = dict(q=A, q_dtype=BF16, lo=A, hi=A, num_pages=9, page_size=64, table=A, max_pages=4, ctx=A, n=A,
             budget=3, first=1, last=1, R=2, M=9, Hq=32, Hkv=8, D=128, lists=A, width=5, out_len=A, **TAIL)
    lib.spec_page_select_workspace_bytes.restype = S
    return caller(lib.spec_page_select, [P, I, P, P, I, I, P, I, P, P, I, I, I, I, I, I, I, I, P, I, P, P, S, P], d)


@pytest.fixture(scope="module")
def attn(lib):  # noqa: F811
    d = dict(q=A, q_dtype=BF16, **CACHE, table=A, max_pages=4, ctx=A, n=A, mask=A, scale=0.1,
             R=2, M=9, Hq=32, Hkv=8, D=128, out=A, lse=None, **TAIL)
    return caller(lib.spec_page_attention, [P, I, P, P, I, P, P, I, I, P, I, P, P, P, F, I, I, I, I, I,
                                            P, P, P, S, P], d)


def test_bad_pages_are_refused(bounds, select, attn):
    for f in (bounds, select, attn):
        assert f(num_pages=0) == EINVAL and f(max_pages=-1) == EINVAL and f(Hkv=0) == EINVAL
        assert f(D=96) == EUNSUPPORTED and f(D=0) == EINVAL
        assert f(page_size=8) == EUNSUPPORTED and f(page_size=48) == EUNSUPPORTED
        assert f(page_size=2048) == EUNSUPPORTED and f(page_size=0) == EINVAL
        assert f(table=None) == EINVAL
        assert f(ws=None) == EWORKSPACE and f(ws=A + 16) == EWORKSPACE and f(ws_bytes=255) == EWORKSPACE
        assert f(R=-1) == EINVAL and f(R=65536) == EUNSUPPORTED
        assert f(R=0) == OK


def test_page_bounds_arguments(bounds):
    assert bounds(cache_dtype=F32) == EDTYPE
    assert bounds(cache_dtype=E4M3) == EINVAL and bounds(cache_dtype=E4M3, k_scale=A + 4) == EINVAL
    assert bounds(max_len=-1) == EINVAL and bounds(max_len=0) == OK
    for k in ("k_cache", "start", "len", "lo", "hi"):
        assert bounds(**{k: None}) == EINVAL, k
    for k in ("k_cache", "lo", "hi"):
        assert bounds(**{k: A + 8}) == EINVAL, k
    big = dict(max_pages=1 << 27, max_len=2147483647, page_size=16)
    assert bounds(**big) == EUNSUPPORTED                            # 2^30 workgroups
    assert bounds(**big, Hkv=1) == EUNSUPPORTED


def test_page_select_arguments(select):
    assert select(q_dtype=F32) == EDTYPE
    assert select(M=0) == EINVAL and select(Hq=0) == EINVAL and select(Hq=30) == EINVAL
    assert select(budget=-1) == EINVAL and select(first=-1) == EINVAL and select(last=-1) == EINVAL
    assert select(first=2, last=2) == EINVAL                        # more than the budget
    assert select(first=2147483647, last=2147483647) == EINVAL
    assert select(M=1025) == EUNSUPPORTED and select(Hq=8 * 65) == EUNSUPPORTED
    assert select(width=4) == EINVAL                                # 3 chosen, 9 nodes over two pages
    assert select(width=5, budget=4) == EINVAL
    assert select(width=5, budget=2147483647, first=0, last=0) == EINVAL
    assert select(width=2147483647, R=0) == OK
    for k in ("q", "lo", "hi", "ctx", "n", "lists", "out_len"):
        assert select(**{k: None}) == EINVAL, k
    for k in ("q", "lo", "hi"):
        assert select(**{k: A + 8}) == EINVAL, k


def test_page_select_workspace(lib, select):  # noqa: F811
    size = lib.spec_page_select_workspace_bytes
    assert size(2, 8, 128, 4) == 256 + 16 * (4 + 256) * 8
    assert size(0, 8, 128, 4) == 256
    assert size(-1, 8, 128, 4) == size(2, 0, 128, 4) == size(2, 8, 96, 4) == size(2, 8, 128, -1) == 0
    assert size(65536, 8, 128, 4) == 0
    assert select(ws_bytes=size(2, 8, 128, 4) - 1) == EWORKSPACE


def test_page_attention_arguments(attn):
    assert attn(q_dtype=F32) == EDTYPE and attn(cache_dtype=F32) == EDTYPE
    assert attn(M=0) == EINVAL and attn(Hq=30) == EINVAL
    assert attn(scale=float("nan")) == EINVAL and attn(scale=float("inf")) == EINVAL
    assert attn(M=1025) == EUNSUPPORTED and attn(Hq=8 * 65) == EUNSUPPORTED
    for k in ("q", "k_cache", "v_cache", "ctx", "n", "out"):
        assert attn(**{k: None}) == EINVAL, k
    for k in ("q", "out", "k_cache"):
        assert attn(**{k: A + 8}) == EINVAL, k
    assert attn(cache_dtype=E4M3, k_scale=A) == EINVAL
    assert attn(max_pages=1 << 28) == EUNSUPPORTED                  # token units past 31 bits


# ---------------------------------------------------------------------------
# the binding, on a stand-in for two GPUs
# ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def sv():
    import lossless_verification_sampling_amd as m
    return m


@pytest.fixture
def gpu(sv, monkeypatch):
    yield fake_gpu.install(sv, monkeypatch)
    sv._attention_bytes.cache_clear()


def binding_calls(sv, index):
    def t(*shape, dtype=torch.float32):
        return fake_gpu.on(index, torch.zeros(shape, dtype=dtype))

    i32, bf = torch.int32, torch.bfloat16
    R, M, D = 2, 3, 64
    n, ctx, table, lists = t(R, dtype=i32), t(R, dtype=i32), t(R, 1, dtype=i32), t(R, 1, 2, dtype=i32)
    page, box, x = t(2, 1, 16, D, dtype=bf), t(2, 1, D, dtype=bf), t(R, M, 1, D, dtype=bf)
    return {
        "spec_page_bounds": lambda **k: sv.spec_page_bounds(page, table, ctx, n, 3, box, box, **k),
        "spec_page_select": lambda **k: sv.spec_page_select(x, box, box, table, ctx, n, 4, 16, **k),
        "spec_page_attention": lambda **k: sv.spec_page_attention(x, page, page, lists, ctx, n, want_lse=True, **k),
    }


@pytest.mark.parametrize("name", ["spec_page_bounds", "spec_page_select", "spec_page_attention"])
def test_binding_devices_and_streams(sv, gpu, name):
    call = binding_calls(sv, 1)[name]
    for _ in range(2):
        call()
    assert [(n, d) for n, d, *_ in gpu.calls] == [("spec_workspace_init", 1), (name, 1), (name, 1)]
    assert gpu.current == 0
    for ws in (None, sv.Workspace("cuda:1", 256)):
        before = len(gpu.calls)
        with pytest.raises(ValueError):
            call(stream=fake_gpu.Stream(0, 7), workspace=ws)
        assert len(gpu.calls) == before
    gpu.taken.clear()
    st = fake_gpu.Stream(1, 9)
    call(stream=st, workspace=sv.Workspace("cuda:1"))
    assert gpu.taken and all(x.pool is st for x in gpu.taken)


def test_binding_refusals(sv, gpu):
    def t(*shape, dtype=torch.float32, index=1):
        return fake_gpu.on(index, torch.zeros(shape, dtype=dtype))

    i32, bf = torch.int32, torch.bfloat16
    x, box, n = t(2, 3, 4, 64, dtype=bf), t(5, 2, 64, dtype=bf), t(2, dtype=i32)
    table, page = t(2, 4, dtype=i32), t(5, 2, 16, 64, dtype=bf)
    good = (x, box, box, table, n, n, 2, 16)
    lists, length = sv.spec_page_select(*good)
    assert tuple(lists.shape) == (2, 2, 2 + 17 // 16 + 1) and tuple(length.shape) == (2,)
    for i, bad in ((0, t(2, 3, 4, 128, dtype=bf)), (0, x.float()), (1, t(5, 2, 64)), (2, t(5, 1, 64, dtype=bf)),
                   (3, t(2, 4)), (3, t(3, 4, dtype=i32)), (4, t(3, dtype=i32)), (5, t(2, dtype=i32, index=0)),
                   (6, -1), (6, 1 << 31), (7, 0)):
        args = list(good)
        args[i] = bad
        with pytest.raises((ValueError, TypeError)):
            sv.spec_page_select(*args)
    with pytest.raises(ValueError):
        sv.spec_page_select(*good, out_lists=t(2, 1, 9, dtype=i32))
    with pytest.raises(ValueError):
        sv.spec_page_attention(x, page, page, table, n, n)          # a table is no list
    with pytest.raises(ValueError):
        sv.spec_page_attention(x, page, page, t(2, 1, 4, dtype=i32), n, n)
    with pytest.raises(ValueError):
        sv.spec_page_bounds(page, table, n, n, 4, t(5, 2, 64, dtype=bf), t(4, 2, 64, dtype=bf))
    with pytest.raises(ValueError):
        sv.spec_page_bounds(page.to(torch.float8_e4m3fn), table, n, n, 4, box, box)   # no scales
    assert not any(c[0] == "spec_page_bounds" for c in gpu.calls)
