"""Host checks of the paged-cache entry points (no GPU needed): bad arguments
are refused before anything is enqueued."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "lossless_verification_sampling_amd", "libspecverify.so")
OK, EINVAL, EDTYPE, EWORKSPACE, EUNSUPPORTED = 0, -1, -2, -3, -5
F32, BF16, E4M3 = 0, 1, 2
P, I, L, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
A = 0x10000                                     # an address that is never touched


@pytest.fixture(scope="module")
def lib():
    assert os.path.exists(LIB), "build the library first (__graft_entry__.build())"
    return ctypes.CDLL(LIB)


def caller(fn, types, defaults):
    fn.restype, fn.argtypes = I, types

    def call(**kw):
        assert set(kw) <= set(defaults), kw
        return fn(*{**defaults, **kw}.values())
    return call


CACHE = dict(k_cache=A, v_cache=A, cache_dtype=BF16, k_scale=None, v_scale=None, num_pages=9,
             page_size=64)
TAIL = dict(ws=A, ws_bytes=1 << 30, stream=None)


@pytest.fixture(scope="module")
def mask(lib):
    return caller(lib.spec_tree_mask, [P, P, P, I, I, I, P, P, P, S, P],
                  dict(parent=A, n=A, ctx=A, R=2, M=9, window=0, pos=A, mask=A, **TAIL))


@pytest.fixture(scope="module")
def write(lib):
    d = dict(q=A, k=A, v=A, dtype=BF16, ld_q=48 * 128, ld_k=48 * 128, ld_v=48 * 128, qw=A, kw=A,
             eps=1e-6, rope=A, max_pos=100, rot=128, inter=0, pos=None, ctx=A, n=A, table=A,
             max_pages=4, R=2, M=9, Hq=32, Hkv=8, D=128, **CACHE, out_q=A, **TAIL)
    return caller(lib.spec_qkv_write, [P, P, P, I, L, L, L, P, P, F, P, I, I, I, P, P, P, P, I, I, I,
                                       I, I, I, P, P, I, P, P, I, I, P, P, S, P], d)


@pytest.fixture(scope="module")
def read(lib):
    d = dict(**CACHE, table=A, max_pages=4, start=A, len=A, R=2, max_len=9, Hkv=8, D=128, out_k=A,
             out_v=A, out_dtype=BF16, **TAIL)
    return caller(lib.spec_kv_read, [P, P, I, P, P, I, I, P, I, P, P, I, I, I, I, P, P, I, P, S, P], d)


@pytest.fixture(scope="module")
def commit(lib):
    d = dict(**CACHE, table=A, max_pages=4, ctx=A, acc=A, path=A, R=2, M=9, Hkv=8, D=128,
             out_ctx=A + 256, **TAIL)
    return caller(lib.spec_kv_commit, [P, P, I, P, P, I, I, P, I, P, P, P, I, I, I, I, P, P, S, P], d)


@pytest.fixture(scope="module")
def attn(lib):
    d = dict(q=A, q_dtype=BF16, **CACHE, table=A, max_pages=4, ctx=A, n=A, mask=A, pos=A, scale=0.1,
             window=0, R=2, M=9, Hq=32, Hkv=8, D=128, out=A, lse=None, **TAIL)
    return caller(lib.spec_tree_attention, [P, I, P, P, I, P, P, I, I, P, I, P, P, P, P, F, I, I, I, I,
                                            I, I, P, P, P, S, P], d)


def test_every_cache_entry_refuses_a_bad_cache(write, read, commit, attn):
    for f in (write, read, commit, attn):
        assert f(num_pages=0) == EINVAL
        assert f(max_pages=-1) == EINVAL
        assert f(Hkv=0) == EINVAL
        assert f(cache_dtype=F32) == EDTYPE and f(cache_dtype=7) == EDTYPE
        assert f(D=96) == EUNSUPPORTED and f(D=0) == EINVAL
        assert f(page_size=8) == EUNSUPPORTED and f(page_size=48) == EUNSUPPORTED
        assert f(page_size=2048) == EUNSUPPORTED and f(page_size=0) == EINVAL
        assert f(k_cache=None) == EINVAL and f(v_cache=None) == EINVAL
        assert f(table=None) == EINVAL
        assert f(cache_dtype=E4M3) == EINVAL                        # scales missing
        assert f(cache_dtype=E4M3, k_scale=A, v_scale=None) == EINVAL
        assert f(k_cache=A + 8) == EINVAL and f(v_cache=A + 2) == EINVAL
        assert f(cache_dtype=E4M3, k_scale=A + 4, v_scale=A) == EINVAL
        assert f(ws=None) == EWORKSPACE and f(ws=A + 16) == EWORKSPACE and f(ws_bytes=255) == EWORKSPACE
        assert f(R=-1) == EINVAL
        assert f(R=0) == OK


def test_tree_mask_arguments(mask):
    assert mask(R=-1) == EINVAL and mask(M=0) == EINVAL and mask(window=-1) == EINVAL
    assert mask(M=1025) == EUNSUPPORTED and mask(R=65536) == EUNSUPPORTED
    for k in ("parent", "n", "ctx", "pos", "mask"):
        assert mask(**{k: None}) == EINVAL, k
    assert mask(ws=None) == EWORKSPACE and mask(ws_bytes=100) == EWORKSPACE
    assert mask(R=0) == OK


def test_qkv_write_arguments(write):
    assert write(M=-1) == EINVAL and write(Hq=-1) == EINVAL and write(eps=-1.0) == EINVAL
    assert write(eps=float("nan")) == EINVAL and write(max_pos=-1) == EINVAL
    assert write(dtype=E4M3) == EDTYPE and write(dtype=5) == EDTYPE
    assert write(rot=24) == EUNSUPPORTED and write(rot=144) == EUNSUPPORTED and write(rot=-16) == EINVAL
    assert write(R=1 << 20, M=1 << 12) == EUNSUPPORTED              # 2^32 tokens
    assert write(Hq=30) == EINVAL                                   # not a multiple of Hkv
    assert write(Hq=0) == EINVAL and write(q=None) == EINVAL
    for k in ("k", "v", "ctx", "n", "out_q", "rope"):
        assert write(**{k: None}) == EINVAL, k
    assert write(rot=0) == EINVAL                                   # a table without a rotation
    assert write(max_pos=0) == EINVAL                               # a rotation without a table
    assert write(ld_q=31 * 128) == EINVAL and write(ld_k=8 * 128 - 8) == EINVAL
    assert write(ld_v=8 * 128 + 4) == EINVAL                        # not 16 bytes
    for k in ("q", "k", "v", "qw", "kw", "rope", "out_q"):
        assert write(**{k: A + 8}) == EINVAL, k
    assert write(M=0) == OK


def test_kv_read_arguments(read):
    assert read(max_len=-1) == EINVAL and read(out_dtype=E4M3) == EDTYPE
    assert read(R=65536) == EUNSUPPORTED
    for k in ("start", "len", "out_k", "out_v"):
        assert read(**{k: None}) == EINVAL, k
    assert read(out_k=A + 8) == EINVAL and read(max_len=0) == OK


def test_kv_commit_arguments(commit):
    assert commit(M=0) == EINVAL and commit(M=1025) == EUNSUPPORTED
    for k in ("ctx", "acc", "path"):
        assert commit(**{k: None}) == EINVAL, k
    assert commit(out_ctx=A) == EINVAL                              # ctx_len itself


def test_tree_attention_arguments(lib, attn):
    w = lib.spec_tree_attention_workspace_bytes
    w.restype, w.argtypes = S, [I] * 5
    assert w(2, 9, 32, 8, 128) > 256 and w(2, 1024, 64, 1, 128) > 256
    assert w(2, 0, 32, 8, 128) == 0 and w(2, 1025, 32, 8, 128) == 0
    assert w(2, 9, 30, 8, 128) == 0 and w(2, 9, 130, 2, 128) == 0 and w(2, 9, 32, 8, 96) == 0
    assert attn(ws_bytes=w(2, 9, 32, 8, 128) - 1) == EWORKSPACE
    assert attn(M=0) == EINVAL and attn(Hq=0) == EINVAL and attn(window=-1) == EINVAL
    assert attn(scale=float("inf")) == EINVAL and attn(scale=float("nan")) == EINVAL
    assert attn(q_dtype=F32) == EDTYPE
    assert attn(Hq=30) == EINVAL and attn(Hq=8 * 65) == EUNSUPPORTED
    assert attn(M=1025) == EUNSUPPORTED and attn(R=65536) == EUNSUPPORTED
    # more units of work than count in 31 bits
    assert attn(R=60000, M=1024, max_pages=1 << 20, page_size=1024) == EUNSUPPORTED
    for k in ("q", "ctx", "n", "out"):
        assert attn(**{k: None}) == EINVAL, k
    assert attn(q=A + 8) == EINVAL and attn(out=A + 8) == EINVAL


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 4, 7])
def test_attention_workspace_covers_smaller_calls(lib, D, G):
    lib.spec_tree_attention_workspace_bytes.restype = S
    last = 0
    for M in list(range(1, 200)) + [256, 1000, 1024]:
        need = lib.spec_tree_attention_workspace_bytes(64, M, 2 * G, 2, D)
        assert need >= last > -1 and need == lib.spec_tree_attention_workspace_bytes(1, M, 2 * G, 2, D)
        last = need


def test_an_empty_write_is_no_fault_whatever_is_null(write):
    """An empty tensor's pointer is null."""
    for size in (dict(R=0), dict(M=0), dict(R=0, M=0)):
        assert write(q=None, out_q=None, **size) == OK
        assert write(q=None, k=None, v=None, out_q=None, ctx=None, n=None, table=None, **size) == OK
        assert write(q=None, Hq=0, out_q=None, **size) == OK
        assert write(Hq=30, **size) == EINVAL and write(Hq=-8, **size) == EINVAL


def test_a_window_over_a_tree_needs_positions(attn):
    """A mask says who is whose ancestor, not how far the context is."""
    assert attn(window=5, pos=None, ws=None) == EINVAL
    # with them, or without a window, or for a chain, the next check is reached
    assert attn(window=5, ws=None) == EWORKSPACE and attn(pos=None, ws=None) == EWORKSPACE
    assert attn(window=5, mask=None, pos=None, ws=None) == EWORKSPACE


def test_more_workgroups_than_a_launch_holds(write, read, commit):
    """2^24 - 1 workgroups of 256 threads are a launch's most."""
    most = (1 << 24) - 1
    assert write(R=1, M=most, ws=None) == EWORKSPACE and write(R=1, M=most + 1) == EUNSUPPORTED
    assert write(R=1 << 12, M=1 << 12, ws=None) == EUNSUPPORTED
    assert read(R=1, max_len=4 * most, ws=None) == EWORKSPACE and read(R=1, max_len=4 * most + 1) == EUNSUPPORTED
    assert commit(R=most, ws=None) == EWORKSPACE and commit(R=most + 1) == EUNSUPPORTED


def test_commit_outputs_are_no_input(commit):
    """A workgroup stores its request's length while its other waves may not have
    read their accepted count yet."""
    assert commit(acc=A + 512, out_ctx=A + 512) == EINVAL
    assert commit(path=A + 512, out_ctx=A + 512) == EINVAL
    assert commit(acc=A + 512, out_ctx=A + 256, ws=None) == EWORKSPACE
    assert commit(acc=A + 512, out_ctx=None, ws=None) == EWORKSPACE
