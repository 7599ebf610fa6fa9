"""Host checks of the draw and truncation entry points (no GPU needed)."""
import pytest
import torch

import fake_gpu
from test_capi_cache_host import A, BF16, E4M3, EDTYPE, EINVAL, EUNSUPPORTED, EWORKSPACE, F32, I, L, OK, P, S, caller, lib  # noqa: F401

TAIL = dict(ws=A, ws_bytes=1 << 30, stream=None)
HEAD = dict(logits=A, dtype=BF16, ld=1000, t=A, k=A, p=A, mp=A, rows=A)


@pytest.fixture(scope="module")
def sample(lib):  # noqa: F811
    d = dict(**HEAD, u=A, R=2, J=3, V=1000, tokens=A, logq=A, kept=A, **TAIL)
    return caller(lib.spec_sample, [P, I, L, P, P, P, P, P, P, I, I, I, P, P, P, P, S, P], d)


@pytest.fixture(scope="module")
def truncate(lib):  # noqa: F811
    d = dict(**HEAD, R=2, J=3, V=1000, out=A + 65536, out_ld=1000, kept=A, **TAIL)
    return caller(lib.spec_truncate_logits, [P, I, L, P, P, P, P, P, I, I, I, P, L, P, P, S, P], d)


def test_arguments(sample, truncate):
    for f in (sample, truncate):
        assert f(R=-1) == EINVAL and f(J=-1) == EINVAL and f(V=0) == EINVAL and f(ld=999) == EINVAL
        assert f(dtype=E4M3) == EDTYPE and f(dtype=9) == EDTYPE
        assert f(V=262145, ld=262145, **({"out_ld": 262145} if f is truncate else {})) == EUNSUPPORTED
        assert f(R=2048, J=2048) == EUNSUPPORTED and f(R=65536, J=65536) == EUNSUPPORTED
        assert f(logits=None) == EINVAL and f(t=None) == EINVAL
        assert f(logits=A + 1) == EINVAL and f(logits=A + 2, dtype=F32) == EINVAL
        assert f(ws=None) == EWORKSPACE and f(ws=A + 8) == EWORKSPACE and f(ws_bytes=255) == EWORKSPACE
        assert f(R=0) == OK and f(J=0) == OK
    assert sample(u=None) == EINVAL and sample(tokens=None) == EINVAL
    assert truncate(out=None) == EINVAL and truncate(out=A + 65537) == EINVAL and truncate(out_ld=999) == EINVAL
    assert truncate(out=A, out_ld=1001) == EINVAL                   # in place, but spaced otherwise


def test_truncation_into_rows_that_overlap(truncate):
    """2 x 3 bf16 rows of 1000: the rows themselves or others, between them or
    apart (EWORKSPACE is what a call that passed the check is stopped by)."""
    def f(off, ld=1000, out_ld=1000, **kw):
        return truncate(out=A + 2 * off, ld=ld, out_ld=out_ld, ws_bytes=0, **kw)
    assert f(0) == f(6000) == f(-6000) == EWORKSPACE
    assert f(1) == f(1000) == f(5999) == f(-1) == f(-5999) == EINVAL
    assert f(0, 2500, 2500) == f(1000, 2500, 2500) == f(1500, 2500, 2500) == f(-1000, 2500, 2500) == EWORKSPACE
    assert f(999, 2500, 2500) == f(1501, 2500, 2500) == f(2500, 2500, 2500) == f(-1501, 2500, 2500) == EINVAL
    assert f(13500, 2500, 2500) == EWORKSPACE and f(12500, 2500, 2500) == f(0, 2500, 2600) == EINVAL
    assert f(13500, 2500, 1000) == f(-6000, 2500, 1000) == EWORKSPACE and f(13499, 2500, 1000) == EINVAL
    # one row has no spacing
    assert f(0, 1000, 1001, R=1, J=1) == f(1000, 1000, 1001, R=1, J=1) == EWORKSPACE
    assert f(999, 1000, 1001, R=1, J=1) == EINVAL


def test_workspace_query(lib, sample, truncate):  # noqa: F811
    size = lib.spec_sample_workspace_bytes
    size.restype = S
    assert size(2, 3, 1000) >= 256 and size(0, 3, 1000) >= 256
    assert size(-1, 3, 1000) == size(2, -1, 1000) == size(2, 3, 0) == size(2, 3, 262145) == size(2048, 2048, 9) == 0
    need = size(2, 3, 1000)
    assert sample(ws_bytes=need - 1) == EWORKSPACE and truncate(ws_bytes=need - 1) == EWORKSPACE


@pytest.fixture(scope="module")
def sv():
    import lossless_verification_sampling_amd as m
    return m


@pytest.fixture
def gpu(sv, monkeypatch):
    sv._sample_bytes.cache_clear()
    yield fake_gpu.install(sv, monkeypatch)
    sv._sample_bytes.cache_clear()


def t(*shape, dtype=torch.float32, index=1):
    return fake_gpu.on(index, torch.zeros(shape, dtype=dtype))


@pytest.mark.parametrize("name", ["spec_sample", "spec_truncate_logits"])
def test_binding_devices_and_streams(sv, gpu, name):
    x, u, T = t(2, 3, 9), t(2, 3), t(2)

    def call(**k):
        return sv.spec_sample(x, u, temperature=T, **k) if name == "spec_sample" else \
            sv.spec_truncate_logits(x, temperature=T, **k)
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
    x, u, T = t(2, 3, 9), t(2, 3), t(2)
    for bad in (t(2, 9), t(2, 3, 9, dtype=torch.float16), t(2, 3, 0), t(2, 9, 3).transpose(1, 2)):
        with pytest.raises((ValueError, TypeError)):
            sv.spec_sample(bad, u, temperature=T)
        with pytest.raises((ValueError, TypeError)):
            sv.spec_truncate_logits(bad, temperature=T)
    for kw in (dict(temperature=t(3)), dict(temperature=t(2, index=0)), dict(temperature=T, top_k=t(2)),
               dict(temperature=T, top_p=t(2, dtype=torch.int32)), dict(temperature=T, min_p=t(2, 1)),
               dict(temperature=T, rows=t(2, dtype=torch.int64))):
        with pytest.raises((ValueError, TypeError)):
            sv.spec_sample(x, u, **kw)
        with pytest.raises((ValueError, TypeError)):
            sv.spec_truncate_logits(x, **kw)
    with pytest.raises(ValueError):
        sv.spec_sample(x, t(2, 2), temperature=T)
    with pytest.raises(ValueError):
        sv.spec_truncate_logits(x, temperature=T, out=t(2, 3, 9, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        sv.spec_truncate_logits(x, temperature=T, out=t(2, 3, 9, index=0))
    assert not any(c[0] in ("spec_sample", "spec_truncate_logits") for c in gpu.calls)
    padded = t(2, 3, 16)[:, :, :9]
    sv.spec_sample(padded, u, temperature=T)
    assert gpu.calls[-1][3][2] == 16
    sv.spec_truncate_logits(padded, temperature=T)
    assert gpu.calls[-1][3][2] == 16 and gpu.calls[-1][3][12] == 9
