"""The Python binding's devices, streams and workspaces, on the CPU with a
stand-in for two GPUs (no GPU needed)."""
import pytest
import torch

import fake_gpu


@pytest.fixture(scope="module")
def sv():
    import lossless_verification_sampling_amd as m
    return m


@pytest.fixture
def gpu(sv, monkeypatch):
    yield fake_gpu.install(sv, monkeypatch)
    sv._attention_bytes.cache_clear()


@pytest.mark.parametrize("name", fake_gpu.NAMES)
def test_calls_run_with_the_tensors_device_current(sv, gpu, name):
    """Stream 0 is the current device's null stream: a call for tensors on GPU 1
    that left GPU 0 current would run there, its workspace's clearing too."""
    call = fake_gpu.calls(sv, 1)[name]
    for _ in range(2):                          # a workspace to clear, and none
        call()
    ran = [(n, d) for n, d, *_ in gpu.calls]
    assert ran == [("spec_workspace_init", 1), (name, 1), (name, 1)]
    assert gpu.current == 0


def test_a_workspace_is_used_on_its_device(sv, gpu):
    ws = sv.Workspace("cuda:1", 256)
    ws.ensure(1 << 20)                          # and when it grows
    sv.spec_workspace_init(ws)
    sv.spec_get_device_status(ws)
    assert {d for _, d, *_ in gpu.calls} == {1} and len(gpu.calls) >= 4
    assert gpu.current == 0


@pytest.mark.parametrize("name", fake_gpu.NAMES)
def test_a_stream_of_another_device_is_refused(sv, gpu, name):
    call = fake_gpu.calls(sv, 1)[name]
    for ws in (None, sv.Workspace("cuda:1", 256)):
        before = len(gpu.calls)
        with pytest.raises(ValueError):
            call(stream=fake_gpu.Stream(0, 7), workspace=ws)
        assert len(gpu.calls) == before
    call()                                      # and nothing is left half done
    assert [n for n, *_ in gpu.calls[-2:]] == ["spec_workspace_init", name]
