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


@pytest.mark.parametrize("name", fake_gpu.NAMES)
def test_a_given_stream_writes_memory_of_its_own(sv, gpu, name):
    """A block that the current stream freed may still be read by what is queued
    there: neither an output nor a workspace for another stream may be one."""
    st = fake_gpu.Stream(1, 9)
    fake_gpu.calls(sv, 1)[name](stream=st)
    assert gpu.taken and all(t.pool is st for t in gpu.taken)
    assert all(t.used == [0] for t in gpu.taken)        # the caller's stream may read them
    assert {n: s for n, _, s, _ in gpu.calls} == {"spec_workspace_init": 9, name: 9}
    assert gpu.streams[1].cuda_stream == 0 and gpu.current == 0


@pytest.mark.parametrize("name", fake_gpu.NAMES)
def test_a_workspace_outlasts_every_stream_it_is_used_on(sv, gpu, name):
    call, ws = fake_gpu.calls(sv, 1)[name], sv.Workspace("cuda:1", 256)
    for st in (9, 9, 8, 9):
        call(stream=fake_gpu.Stream(1, st), workspace=ws)
    with torch.cuda.stream(fake_gpu.Stream(1, 5)):
        call(workspace=ws)
    assert ws.buf.pool.cuda_stream == 0 and ws.buf.used == [9, 8, 5]


def test_a_workspace_that_grows_in_small_steps_keeps_little(sv, gpu):
    """The buffers that it outgrew are kept for captured graphs."""
    ws, last = sv.Workspace("cuda:1", 256), 0
    for need in range(70000, 3000000, 4096):
        assert ws.ensure(need).numel() >= need and ws.nbytes == ws.buf.numel()
        last = need
    assert sum(t.numel() for t in gpu.taken) <= 4 * last


def test_status_words_of_outgrown_buffers_count(sv, gpu):
    ws = sv.Workspace("cuda:1", 1 << 16)
    for _ in range(2):
        ws.ensure(ws.nbytes + 1)
    first, second, last = (t.data_ptr() for t in gpu.taken)
    gpu.status = {first: 1, second: 2}          # a replay's, and one from before the growth
    assert sv.spec_get_device_status(ws, clear=False) == 3
    assert sv.spec_get_device_status(ws) == 3
    assert sv.spec_get_device_status(ws) == 0
    gpu.status[last] = 1
    assert sv.spec_get_device_status(ws) == 1 and not any(gpu.status.values())
    sv.spec_get_device_status(ws, stream=fake_gpu.Stream(1, 9))
    assert [(d, s) for _, d, s, _ in gpu.calls[-3:]] == [(1, 9)] * 3
    assert sv.spec_get_device_status(sv.Workspace("cuda:1")) == 0


@pytest.mark.parametrize("name", fake_gpu.NAMES)
def test_a_workspace_taken_inside_a_capture_is_the_graphs(sv, gpu, name):
    """What a capture records has not run: the buffer that it took holds whatever
    its memory held.  Calls outside take one of their own, and clear it."""
    call = fake_gpu.calls(sv, 1)[name]
    gpu.capturing = True
    call()
    call()
    assert [n for n, *_ in gpu.calls] == ["spec_workspace_init", name, name]
    inside = gpu.calls[0][3][0].value
    gpu.capturing = False
    gpu.calls.clear()
    call()
    call()
    gpu.capturing = True                        # a later capture finds a cleared one
    call()
    assert [n for n, *_ in gpu.calls] == ["spec_workspace_init", name, name, name]
    assert gpu.calls[0][3][0].value != inside


def test_the_status_of_a_workspace_taken_inside_a_capture(sv, gpu):
    """Its status word counts, unless it holds what no call writes."""
    ws = sv.Workspace("cuda:1")
    gpu.capturing = True
    ws.ensure(256)
    gpu.capturing = False
    first = ws.buf.data_ptr()
    ws.ensure(256)
    last = ws.buf.data_ptr()
    gpu.status = {first: 0xffffffff, last: 1}
    assert sv.spec_get_device_status(ws) == 1
    gpu.status = {first: 2, last: 1}
    assert sv.spec_get_device_status(ws) == 3 and not any(gpu.status.values())


@pytest.mark.parametrize("name,arg", [("spec_tree_mask", "window"), ("spec_tree_attention", "window"),
                                      ("spec_schedule_verify_len", "topk"), ("spec_sts_calibrate", "bins")])
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1, 2 ** 64 + 1])
def test_numbers_past_32_bits_are_refused(sv, gpu, name, arg, value):
    """ctypes would keep their low 32 bits: a window of 2^32 + 5 would be one of 5."""
    with pytest.raises(ValueError):
        fake_gpu.calls(sv, 1)[name](**{arg: value})
    assert not [n for n, *_ in gpu.calls if n == name]
    fake_gpu.calls(sv, 1)[name](**{arg: 2 ** 31 - 1})
    assert [n for n, *_ in gpu.calls if n == name]
