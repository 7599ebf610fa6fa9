"""A stand-in for two GPUs, so that the binding's handling of devices, streams
and workspaces is seen on the CPU: which device is current, and which stream,
when memory is taken and when the library is called."""
from __future__ import annotations

import ctypes

import torch


class Stream:
    def __init__(self, index, handle):
        self.device, self.device_index, self.cuda_stream = torch.device("cuda", index), index, handle


class Tensor(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    index, pool = 1, None                       # pool: the stream whose memory it is

    device = property(lambda self: torch.device("cuda", self.index))
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index

    def record_stream(self, stream):
        self.used = getattr(self, "used", []) + [stream.cuda_stream]


def on(index, x):
    t = x.as_subclass(Tensor)
    t.index = index
    return t


class Fake:
    """calls: (name, current device, stream handle) of every library call;
    taken: every tensor that was allocated."""

    def __init__(self):
        self.current = 0
        self.streams = {0: Stream(0, 0), 1: Stream(1, 0)}      # current ones
        self.calls, self.taken, self.status = [], [], {}

    # ---- torch
    def empty(self, *shape, dtype=torch.float32, device=None, **_):
        if len(shape) == 1 and not isinstance(shape[0], int):
            shape = tuple(shape[0])
        d = torch.device(device)
        t = on(self.current if d.index is None else d.index, self.real_empty(shape, dtype=dtype))
        t.pool = self.streams[t.index]
        self.taken.append(t)
        return t

    def device(self, d):
        index = d if isinstance(d, int) else d.index

        class Guard:
            def __enter__(_):
                _.was, self.current = self.current, self.current if index is None else index

            def __exit__(_, *e):
                self.current = _.was
        return Guard()

    def stream(self, s):
        class Guard:
            def __enter__(_):
                if s is not None:
                    _.was = self.current, self.streams[s.device_index]
                    self.current = s.device_index
                    self.streams[s.device_index] = s

            def __exit__(_, *e):
                if s is not None:
                    self.current, self.streams[s.device_index] = _.was
        return Guard()

    def current_stream(self, d=None):
        index = d if isinstance(d, int) or d is None else torch.device(d).index
        return self.streams[self.current if index is None else index]

    # ---- the library
    def __getattr__(self, name):
        if not name.startswith("spec_"):
            raise AttributeError(name)

        def call(*args):
            if name.endswith("_bytes"):
                return 1 << 16
            if name == "spec_get_device_status":
                at = args[0].value
                args[1]._obj.value = self.status.get(at, 0)
                if args[2]:
                    self.status[at] = 0
            self.calls.append((name, self.current, args[-1], args))
            return 0
        return call


def install(sv, monkeypatch):
    f = Fake()
    f.real_empty = torch.empty
    monkeypatch.setattr(sv, "_lib", f)
    monkeypatch.setattr(sv, "_default_ws", {})
    monkeypatch.setattr(torch, "empty", f.empty)
    monkeypatch.setattr(torch.cuda, "device", f.device)
    monkeypatch.setattr(torch.cuda, "stream", f.stream)
    monkeypatch.setattr(torch.cuda, "current_stream", f.current_stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: f.current)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: getattr(f, "capturing", False))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: f.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: f.streams[d].cuda_stream,
                        raising=False)
    sv._attention_bytes.cache_clear()
    return f


def calls(sv, index):
    """Every entry point with inputs on GPU `index`: name -> function of (the
    keywords stream and workspace)."""
    def t(*shape, dtype=torch.float32):
        return on(index, torch.zeros(shape, dtype=dtype))

    i32, bf = torch.int32, torch.bfloat16
    R, M, V, D = 2, 3, 7, 64
    n, ctx, table = t(R, dtype=i32), t(R, dtype=i32), t(R, 1, dtype=i32)
    page = t(2, 1, 16, D, dtype=bf)
    x = t(R, M, 1, D, dtype=bf)
    L = t(R, M, V)
    u = t(R, M)
    draft = (t(R, M - 1, V), t(R, M - 1, dtype=i32), n, t(R), t(R, M - 1), u)
    rank, hid = 4, 5
    W = t(V, rank, dtype=bf), t(rank, V, dtype=bf)
    return {
        "spec_verify_batch": lambda **k: sv.spec_verify_batch(L, *draft, **k),
        "spec_tv_accept_rate": lambda **k: sv.spec_tv_accept_rate(L[0], L[1], t(M), **k),
        "spec_schedule_verify_len": lambda **k: sv.spec_schedule_verify_len(u, t(9), **k),
        "spec_sts_calibrate": lambda **k: sv.spec_sts_calibrate(
            u, n, t(4, dtype=torch.float64), want_curve=True, **k),
        "spec_tree_verify": lambda **k: sv.spec_tree_verify(
            L, t(R, M, dtype=i32), t(R, M, dtype=i32), n, 2, **k),
        "spec_rnn_draft_sample": lambda **k: sv.spec_rnn_draft_sample(
            L, *W, t(R, M, hid), t(2 * rank + hid, 2 * rank, dtype=bf), t(2 * rank), n, t(R), u,
            want_state=True, **k),
        "spec_markov_draft_sample": lambda **k: sv.spec_markov_draft_sample(L, *W, n, t(R), u, **k),
        "spec_tree_mask": lambda **k: sv.spec_tree_mask(t(R, M, dtype=i32), n, ctx, **k),
        "spec_qkv_write": lambda **k: sv.spec_qkv_write(x, x, page, page, table, ctx, n, q=x, **k),
        "spec_kv_read": lambda **k: sv.spec_kv_read(page, page, table, ctx, n, 3, **k),
        "spec_kv_commit": lambda **k: sv.spec_kv_commit(
            page, page, table, ctx, n, t(R, M, dtype=i32), **k),
        "spec_tree_attention": lambda **k: sv.spec_tree_attention(
            x, page, page, table, ctx, n, want_lse=True, **k),
    }


NAMES = ("spec_verify_batch", "spec_tv_accept_rate", "spec_schedule_verify_len", "spec_sts_calibrate",
         "spec_tree_verify", "spec_rnn_draft_sample", "spec_markov_draft_sample", "spec_tree_mask",
         "spec_qkv_write", "spec_kv_read", "spec_kv_commit", "spec_tree_attention")


def handle(p):
    """The address a pointer argument holds."""
    return p.value if isinstance(p, ctypes.c_void_p) else p
