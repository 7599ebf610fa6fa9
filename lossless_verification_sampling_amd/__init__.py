"""Python binding of libspecverify (batched lossless speculative-sampling
verification and the Markov-head draft on MI355X).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in include/specverify.h.  The functions keep
the C names.  Tensors must be contiguous CUDA (HIP) tensors on one device;
logits are torch.float32 or torch.bfloat16.  Work is enqueued on the current
torch stream of that device, or on `stream` (one of that device), and nothing
synchronises except spec_get_device_status.  Outputs that are not given are
memory of the stream that the call runs on, as torch's own would be under
torch.cuda.stream(stream), and are not given away before the current stream is
done with them.

The library must have been built (``python -m
lossless_verification_sampling_amd._build`` or ``__graft_entry__.build()``);
importing this module without it raises, there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libspecverify.so")

SPEC_F32, SPEC_BF16, SPEC_E4M3 = 0, 1, 2
SPEC_OK = 0
SPEC_ETOOLARGE = -6
SPEC_NOALLOC_SCRATCH_BYTES = 32 << 20
SPEC_DEV_BAD_REQUEST = 0x1
SPEC_DEV_SPIN_TIMEOUT = 0x2
SPEC_MAX_VOCAB = 2097152
SPEC_MAX_VERIFY_VOCAB = 262144
SPEC_SCHED_MAX_POOL = 8192
SPEC_RNN_MAX_HIDDEN = 3072
SPEC_STS_MAX_BINS = 24
SPEC_STS_MAX_GRID = 1024
SPEC_STS_MAX_BLOCKS = 1 << 24
SPEC_TREE_MAX_NODES = 1024
SPEC_PATH_SPLIT, SPEC_PATH_HELD = 0, 1

EXPORTED = (
    "spec_version",
    "spec_status_string",
    "spec_verify_workspace_bytes",
    "spec_verify_path",
    "spec_workspace_init",
    "spec_verify_batch",
    "spec_verify_batch_noalloc",
    "spec_tv_workspace_bytes",
    "spec_tv_accept_rate",
    "spec_markov_workspace_bytes",
    "spec_rnn_workspace_bytes",
    "spec_rnn_draft_sample",
    "spec_schedule_workspace_bytes",
    "spec_schedule_verify_len",
    "spec_sts_workspace_bytes",
    "spec_sts_calibrate",
    "spec_tree_workspace_bytes",
    "spec_tree_verify",
    "spec_markov_draft_sample",
    "spec_cache_workspace_bytes",
    "spec_tree_mask",
    "spec_qkv_write",
    "spec_kv_read",
    "spec_kv_commit",
    "spec_tree_attention_workspace_bytes",
    "spec_tree_attention",
    "spec_page_bounds",
    "spec_page_select_workspace_bytes",
    "spec_page_select",
    "spec_page_attention",
    "spec_sample_workspace_bytes",
    "spec_sample",
    "spec_truncate_logits",
    "spec_get_device_status",
    "spec_time_stats_launch",
)


class SpecError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {spec_status_string(status)} ({status})")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build the HIP library first "
                          "(python -m lossless_verification_sampling_amd._build)")
    lib = ctypes.CDLL(LIB_PATH)
    p, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.spec_version.restype = i
    lib.spec_version.argtypes = []
    lib.spec_status_string.restype = ctypes.c_char_p
    lib.spec_status_string.argtypes = [i]
    lib.spec_verify_workspace_bytes.restype = sz
    lib.spec_verify_workspace_bytes.argtypes = [i, i, i]
    lib.spec_verify_path.restype = i
    lib.spec_verify_path.argtypes = [i, i, i, i, i]
    lib.spec_tv_workspace_bytes.restype = sz
    lib.spec_tv_workspace_bytes.argtypes = [i, i]
    lib.spec_markov_workspace_bytes.restype = sz
    lib.spec_markov_workspace_bytes.argtypes = [i, i, i, i]
    lib.spec_workspace_init.restype = i
    lib.spec_workspace_init.argtypes = [p, sz, p]
    lib.spec_verify_batch.restype = i
    lib.spec_verify_batch.argtypes = [p, i, p, i, p, p, p, p, p, i, i, i, p, p, p, p, p, p, sz, p]
    lib.spec_time_stats_launch.restype = i
    lib.spec_time_stats_launch.argtypes = [p, p, i]
    lib.spec_verify_batch_noalloc.restype = i
    lib.spec_verify_batch_noalloc.argtypes = [p, i, p, i, p, p, p, p, p, i, i, i, p, p, p, p, p,
                                              p]
    lib.spec_tv_accept_rate.restype = i
    lib.spec_tv_accept_rate.argtypes = [p, p, i, p, i, i, p, p, p, sz, p]
    lib.spec_markov_draft_sample.restype = i
    lib.spec_markov_draft_sample.argtypes = [p, i, p, p, i, p, p, p, i, i, i, i, p, p, p, sz, p]
    lib.spec_rnn_workspace_bytes.restype = sz
    lib.spec_rnn_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.spec_rnn_draft_sample.restype = i
    lib.spec_rnn_draft_sample.argtypes = [p, i, p, p, i, p, i, p, p, p, p, p, i, i, i, i, p, p, p,
                                          p, sz, p]
    lib.spec_schedule_workspace_bytes.restype = sz
    lib.spec_schedule_workspace_bytes.argtypes = []
    lib.spec_schedule_verify_len.restype = i
    lib.spec_schedule_verify_len.argtypes = [p, p, i, i, i, i, p, p, p, sz, p]
    lib.spec_sts_workspace_bytes.restype = sz
    lib.spec_sts_workspace_bytes.argtypes = [i, i, i, i]
    lib.spec_sts_calibrate.restype = i
    lib.spec_sts_calibrate.argtypes = [p, p, p, i, i, i, i, p, p, p, p, sz, p]
    lib.spec_tree_workspace_bytes.restype = sz
    lib.spec_tree_workspace_bytes.argtypes = [i, i, i]
    lib.spec_tree_verify.restype = i
    lib.spec_tree_verify.argtypes = [p, i, p, p, p, i, i, i, i, p, p, p, p, sz, p]
    f, l = ctypes.c_float, ctypes.c_int64
    lib.spec_cache_workspace_bytes.restype = sz
    lib.spec_cache_workspace_bytes.argtypes = []
    lib.spec_tree_mask.restype = i
    lib.spec_tree_mask.argtypes = [p, p, p, i, i, i, p, p, p, sz, p]
    lib.spec_qkv_write.restype = i
    lib.spec_qkv_write.argtypes = [p, p, p, i, l, l, l, p, p, f, p, i, i, i, p, p, p, p, i, i, i,
                                   i, i, i, p, p, i, p, p, i, i, p, p, sz, p]
    lib.spec_kv_read.restype = i
    lib.spec_kv_read.argtypes = [p, p, i, p, p, i, i, p, i, p, p, i, i, i, i, p, p, i, p, sz, p]
    lib.spec_kv_commit.restype = i
    lib.spec_kv_commit.argtypes = [p, p, i, p, p, i, i, p, i, p, p, p, i, i, i, i, p, p, sz, p]
    lib.spec_tree_attention_workspace_bytes.restype = sz
    lib.spec_tree_attention_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.spec_tree_attention.restype = i
    lib.spec_tree_attention.argtypes = [p, i, p, p, i, p, p, i, i, p, i, p, p, p, p, f, i, i, i, i,
                                        i, i, p, p, p, sz, p]
    lib.spec_page_bounds.restype = i
    lib.spec_page_bounds.argtypes = [p, i, p, i, i, p, i, p, p, i, i, i, i, p, p, p, sz, p]
    lib.spec_page_select_workspace_bytes.restype = sz
    lib.spec_page_select_workspace_bytes.argtypes = [i, i, i, i]
    lib.spec_page_select.restype = i
    lib.spec_page_select.argtypes = [p, i, p, p, i, i, p, i, p, p, i, i, i, i, i, i, i, i, p, i, p,
                                     p, sz, p]
    lib.spec_page_attention.restype = i
    lib.spec_page_attention.argtypes = [p, i, p, p, i, p, p, i, i, p, i, p, p, p, f, i, i, i, i, i,
                                        p, p, p, sz, p]
    lib.spec_sample_workspace_bytes.restype = sz
    lib.spec_sample_workspace_bytes.argtypes = [i, i, i]
    lib.spec_sample.restype = i
    lib.spec_sample.argtypes = [p, i, l, p, p, p, p, p, p, i, i, i, p, p, p, p, sz, p]
    lib.spec_truncate_logits.restype = i
    lib.spec_truncate_logits.argtypes = [p, i, l, p, p, p, p, p, i, i, i, p, l, p, p, sz, p]
    lib.spec_get_device_status.restype = i
    lib.spec_get_device_status.argtypes = [p, ctypes.POINTER(ctypes.c_uint32), i, p]
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    return _lib


def spec_version() -> int:
    return int(_lib.spec_version())


def spec_status_string(status: int) -> str:
    return _lib.spec_status_string(int(status)).decode()


def spec_verify_workspace_bytes(R: int, gamma: int, V: int) -> int:
    return int(_lib.spec_verify_workspace_bytes(R, gamma, V))


def spec_verify_path(R: int, gamma: int, V: int, target_dtype, draft_dtype) -> int:
    """SPEC_PATH_HELD or SPEC_PATH_SPLIT: the launch sequence a
    spec_verify_batch call of this shape takes on the current device (16-byte
    aligned rows); dtypes as torch dtypes or SPEC_F32 / SPEC_BF16."""
    def code(d):
        if isinstance(d, torch.dtype):
            return SPEC_BF16 if d == torch.bfloat16 else SPEC_F32
        return int(d)
    st = int(_lib.spec_verify_path(R, gamma, V, code(target_dtype), code(draft_dtype)))
    if st < 0:
        _raise(st, "spec_verify_path")
    return st


def spec_tv_workspace_bytes(N: int, V: int) -> int:
    return int(_lib.spec_tv_workspace_bytes(N, V))


def spec_markov_workspace_bytes(R: int, gamma: int, V: int, rank: int) -> int:
    return int(_lib.spec_markov_workspace_bytes(R, gamma, V, rank))


def spec_rnn_workspace_bytes(R: int, gamma: int, V: int, rank: int, hidden: int) -> int:
    return int(_lib.spec_rnn_workspace_bytes(R, gamma, V, rank, hidden))


def spec_schedule_workspace_bytes() -> int:
    return int(_lib.spec_schedule_workspace_bytes())


def spec_sts_workspace_bytes(N: int, gamma: int, G: int, bins: int) -> int:
    return int(_lib.spec_sts_workspace_bytes(N, gamma, G, bins))


def spec_tree_workspace_bytes(R: int, M: int, V: int) -> int:
    return int(_lib.spec_tree_workspace_bytes(R, M, V))


def spec_cache_workspace_bytes() -> int:
    return int(_lib.spec_cache_workspace_bytes())


def spec_tree_attention_workspace_bytes(R: int, M: int, Hq: int, Hkv: int, D: int) -> int:
    return int(_lib.spec_tree_attention_workspace_bytes(R, M, Hq, Hkv, D))


def spec_page_select_workspace_bytes(R: int, Hkv: int, D: int, max_pages: int) -> int:
    return int(_lib.spec_page_select_workspace_bytes(R, Hkv, D, max_pages))


def spec_sample_workspace_bytes(R: int, J: int, V: int) -> int:
    return int(_lib.spec_sample_workspace_bytes(R, J, V))


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _stream_of(stream: Optional[torch.cuda.Stream], dev: int) -> int:
    """Handle of the stream that a call for device `dev` runs on."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, expected cuda:{dev}")
    return stream.cuda_stream


def _c_int(value, name: str) -> int:
    """`value` as a C int (ctypes keeps the low 32 bits of any integer)."""
    value = int(value)
    if not -1 << 31 <= value < 1 << 31:
        raise ValueError(f"{name} is not a 32-bit number: {value}")
    return value


def _run(dev: int, call, *args) -> int:
    """call(*args) with device `dev` current: stream 0 is the current device's."""
    if torch._C._cuda_getDevice() == dev:
        return call(*args)
    with torch.cuda.device(dev):
        return call(*args)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SPEC_F32
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _check(t: Optional[torch.Tensor], name: str, dtype=None, shape=None, device=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _raise(status: int, what: str):
    if status != SPEC_OK:
        raise SpecError(status, what)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """torch.empty from the memory of the stream the call runs on: what the
    current stream frees may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if here.cuda_stream != stream.cuda_stream:
        t.record_stream(here)
    return t


def _capturing(stream) -> bool:
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _init(buf: torch.Tensor, stream):
    dev = buf.get_device()
    _raise(_run(dev, _lib.spec_workspace_init, _ptr(buf), buf.numel(), _stream_of(stream, dev)),
           "spec_workspace_init")


class Workspace:
    """A device buffer for the library's cross-workgroup exchange, initialised
    once with spec_workspace_init and grown on demand, to twice its size at
    least.  The buffers it outgrew, together smaller than the present one, are
    kept for as long as it is: captured graphs go on writing to them.  Calls that
    share a workspace must be stream-ordered.  Give it its size before a capture:
    a buffer taken inside one is cleared by every replay, its status word too."""

    def __init__(self, device=None, nbytes: int = 0):
        self.device = torch.device(device if device is not None else "cuda")
        self.buf: Optional[torch.Tensor] = None
        self._outgrown = []
        self._recorded = False  # buf was taken inside a capture: cleared by the replays alone
        self._streams = set()  # handles of the streams that buf is known to be used on
        if nbytes:
            self.ensure(nbytes)

    def ensure(self, nbytes: int, stream=None) -> torch.Tensor:
        small = self.buf is None or self.buf.numel() < nbytes
        inside = (small or self._recorded) and _capturing(stream)
        if small or self._recorded and not inside:
            n = max(int(nbytes), 1 << 16, 2 * self.nbytes)
            n = (n + 255) // 256 * 256
            buf = _empty((n,), torch.uint8, self.device, stream)
            _init(buf, stream)
            if self.buf is not None:
                self._outgrown.append(self.buf)
            self.buf = buf
            self._recorded = inside
            self._streams = {_stream_of(stream, buf.get_device())}
        handle = _stream_of(stream, self.buf.get_device())
        if handle not in self._streams:  # its memory stays until that stream is done, too
            self.buf.record_stream(stream if stream is not None else
                                   torch.cuda.current_stream(self.buf.device))
            self._streams.add(handle)
        return self.buf

    @property
    def nbytes(self) -> int:
        return 0 if self.buf is None else self.buf.numel()


_default_ws = {}


def default_workspace(device) -> Workspace:
    """The device's workspace for calls that give none.  There is one: calls on
    several streams at a time need workspaces of their own."""
    device = torch.device(device)
    key = (device.type, device.index if device.index is not None else torch.cuda.current_device())
    ws = _default_ws.get(key)
    if ws is None:
        ws = Workspace(torch.device("cuda", key[1]))
        _default_ws[key] = ws
    return ws


def spec_workspace_init(workspace: Workspace, stream=None) -> None:
    if workspace.buf is not None:
        _init(workspace.buf, stream)


def spec_get_device_status(workspace: Workspace, clear: bool = True, stream=None) -> int:
    """Synchronises the stream and returns the OR of SPEC_DEV_* bits, those in
    the buffers that the workspace outgrew (a replayed graph's, or from before
    it grew) among them."""
    found = 0
    for buf in workspace._outgrown + [workspace.buf]:
        if buf is not None:
            bits, dev = ctypes.c_uint32(0), buf.get_device()
            _raise(_run(dev, _lib.spec_get_device_status, _ptr(buf), ctypes.byref(bits),
                        int(clear), _stream_of(stream, dev)), "spec_get_device_status")
            # (unknown bits: taken inside a capture and not replayed yet, the word
            # is what its memory held before)
            if not bits.value & ~(SPEC_DEV_BAD_REQUEST | SPEC_DEV_SPIN_TIMEOUT):
                found |= bits.value
    return found


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def _verify_io(target_logits, draft_logits, draft_tokens, verify_len, temperature, u_accept,
               u_sample, out, want_cstar, want_resid, want_logq, stream):
    """Checks the inputs of a verification call and returns (R, gamma, V, outputs)
    with the missing output tensors allocated."""
    R, G1, V = target_logits.shape
    gamma = G1 - 1
    dev = target_logits.device
    _check(target_logits, "target_logits", device=dev)
    _check(draft_logits, "draft_logits", shape=(R, gamma, V), device=dev)
    _check(draft_tokens, "draft_tokens", torch.int32, (R, gamma), dev)
    _check(verify_len, "verify_len", torch.int32, (R,), dev)
    _check(temperature, "temperature", torch.float32, (R,), dev)
    _check(u_accept, "u_accept", torch.float32, (R, gamma), dev)
    _check(u_sample, "u_sample", torch.float32, (R, G1), dev)
    if out is None:
        out = {}
    o_tok = out.get("tokens")
    if o_tok is None:
        o_tok = _empty((R, G1), torch.int32, dev, stream)
    o_n = out.get("num_accepted")
    if o_n is None:
        o_n = _empty((R,), torch.int32, dev, stream)
    o_cs = out.get("cstar")
    if o_cs is None and want_cstar:
        o_cs = _empty((R, gamma), torch.float32, dev, stream)
    o_rs = out.get("resid_mass")
    if o_rs is None and want_resid:
        o_rs = _empty((R, gamma), torch.float32, dev, stream)
    o_lq = out.get("logq")
    if o_lq is None and want_logq:
        o_lq = _empty((R, G1), torch.float32, dev, stream)
    _check(o_tok, "out tokens", torch.int32, (R, G1), dev)
    _check(o_n, "out num_accepted", torch.int32, (R,), dev)
    _check(o_cs, "out cstar", torch.float32, (R, gamma), dev)
    _check(o_rs, "out resid_mass", torch.float32, (R, gamma), dev)
    _check(o_lq, "out logq", torch.float32, (R, G1), dev)
    return R, gamma, V, dict(tokens=o_tok, num_accepted=o_n, cstar=o_cs, resid_mass=o_rs,
                             logq=o_lq)


def spec_verify_batch(target_logits: torch.Tensor, draft_logits: Optional[torch.Tensor],
                      draft_tokens: Optional[torch.Tensor], verify_len: torch.Tensor,
                      temperature: torch.Tensor, u_accept: Optional[torch.Tensor],
                      u_sample: torch.Tensor, *, out: Optional[dict] = None,
                      want_cstar: bool = True, want_resid: bool = True, want_logq: bool = True,
                      workspace: Optional[Workspace] = None, stream=None) -> dict:
    """Batched verification.  target_logits [R, gamma+1, V], draft_logits
    [R, gamma, V] (float32 / bfloat16), draft_tokens [R, gamma] int32,
    verify_len [R] int32, temperature [R] float32, u_accept [R, gamma] and
    u_sample [R, gamma+1] float32.  Returns dict(tokens, num_accepted, cstar,
    resid_mass, logq); `out` may supply preallocated output tensors."""
    R, gamma, V, o = _verify_io(target_logits, draft_logits, draft_tokens, verify_len,
                                temperature, u_accept, u_sample, out, want_cstar, want_resid,
                                want_logq, stream)
    dev = target_logits.device
    ws = workspace or default_workspace(dev)
    need = spec_verify_workspace_bytes(R, gamma, V)
    if need == 0:
        raise SpecError(-5, "spec_verify_workspace_bytes")
    buf = ws.ensure(need, stream)
    d_dtype = _dtype(draft_logits) if draft_logits is not None else SPEC_F32
    st = _run(dev.index, _lib.spec_verify_batch, _ptr(target_logits), _dtype(target_logits),
              _ptr(draft_logits), d_dtype, _ptr(draft_tokens), _ptr(verify_len), _ptr(temperature),
              _ptr(u_accept), _ptr(u_sample), R, gamma, V, _ptr(o["tokens"]),
              _ptr(o["num_accepted"]), _ptr(o["cstar"]), _ptr(o["resid_mass"]), _ptr(o["logq"]),
              _ptr(buf), buf.numel(), _stream_of(stream, dev.index))
    _raise(st, "spec_verify_batch")
    return o


def spec_verify_batch_noalloc(target_logits: torch.Tensor, draft_logits: Optional[torch.Tensor],
                              draft_tokens: Optional[torch.Tensor], verify_len: torch.Tensor,
                              temperature: torch.Tensor, u_accept: Optional[torch.Tensor],
                              u_sample: torch.Tensor, *, out: dict, stream=None) -> dict:
    """spec_verify_batch on the library's fixed per-device scratch instead of
    a workspace (no allocation in the library).  `out` must hold every output
    tensor the call writes (tokens, num_accepted; cstar, resid_mass, logq or
    None), so that the call allocates nothing here either."""
    for k in ("tokens", "num_accepted", "cstar", "resid_mass", "logq"):
        if k not in out:
            raise ValueError(f"spec_verify_batch_noalloc: out[{k!r}] must be given "
                             "(a tensor, or None for an optional output)")
    R, gamma, V, o = _verify_io(target_logits, draft_logits, draft_tokens, verify_len,
                                temperature, u_accept, u_sample, out, False, False, False,
                                stream)
    dev = target_logits.device
    d_dtype = _dtype(draft_logits) if draft_logits is not None else SPEC_F32
    st = _run(dev.index, _lib.spec_verify_batch_noalloc, _ptr(target_logits), _dtype(target_logits),
              _ptr(draft_logits), d_dtype, _ptr(draft_tokens), _ptr(verify_len), _ptr(temperature),
              _ptr(u_accept), _ptr(u_sample), R, gamma, V, _ptr(o["tokens"]),
              _ptr(o["num_accepted"]), _ptr(o["cstar"]), _ptr(o["resid_mass"]), _ptr(o["logq"]),
              _stream_of(stream, dev.index))
    _raise(st, "spec_verify_batch_noalloc")
    return o


def spec_time_stats_launch(before, after) -> None:
    """Times the statistics launch of the calling thread's next len(before)
    verification calls: `before` and `after` are sequences of hipEvent_t
    handles (ints) that the library records around that launch.  The arrays
    are kept alive here until the next call of this function."""
    global _timing_arrays
    n = len(before)
    if len(after) != n:
        raise ValueError("spec_time_stats_launch: before and after differ in length")
    arr_t = ctypes.c_void_p * max(n, 1)
    _timing_arrays = (arr_t(*before), arr_t(*after))
    _raise(_lib.spec_time_stats_launch(_timing_arrays[0], _timing_arrays[1], n),
           "spec_time_stats_launch")


_timing_arrays = None


def spec_tv_accept_rate(draft_logits: torch.Tensor, target_logits: torch.Tensor,
                        temperature: torch.Tensor, *, want_resid: bool = True,
                        workspace: Optional[Workspace] = None, stream=None):
    """c* and Res of N row pairs [N, V]; returns (cstar [N], resid_mass [N] or None)."""
    N, V = target_logits.shape
    dev = target_logits.device
    _check(target_logits, "target_logits", device=dev)
    _check(draft_logits, "draft_logits", target_logits.dtype, (N, V), dev)
    _check(temperature, "temperature", torch.float32, (N,), dev)
    cs = _empty((N,), torch.float32, dev, stream)
    rs = _empty((N,), torch.float32, dev, stream) if want_resid else None
    ws = workspace or default_workspace(dev)
    need = spec_tv_workspace_bytes(N, V)
    if need == 0:
        raise SpecError(-5, "spec_tv_workspace_bytes")
    buf = ws.ensure(need, stream)
    st = _run(dev.index, _lib.spec_tv_accept_rate, _ptr(draft_logits), _ptr(target_logits),
              _dtype(target_logits), _ptr(temperature), N, V, _ptr(cs), _ptr(rs), _ptr(buf),
              buf.numel(), _stream_of(stream, dev.index))
    _raise(st, "spec_tv_accept_rate")
    return cs, rs


def spec_schedule_verify_len(confidence: torch.Tensor, sps: torch.Tensor, *, topk: int = -1,
                             out_len: Optional[torch.Tensor] = None,
                             out_theta: Optional[torch.Tensor] = None,
                             workspace: Optional[Workspace] = None, stream=None):
    """Confidence-scheduled verify lengths.  confidence [R, gamma] float32 in
    [0, 1], sps [bmax + 1] float32 (steps per second at batch size B).  topk < 0:
    greedy admission with early stop; topk >= 0: the top-K variant.  Returns
    (lengths [R] int32, theta [1] float64)."""
    R, gamma = confidence.shape
    dev = confidence.device
    _check(confidence, "confidence", torch.float32, (R, gamma), dev)
    _check(sps, "sps", torch.float32, None, dev)
    if sps.dim() != 1 or sps.numel() < 1:
        raise ValueError("sps must be a non-empty 1-D table")
    ln = out_len if out_len is not None else _empty((R,), torch.int32, dev, stream)
    th = out_theta if out_theta is not None else _empty((1,), torch.float64, dev, stream)
    _check(ln, "out_len", torch.int32, (R,), dev)
    _check(th, "out_theta", torch.float64, (1,), dev)
    ws = workspace or default_workspace(dev)
    buf = ws.ensure(spec_schedule_workspace_bytes(), stream)
    st = _run(dev.index, _lib.spec_schedule_verify_len, _ptr(confidence), _ptr(sps), R, gamma,
              sps.numel() - 1, _c_int(topk, "topk"), _ptr(ln), _ptr(th), _ptr(buf), buf.numel(),
              _stream_of(stream, dev.index))
    _raise(st, "spec_schedule_verify_len")
    return ln, th


def spec_sts_calibrate(conf_logits: torch.Tensor, accepted_len: torch.Tensor, grid: torch.Tensor,
                       *, bins: int = 15, want_curve: bool = False,
                       workspace: Optional[Workspace] = None, stream=None):
    """Sequential temperature scaling of the confidence head on a held-out
    set.  conf_logits [N, gamma] float32 raw logits, accepted_len [N] int32
    (accepted prefix length per block), grid [G] float64 candidate
    temperatures.  Returns (temperatures [gamma] float64, ece [gamma] float64,
    curves [gamma, G] float64 or None)."""
    N, gamma = conf_logits.shape
    G = grid.numel()
    dev = conf_logits.device
    _check(conf_logits, "conf_logits", torch.float32, (N, gamma), dev)
    _check(accepted_len, "accepted_len", torch.int32, (N,), dev)
    _check(grid, "grid", torch.float64, (G,), dev)
    temps = _empty((gamma,), torch.float64, dev, stream)
    ece = _empty((gamma,), torch.float64, dev, stream)
    curve = _empty((gamma, G), torch.float64, dev, stream) if want_curve else None
    need = spec_sts_workspace_bytes(max(N, 1), gamma, G, bins)
    if need == 0:
        raise ValueError(f"spec_sts_calibrate: unsupported sizes N={N} G={G} bins={bins}")
    ws = workspace or default_workspace(dev)
    buf = ws.ensure(need, stream)
    st = _run(dev.index, _lib.spec_sts_calibrate, _ptr(conf_logits), _ptr(accepted_len), _ptr(grid),
              N, gamma, G, _c_int(bins, "bins"), _ptr(temps), _ptr(ece),
              _ptr(curve) if curve is not None else None, _ptr(buf), buf.numel(),
              _stream_of(stream, dev.index))
    _raise(st, "spec_sts_calibrate")
    return temps, ece, curve


def spec_tree_verify(logits: torch.Tensor, parent: torch.Tensor, tokens: torch.Tensor,
                     n_nodes: torch.Tensor, max_depth: int, *,
                     workspace: Optional[Workspace] = None, stream=None):
    """Greedy (T = 0) tree verification.  logits [R, M, V] float32 or
    bfloat16 (row v: the target's next-token logits after the path to node v),
    parent / tokens [R, M] int32, n_nodes [R] int32, max_depth a bound on every
    tree's depth (deeper trees are rejected).  Returns (accepted [R], path [R, M], committed tokens [R, M])
    as int32."""
    R, M, V = logits.shape
    dev = logits.device
    _check(logits, "logits", logits.dtype, (R, M, V), dev)
    for t, nm in ((parent, "parent"), (tokens, "tokens")):
        _check(t, nm, torch.int32, (R, M), dev)
    _check(n_nodes, "n_nodes", torch.int32, (R,), dev)
    acc = _empty((R,), torch.int32, dev, stream)
    path = _empty((R, M), torch.int32, dev, stream)
    tok = _empty((R, M), torch.int32, dev, stream)
    need = spec_tree_workspace_bytes(max(R, 1), M, V)
    if need == 0:
        raise ValueError(f"spec_tree_verify: unsupported sizes M={M} V={V}")
    ws = workspace or default_workspace(dev)
    buf = ws.ensure(need, stream)
    st = _run(dev.index, _lib.spec_tree_verify, _ptr(logits), _dtype(logits), _ptr(parent),
              _ptr(tokens), _ptr(n_nodes), R, M, V, _c_int(max_depth, "max_depth"), _ptr(acc),
              _ptr(path), _ptr(tok), _ptr(buf), buf.numel(), _stream_of(stream, dev.index))
    _raise(st, "spec_tree_verify")
    return acc, path, tok


def spec_rnn_draft_sample(U: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor,
                          hidden_states: torch.Tensor, Wg: torch.Tensor, bg: torch.Tensor,
                          anchor: torch.Tensor, temperature: torch.Tensor, u_draft: torch.Tensor,
                          *, want_state: bool = False, out_tokens: Optional[torch.Tensor] = None,
                          out_logits: Optional[torch.Tensor] = None,
                          workspace: Optional[Workspace] = None, stream=None):
    """RNN-head draft.  As spec_markov_draft_sample plus hidden_states
    [R, gamma, hidden] float32, Wg [2 rank + hidden, 2 rank] bfloat16, bg
    [2 rank] float32.  Returns (tokens, logits, states [R, gamma, rank] float32
    or None)."""
    R, gamma, V = U.shape
    rank = W1.shape[1]
    hidden = hidden_states.shape[2]
    dev = U.device
    _check(U, "U", device=dev)
    _check(W1, "W1", torch.bfloat16, (V, rank), dev)
    _check(W2, "W2", torch.bfloat16, (rank, V), dev)
    _check(hidden_states, "hidden_states", torch.float32, (R, gamma, hidden), dev)
    _check(Wg, "Wg", torch.bfloat16, (2 * rank + hidden, 2 * rank), dev)
    _check(bg, "bg", torch.float32, (2 * rank,), dev)
    _check(anchor, "anchor", torch.int32, (R,), dev)
    _check(temperature, "temperature", torch.float32, (R,), dev)
    _check(u_draft, "u_draft", torch.float32, (R, gamma), dev)
    tok = out_tokens if out_tokens is not None else _empty((R, gamma), torch.int32, dev, stream)
    lg = out_logits if out_logits is not None else _empty((R, gamma, V), torch.float32, dev, stream)
    stt = _empty((R, gamma, rank), torch.float32, dev, stream) if want_state else None
    _check(tok, "out_tokens", torch.int32, (R, gamma), dev)
    _check(lg, "out_logits", torch.float32, (R, gamma, V), dev)
    ws = workspace or default_workspace(dev)
    need = spec_rnn_workspace_bytes(R, gamma, V, rank, hidden)
    if need == 0:
        raise SpecError(-5, "spec_rnn_workspace_bytes")
    buf = ws.ensure(need, stream)
    st = _run(dev.index, _lib.spec_rnn_draft_sample, _ptr(U), _dtype(U), _ptr(W1), _ptr(W2),
              SPEC_BF16, _ptr(hidden_states), hidden, _ptr(Wg), _ptr(bg), _ptr(anchor),
              _ptr(temperature), _ptr(u_draft), R, gamma, V, rank, _ptr(tok), _ptr(lg), _ptr(stt),
              _ptr(buf), buf.numel(), _stream_of(stream, dev.index))
    _raise(st, "spec_rnn_draft_sample")
    return tok, lg, stt


def spec_markov_draft_sample(U: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor,
                             anchor: torch.Tensor, temperature: torch.Tensor,
                             u_draft: torch.Tensor, *, out_tokens: Optional[torch.Tensor] = None,
                             out_logits: Optional[torch.Tensor] = None,
                             workspace: Optional[Workspace] = None, stream=None):
    """Markov-head draft.  U [R, gamma, V] (float32 / bfloat16), W1 [V, rank],
    W2 [rank, V] bfloat16, anchor [R] int32, temperature [R], u_draft
    [R, gamma] float32.  Returns (tokens [R, gamma] int32, logits [R, gamma, V]
    float32)."""
    R, gamma, V = U.shape
    rank = W1.shape[1]
    dev = U.device
    _check(U, "U", device=dev)
    _check(W1, "W1", torch.bfloat16, (V, rank), dev)
    _check(W2, "W2", torch.bfloat16, (rank, V), dev)
    _check(anchor, "anchor", torch.int32, (R,), dev)
    _check(temperature, "temperature", torch.float32, (R,), dev)
    _check(u_draft, "u_draft", torch.float32, (R, gamma), dev)
    tok = out_tokens if out_tokens is not None else _empty((R, gamma), torch.int32, dev, stream)
    lg = out_logits if out_logits is not None else _empty((R, gamma, V), torch.float32, dev, stream)
    _check(tok, "out_tokens", torch.int32, (R, gamma), dev)
    _check(lg, "out_logits", torch.float32, (R, gamma, V), dev)
    ws = workspace or default_workspace(dev)
    need = spec_markov_workspace_bytes(R, gamma, V, rank)
    if need == 0:
        raise SpecError(-5, "spec_markov_workspace_bytes")
    buf = ws.ensure(need, stream)
    st = _run(dev.index, _lib.spec_markov_draft_sample, _ptr(U), _dtype(U), _ptr(W1), _ptr(W2),
              SPEC_BF16, _ptr(anchor), _ptr(temperature), _ptr(u_draft), R, gamma, V, rank,
              _ptr(tok), _ptr(lg), _ptr(buf), buf.numel(), _stream_of(stream, dev.index))
    _raise(st, "spec_markov_draft_sample")
    return tok, lg


# ---------------------------------------------------------------------------
# the paged key/value cache and attention over it
# ---------------------------------------------------------------------------

def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _all(dev: int, *specs):
    """Checks (tensor, name, dtype, shape) for dense tensors on device `dev`;
    a tensor may be None.  (The quick way through; _check words the error.)"""
    for t, name, dtype, shape in specs:
        if t is not None and (t.dtype is not dtype or t.shape != shape or
                              t.get_device() != dev or not t.is_contiguous()):
            _check(t, name, dtype, shape, torch.device("cuda", dev))


_CACHE_CODES = {torch.bfloat16: SPEC_BF16, torch.float8_e4m3fn: SPEC_E4M3}


def _cache(k_cache, v_cache, k_scale, v_scale, page_table, R, dev, lists=False):
    """Checks a layer's pages on device `dev` and returns (dtype code, P, Hkv,
    page size, D, page table width).  lists: the table has a row per key head."""
    dtype = k_cache.dtype
    code = _CACHE_CODES.get(dtype)
    if code is None:
        raise TypeError(f"cache pages must be bfloat16 or float8_e4m3fn, got {dtype}")
    shape = k_cache.shape
    _need(len(shape) == 4, "k_cache must be [pages, heads, page size, D]")
    if lists:
        _need(page_table.dim() == 3, "page_lists must be [R, heads, list_pages]")
        name, rows = "page_lists", (R, shape[1])
    else:
        _need(page_table.dim() == 2, "page_table must be [R, max_pages]")
        name, rows = "page_table", (R,)
    wide = page_table.shape[-1]
    if code == SPEC_E4M3:
        _need(k_scale is not None and v_scale is not None, "e4m3 pages need k_scale and v_scale")
    else:
        _need(k_scale is None and v_scale is None, "bfloat16 pages have no scales")
    _all(dev, (k_cache, "k_cache", dtype, shape), (v_cache, "v_cache", dtype, shape),
         (k_scale, "k_scale", torch.float32, shape[:3]),
         (v_scale, "v_scale", torch.float32, shape[:3]),
         (page_table, name, torch.int32, rows + (wide,)))
    P, Hkv, size, D = shape
    return code, P, Hkv, size, D, wide


def _device(t: torch.Tensor, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a device tensor")
    return dev


def _raw(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _ordered_heads(t: torch.Tensor, name: str, shape, dev: int) -> int:
    """Elements from one token's heads to the next of [R, M, H, D] whose
    tokens are evenly spaced and whose heads are dense."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    R, M, H, D = shape
    s0, s1, s2, s3 = t.stride()
    row = H * D
    ld = s1 if M > 1 else s0 if R > 1 else row
    if ((s3 != 1 and D > 1) or (s2 != D and H > 1) or ld < row or
            (s0 != M * ld and R > 1 and M > 1)) and t.numel():
        raise ValueError(f"{name} must hold dense heads at evenly spaced tokens")
    return ld if ld > row else row


@functools.lru_cache(maxsize=256)
def _attention_bytes(*sizes) -> int:
    return _lib.spec_tree_attention_workspace_bytes(*sizes)


def _cache_buf(workspace, dev: int, need: int, stream):
    """(address, bytes, handle of the stream the call runs on)."""
    ws = workspace or _default_ws.get(("cuda", dev)) or default_workspace(torch.device("cuda", dev))
    handle = _stream_of(stream, dev)
    buf = ws.buf
    if buf is None or buf.numel() < need or handle not in ws._streams or ws._recorded:
        if ws.device.index not in (None, dev):
            raise ValueError(f"workspace is on {ws.device}, expected cuda:{dev}")
        buf = ws.ensure(need, stream)
    if buf.get_device() != dev:
        raise ValueError(f"workspace is on {buf.device}, expected cuda:{dev}")
    return buf.data_ptr(), buf.numel(), handle


def spec_tree_mask(parent: torch.Tensor, n_nodes: torch.Tensor, ctx_len: torch.Tensor, *,
                   window: int = 0, out_positions: Optional[torch.Tensor] = None,
                   out_mask: Optional[torch.Tensor] = None,
                   workspace: Optional[Workspace] = None, stream=None):
    """Positions and ancestor bits of drafted trees, once a step for all
    layers.  parent [R, M], n_nodes [R], ctx_len [R] int32.  Returns
    (positions [R, M] int32, mask [R, M, (M + 31) // 32] int32 bit words)."""
    R, M = shape = parent.shape
    dev = _device(parent, "parent")
    words = (R, M, (M + 31) // 32)
    i32 = torch.int32
    pos = out_positions if out_positions is not None else _empty(shape, i32, parent.device, stream)
    mask = out_mask if out_mask is not None else _empty(words, i32, parent.device, stream)
    _all(dev, (parent, "parent", i32, shape), (n_nodes, "n_nodes", i32, (R,)),
         (ctx_len, "ctx_len", i32, (R,)), (pos, "out_positions", i32, shape),
         (mask, "out_mask", i32, words))
    buf, size, queue = _cache_buf(workspace, dev, 256, stream)
    st = _run(dev, _lib.spec_tree_mask, parent.data_ptr(), n_nodes.data_ptr(), ctx_len.data_ptr(),
              R, M, _c_int(window, "window"), pos.data_ptr(), mask.data_ptr(), buf, size, queue)
    if st:
        _raise(st, "spec_tree_mask")
    return pos, mask


def spec_qkv_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   page_table: torch.Tensor, ctx_len: torch.Tensor, n_nodes: torch.Tensor, *,
                   q: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                   k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   rope: Optional[torch.Tensor] = None, interleaved: bool = False,
                   positions: Optional[torch.Tensor] = None,
                   k_scale: Optional[torch.Tensor] = None,
                   v_scale: Optional[torch.Tensor] = None, out_q: Optional[torch.Tensor] = None,
                   workspace: Optional[Workspace] = None, stream=None) -> Optional[torch.Tensor]:
    """Norms of queries and keys, the position rotation and the cache write in
    one pass.  k, v [R, M, Hkv, D] and q [R, M, Hq, D] float32 or bfloat16
    (parts of one projection's output: tokens evenly spaced, heads dense),
    weights [D] of that type, rope [max_pos, rot / 2, 2] float32 (cos, sin),
    positions [R, M] int32 (ctx_len + index without).  Token v < n_nodes[r] of
    request r goes to cache token ctx_len[r] + v.  Returns the queries
    [R, M, Hq, D] bfloat16 (out_q), or None without q."""
    shape = k.shape
    _need(len(shape) == 4 and v.shape == shape, "k and v must be [R, M, heads, D], both alike")
    R, M, Hkv, D = shape
    dev = _device(k, "k")
    code, P, H, size, Dc, wide = _cache(k_cache, v_cache, k_scale, v_scale, page_table, R, dev)
    _need(H == Hkv and Dc == D, "k, v and the cache differ in heads or D")
    dtype = k.dtype
    dt = _dtype(k)
    _need(v.dtype is dtype and (q is None or q.dtype is dtype), "q, k and v differ in type")
    ld_k, ld_v = _ordered_heads(k, "k", shape, dev), _ordered_heads(v, "v", shape, dev)
    Hq = ld_q = 0
    if q is not None:
        qs = q.shape
        _need(len(qs) == 4 and qs[0] == R and qs[1] == M and qs[3] == D, "q must be [R, M, Hq, D]")
        Hq, ld_q = qs[2], _ordered_heads(q, "q", qs, dev)
        if out_q is None:
            out_q = _empty(qs, torch.bfloat16, k.device, stream)
    else:
        qs = None
        _need(q_weight is None and out_q is None, "q_weight and out_q belong to q")
    max_pos = rot = 0
    rs = None
    if rope is not None:
        rs = rope.shape
        _need(len(rs) == 3 and rs[2] == 2, "rope must be [max_pos, rot / 2, 2]")
        max_pos, rot = rs[0], 2 * rs[1]
    i32 = torch.int32
    _all(dev, (out_q, "out_q", torch.bfloat16, qs), (q_weight, "q_weight", dtype, (D,)),
         (k_weight, "k_weight", dtype, (D,)), (rope, "rope", torch.float32, rs),
         (positions, "positions", i32, (R, M)), (ctx_len, "ctx_len", i32, (R,)),
         (n_nodes, "n_nodes", i32, (R,)))
    buf, room, queue = _cache_buf(workspace, dev, 256, stream)
    st = _run(dev, _lib.spec_qkv_write, _raw(q), k.data_ptr(), v.data_ptr(), dt, ld_q, ld_k, ld_v,
              _raw(q_weight), _raw(k_weight), eps, _raw(rope), max_pos, rot, int(interleaved),
              _raw(positions), ctx_len.data_ptr(), n_nodes.data_ptr(), page_table.data_ptr(), wide,
              R, M, Hq, Hkv, D, k_cache.data_ptr(), v_cache.data_ptr(), code, _raw(k_scale),
              _raw(v_scale), P, size, _raw(out_q), buf, room, queue)
    if st:
        _raise(st, "spec_qkv_write")
    return out_q


def spec_kv_read(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                 start: torch.Tensor, length: torch.Tensor, max_len: int, *,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                 dtype: torch.dtype = torch.bfloat16, out_k: Optional[torch.Tensor] = None,
                 out_v: Optional[torch.Tensor] = None, workspace: Optional[Workspace] = None,
                 stream=None):
    """Reads tokens start[r] .. start[r] + length[r] - 1 of every request.
    Returns (k, v) [R, max_len, Hkv, D] in `dtype` (bfloat16 or float32, or
    that of a given output); rows past length[r] are left as they were."""
    R, dev = page_table.shape[0], _device(k_cache, "k_cache")
    code, P, Hkv, size, D, wide = _cache(k_cache, v_cache, k_scale, v_scale, page_table, R, dev)
    max_len = _c_int(max_len, "max_len")
    _need(max_len >= 0, "max_len must not be negative")
    given = out_k if out_k is not None else out_v
    if given is not None:
        dtype = given.dtype
    shape = (R, max_len, Hkv, D)
    if out_k is None:
        out_k = _empty(shape, dtype, k_cache.device, stream)
    if out_v is None:
        out_v = _empty(shape, dtype, k_cache.device, stream)
    _all(dev, (start, "start", torch.int32, (R,)), (length, "length", torch.int32, (R,)),
         (out_k, "out_k", dtype, shape), (out_v, "out_v", dtype, shape))
    buf, room, queue = _cache_buf(workspace, dev, 256, stream)
    st = _run(dev, _lib.spec_kv_read, k_cache.data_ptr(), v_cache.data_ptr(), code, _raw(k_scale),
              _raw(v_scale), P, size, page_table.data_ptr(), wide, start.data_ptr(),
              length.data_ptr(), R, max_len, Hkv, D, out_k.data_ptr(), out_v.data_ptr(),
              _dtype(out_k), buf, room, queue)
    if st:
        _raise(st, "spec_kv_read")
    return out_k, out_v


def spec_kv_commit(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                   ctx_len: torch.Tensor, accepted: torch.Tensor, path: torch.Tensor, *,
                   k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                   out_ctx_len: Optional[torch.Tensor] = None,
                   workspace: Optional[Workspace] = None, stream=None) -> torch.Tensor:
    """Moves the accepted path's rows (spec_tree_verify's accepted [R] and path
    [R, M]) behind the context, in place.  Returns the new context lengths."""
    R, M = path.shape
    dev = _device(k_cache, "k_cache")
    code, P, Hkv, size, D, wide = _cache(k_cache, v_cache, k_scale, v_scale, page_table, R, dev)
    i32 = torch.int32
    if out_ctx_len is None:
        out_ctx_len = _empty((R,), i32, k_cache.device, stream)
    _all(dev, (ctx_len, "ctx_len", i32, (R,)), (accepted, "accepted", i32, (R,)),
         (path, "path", i32, (R, M)), (out_ctx_len, "out_ctx_len", i32, (R,)))
    buf, room, queue = _cache_buf(workspace, dev, 256, stream)
    st = _run(dev, _lib.spec_kv_commit, k_cache.data_ptr(), v_cache.data_ptr(), code, _raw(k_scale),
              _raw(v_scale), P, size, page_table.data_ptr(), wide, ctx_len.data_ptr(),
              accepted.data_ptr(), path.data_ptr(), R, M, Hkv, D, out_ctx_len.data_ptr(), buf, room,
              queue)
    if st:
        _raise(st, "spec_kv_commit")
    return out_ctx_len


def spec_tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        page_table: torch.Tensor, ctx_len: torch.Tensor, n_nodes: torch.Tensor, *,
                        mask: Optional[torch.Tensor] = None,
                        positions: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                        window: int = 0, k_scale: Optional[torch.Tensor] = None,
                        v_scale: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, want_lse: bool = False,
                        out_lse: Optional[torch.Tensor] = None,
                        workspace: Optional[Workspace] = None, stream=None):
    """Attention of the drafted tokens q [R, M, Hq, D] bfloat16 over the paged
    cache: the context and, by `mask` (spec_tree_mask), their ancestors; without
    a mask the tokens are a chain.  A mask with a window needs `positions`
    (spec_tree_mask) too.  scale defaults to D ** -0.5.  Returns
    (out [R, M, Hq, D] bfloat16, log-sum-exp [R, M, Hq] float32 or None)."""
    shape = q.shape
    _need(len(shape) == 4, "q must be [R, M, Hq, D]")
    R, M, Hq, D = shape
    dev = _device(q, "q")
    code, P, Hkv, size, Dc, wide = _cache(k_cache, v_cache, k_scale, v_scale, page_table, R, dev)
    _need(Dc == D, "q and the cache differ in D")
    if out is None:
        out = _empty(shape, torch.bfloat16, q.device, stream)
    if out_lse is None and want_lse:
        out_lse = _empty(shape[:3], torch.float32, q.device, stream)
    i32 = torch.int32
    _all(dev, (q, "q", torch.bfloat16, shape), (ctx_len, "ctx_len", i32, (R,)),
         (n_nodes, "n_nodes", i32, (R,)), (mask, "mask", i32, (R, M, (M + 31) // 32)),
         (positions, "positions", i32, (R, M)), (out, "out", torch.bfloat16, shape),
         (out_lse, "out_lse", torch.float32, shape[:3]))
    need = _attention_bytes(R, M, Hq, Hkv, D)
    if need == 0:
        raise SpecError(-5, "spec_tree_attention_workspace_bytes")
    buf, room, queue = _cache_buf(workspace, dev, need, stream)
    st = _run(dev, _lib.spec_tree_attention, q.data_ptr(), SPEC_BF16, k_cache.data_ptr(),
              v_cache.data_ptr(), code, _raw(k_scale), _raw(v_scale), P, size,
              page_table.data_ptr(), wide, ctx_len.data_ptr(), n_nodes.data_ptr(), _raw(mask),
              _raw(positions), D ** -0.5 if scale is None else scale, _c_int(window, "window"), R,
              M, Hq, Hkv, D, out.data_ptr(), _raw(out_lse), buf, room, queue)
    if st:
        _raise(st, "spec_tree_attention")
    return out, out_lse


# ---------------------------------------------------------------------------
# drafting over a budget of the cache's pages
# ---------------------------------------------------------------------------

def spec_page_bounds(k_cache: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor,
                     length: torch.Tensor, max_len: int, k_min: torch.Tensor,
                     k_max: torch.Tensor, *, k_scale: Optional[torch.Tensor] = None,
                     workspace: Optional[Workspace] = None, stream=None) -> None:
    """Least and largest key values, k_min and k_max [pages, Hkv, D] bfloat16,
    of the pages that hold tokens start[r] .. start[r] + length[r] - 1
    (length[r] <= max_len), over each page's tokens up to the last of them."""
    R, dev = page_table.shape[0], _device(k_cache, "k_cache")
    code, P, Hkv, size, D, wide = _cache(k_cache, k_cache, k_scale, k_scale, page_table, R, dev)
    bounds = (P, Hkv, D)
    _all(dev, (start, "start", torch.int32, (R,)), (length, "length", torch.int32, (R,)),
         (k_min, "k_min", torch.bfloat16, bounds), (k_max, "k_max", torch.bfloat16, bounds))
    buf, room, queue = _cache_buf(workspace, dev, 256, stream)
    st = _run(dev, _lib.spec_page_bounds, k_cache.data_ptr(), code, _raw(k_scale), P, size,
              page_table.data_ptr(), wide, start.data_ptr(), length.data_ptr(), R,
              _c_int(max_len, "max_len"), Hkv, D, k_min.data_ptr(), k_max.data_ptr(), buf, room,
              queue)
    if st:
        _raise(st, "spec_page_bounds")


def spec_page_select(q: torch.Tensor, k_min: torch.Tensor, k_max: torch.Tensor,
                     page_table: torch.Tensor, ctx_len: torch.Tensor, n_nodes: torch.Tensor,
                     budget: int, page_size: int, *, first: int = 0, last: int = 0,
                     out_lists: Optional[torch.Tensor] = None,
                     out_len: Optional[torch.Tensor] = None,
                     workspace: Optional[Workspace] = None, stream=None):
    """Page lists of a step's queries q [R, M, Hq, D] bfloat16: for every key
    head the `budget` full context pages (the first `first` and the last `last`
    among them) with the best bounds, then the pages of the context's end and
    of the nodes.  Returns (lists [R, Hkv, list_pages] int32, listed context
    tokens [R] int32) for spec_page_attention."""
    shape = q.shape
    _need(len(shape) == 4, "q must be [R, M, Hq, D]")
    R, M, Hq, D = shape
    dev = _device(q, "q")
    _need(k_min.dim() == 3 and k_min.shape[2] == D, "k_min must be [pages, heads, D] with q's D")
    bounds = k_min.shape
    P, Hkv = bounds[0], bounds[1]
    _need(page_table.dim() == 2, "page_table must be [R, max_pages]")
    wide, i32 = page_table.shape[1], torch.int32
    budget, page_size = _c_int(budget, "budget"), _c_int(page_size, "page_size")
    _need(budget >= 0 and page_size > 0, "budget must not be negative, page_size positive")
    if out_lists is None:
        out_lists = _empty((R, Hkv, min(budget, wide) + (M + page_size - 2) // page_size + 1), i32,
                           q.device, stream)
    if out_len is None:
        out_len = _empty((R,), i32, q.device, stream)
    _need(out_lists.dim() == 3, "out_lists must be [R, heads, list_pages]")
    width = out_lists.shape[2]
    _all(dev, (q, "q", torch.bfloat16, shape), (k_min, "k_min", torch.bfloat16, bounds),
         (k_max, "k_max", torch.bfloat16, bounds), (page_table, "page_table", i32, (R, wide)),
         (ctx_len, "ctx_len", i32, (R,)), (n_nodes, "n_nodes", i32, (R,)),
         (out_lists, "out_lists", i32, (R, Hkv, width)), (out_len, "out_len", i32, (R,)))
    need = spec_page_select_workspace_bytes(R, Hkv, D, wide)
    if need == 0:
        raise SpecError(-5, "spec_page_select_workspace_bytes")
    buf, room, queue = _cache_buf(workspace, dev, need, stream)
    st = _run(dev, _lib.spec_page_select, q.data_ptr(), SPEC_BF16, k_min.data_ptr(),
              k_max.data_ptr(), P, page_size, page_table.data_ptr(), wide, ctx_len.data_ptr(),
              n_nodes.data_ptr(), budget, _c_int(first, "first"), _c_int(last, "last"), R, M, Hq,
              Hkv, D, out_lists.data_ptr(), width, out_len.data_ptr(), buf, room, queue)
    if st:
        _raise(st, "spec_page_select")
    return out_lists, out_len


def spec_page_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        page_lists: torch.Tensor, list_len: torch.Tensor, n_nodes: torch.Tensor, *,
                        mask: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                        k_scale: Optional[torch.Tensor] = None,
                        v_scale: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, want_lse: bool = False,
                        out_lse: Optional[torch.Tensor] = None,
                        workspace: Optional[Workspace] = None, stream=None):
    """spec_tree_attention over page lists of each key head's own (page_lists
    [R, Hkv, list_pages], list_len [R] int32, as spec_page_select writes them):
    q [R, M, Hq, D] bfloat16 sees the list_len[r] listed context tokens and, by
    `mask` (spec_tree_mask; without one the tokens are a chain), its
    ancestors.  Returns (out [R, M, Hq, D] bfloat16, log-sum-exp [R, M, Hq]
    float32 or None)."""
    shape = q.shape
    _need(len(shape) == 4, "q must be [R, M, Hq, D]")
    R, M, Hq, D = shape
    dev = _device(q, "q")
    code, P, Hkv, size, Dc, wide = _cache(k_cache, v_cache, k_scale, v_scale, page_lists, R, dev,
                                          lists=True)
    _need(Dc == D, "q and the cache differ in D")
    if out is None:
        out = _empty(shape, torch.bfloat16, q.device, stream)
    if out_lse is None and want_lse:
        out_lse = _empty(shape[:3], torch.float32, q.device, stream)
    i32 = torch.int32
    _all(dev, (q, "q", torch.bfloat16, shape), (list_len, "list_len", i32, (R,)),
         (n_nodes, "n_nodes", i32, (R,)), (mask, "mask", i32, (R, M, (M + 31) // 32)),
         (out, "out", torch.bfloat16, shape), (out_lse, "out_lse", torch.float32, shape[:3]))
    need = _attention_bytes(R, M, Hq, Hkv, D)
    if need == 0:
        raise SpecError(-5, "spec_tree_attention_workspace_bytes")
    buf, room, queue = _cache_buf(workspace, dev, need, stream)
    st = _run(dev, _lib.spec_page_attention, q.data_ptr(), SPEC_BF16, k_cache.data_ptr(),
              v_cache.data_ptr(), code, _raw(k_scale), _raw(v_scale), P, size,
              page_lists.data_ptr(), wide, list_len.data_ptr(), n_nodes.data_ptr(), _raw(mask),
              D ** -0.5 if scale is None else scale, R, M, Hq, Hkv, D, out.data_ptr(),
              _raw(out_lse), buf, room, queue)
    if st:
        _raise(st, "spec_page_attention")
    return out, out_lse


# ---------------------------------------------------------------------------
# truncated distributions
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=256)
def _sample_bytes(*sizes) -> int:
    return _lib.spec_sample_workspace_bytes(*sizes)


def _spaced_rows(t: torch.Tensor, name: str, shape, dev: int) -> int:
    """Elements from one row to the next of [R, J, V] whose rows are evenly
    spaced and dense."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")
    R, J, V = shape
    s0, s1, s2 = t.stride()
    ld = s1 if J > 1 else s0 if R > 1 else V
    if ((s2 != 1 and V > 1) or ld < V or (s0 != J * ld and R > 1 and J > 1)) and t.numel():
        raise ValueError(f"{name} must hold dense rows, evenly spaced")
    return ld if ld > V else V


def _settings(logits, temperature, top_k, top_p, min_p, rows):
    """Checks what spec_sample and spec_truncate_logits share; returns (device,
    logits' type code and spacing)."""
    shape = logits.shape
    _need(len(shape) == 3, "logits must be [R, J, V]")
    _need(shape[2] > 0, "logits must have ids")
    dev = _device(logits, "logits")
    dt = _dtype(logits)
    per = (shape[0],)
    _need(temperature is not None, "temperature is needed")
    _all(dev, (temperature, "temperature", torch.float32, per), (top_k, "top_k", torch.int32, per),
         (top_p, "top_p", torch.float32, per), (min_p, "min_p", torch.float32, per),
         (rows, "rows", torch.int32, per))
    return dev, dt, _spaced_rows(logits, "logits", shape, dev)


def spec_sample(logits: torch.Tensor, u: torch.Tensor, *, temperature: torch.Tensor,
                top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
                min_p: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
                out: Optional[dict] = None, want_logq: bool = True, want_kept: bool = True,
                workspace: Optional[Workspace] = None, stream=None) -> dict:
    """One token of every row of logits [R, J, V] (float32 or bfloat16; rows
    dense and evenly spaced) under temperature, top-k, top-p and min-p ([R]
    each, top_k int32, the others float32) with uniforms u [R, J] float32;
    rows [R] int32 limits how many of a request's rows are in use.  Returns
    dict(tokens, logq, kept) [R, J]; `out` may supply them."""
    dev, dt, ld = _settings(logits, temperature, top_k, top_p, min_p, rows)
    R, J, V = logits.shape
    out = {} if out is None else out
    tokens, logq, kept = out.get("tokens"), out.get("logq"), out.get("kept")
    shape, i32, f32 = (R, J), torch.int32, torch.float32
    if tokens is None:
        tokens = _empty(shape, i32, logits.device, stream)
    if logq is None and want_logq:
        logq = _empty(shape, f32, logits.device, stream)
    if kept is None and want_kept:
        kept = _empty(shape, i32, logits.device, stream)
    _all(dev, (u, "u", f32, shape), (tokens, "out tokens", i32, shape),
         (logq, "out logq", f32, shape), (kept, "out kept", i32, shape))
    need = _sample_bytes(R, J, V)
    if need == 0:
        raise SpecError(-5, "spec_sample_workspace_bytes")
    buf, room, queue = _cache_buf(workspace, dev, need, stream)
    st = _run(dev, _lib.spec_sample, logits.data_ptr(), dt, ld, temperature.data_ptr(),
              _raw(top_k), _raw(top_p), _raw(min_p), _raw(rows), u.data_ptr(), R, J, V,
              tokens.data_ptr(), _raw(logq), _raw(kept), buf, room, queue)
    if st:
        _raise(st, "spec_sample")
    return {"tokens": tokens, "logq": logq, "kept": kept}


def spec_truncate_logits(logits: torch.Tensor, *, temperature: torch.Tensor,
                         top_k: Optional[torch.Tensor] = None,
                         top_p: Optional[torch.Tensor] = None,
                         min_p: Optional[torch.Tensor] = None,
                         rows: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                         out_kept: Optional[torch.Tensor] = None, want_kept: bool = True,
                         workspace: Optional[Workspace] = None, stream=None):
    """The rows of logits [R, J, V] with the ids that temperature, top-k, top-p
    and min-p leave out at -inf (arguments as spec_sample's), for
    spec_verify_batch.  `out` may be `logits` itself; rows not in use are left
    as they were.  Returns (out [R, J, V], kept ids [R, J] int32 or None)."""
    dev, dt, ld = _settings(logits, temperature, top_k, top_p, min_p, rows)
    R, J, V = shape = logits.shape
    if out is None:
        out = _empty(shape, logits.dtype, logits.device, stream)
    if out_kept is None and want_kept:
        out_kept = _empty((R, J), torch.int32, logits.device, stream)
    _need(out.dtype is logits.dtype and out.shape == shape, "out must be like logits")
    out_ld = _spaced_rows(out, "out", shape, dev)
    _all(dev, (out_kept, "out_kept", torch.int32, (R, J)))
    need = _sample_bytes(R, J, V)
    if need == 0:
        raise SpecError(-5, "spec_sample_workspace_bytes")
    buf, room, queue = _cache_buf(workspace, dev, need, stream)
    st = _run(dev, _lib.spec_truncate_logits, logits.data_ptr(), dt, ld, temperature.data_ptr(),
              _raw(top_k), _raw(top_p), _raw(min_p), _raw(rows), R, J, V, out.data_ptr(), out_ld,
              _raw(out_kept), buf, room, queue)
    if st:
        _raise(st, "spec_truncate_logits")
    return out, out_kept
