"""Python binding of libhg (include/hg.h): argument marshalling only.

Every function here has the name of the C entry point it calls and does no
computation of its own: it checks torch tensors' device, dtype, shape and
contiguity, turns them into raw device pointers, and calls the library. The
gather itself runs only in the library's CUDA kernels; if libhg.so cannot be
loaded every call raises.
"""

from __future__ import annotations

import ctypes
import os
import struct
from typing import Sequence

import torch

from . import _build

HG_OK, HG_ERR_ARG, HG_ERR_ROWS, HG_ERR_CAPTURE, HG_ERR_CUDA, HG_ERR_TIMEOUT, HG_ERR_STATE = range(7)
HG_MAX_TP = 32
HG_MAX_BEAMS, HG_MAX_PICKS, HG_MAX_STATES = 64, 128, 256


class HGError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} (status {status})")


class _Options(ctypes.Structure):
    _fields_ = [("poll_timeout_ns", ctypes.c_uint64), ("elems_per_lane", ctypes.c_int),
                ("ctas", ctypes.c_int), ("prefetch", ctypes.c_int), ("cooperative", ctypes.c_int),
                ("device_parity", ctypes.c_int), ("autotune", ctypes.c_int),
                ("timeline_calls", ctypes.c_int)]


_LIB: ctypes.CDLL | None = None


def library_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load libhg.so (built in-tree by ``_build.build()``); raises if absent."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with tp_vocab_logits_gb300._build.build()")
    lib = ctypes.CDLL(path)
    vp, vpp, i, st = ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_void_p
    lib.hg_create.argtypes = [i, i, i, ctypes.POINTER(i), i, ctypes.POINTER(vp)]
    lib.hg_create_ex.argtypes = [i, i, i, ctypes.POINTER(i), i, ctypes.POINTER(_Options),
                                 ctypes.POINTER(vp)]
    lib.hg_destroy.argtypes = [vp]
    lib.hg_gather.argtypes = [vp, vpp, vpp, i, st]
    lib.hg_gather_host.argtypes = [vp, vpp, vpp, i, st]
    lib.hg_sync.argtypes = [vp, st]
    lib.hg_rearm.argtypes = [vp, st]
    lib.hg_parity.argtypes = [vp]
    lib.hg_mailbox.argtypes = [vp, i, ctypes.POINTER(vp), ctypes.POINTER(ctypes.c_size_t)]
    ip = ctypes.POINTER(i)
    lib.hg_launch_shape.argtypes = [vp, i, ip, ip, ip, ip]
    lib.hg_debug_skip_push.argtypes = [vp, i]
    lib.hg_stock_gather.argtypes = [i, i, vpp, vpp, i, st]
    lib.hg_gather_fused.argtypes = [vp, vpp, vpp, vpp, vpp, i, i, st]
    lib.hg_gather_stats.argtypes = [vp, vpp, vpp, i, vp, st]
    lib.hg_timeline.argtypes = [vp, ctypes.POINTER(vp), ip, ip, ip]
    lib.hg_probe.argtypes = [i, i, i, vp, st]
    lib.hg_probe_scratch_bytes.argtypes = [i, i]
    lib.hg_probe_scratch_bytes.restype = ctypes.c_size_t
    sz, f = ctypes.c_size_t, ctypes.c_float
    lib.hg_vocab_create.argtypes = [i, i, i, i, i, i, i, sz, vpp]
    lib.hg_vocab_destroy.argtypes = [vp]
    lib.hg_vocab_workspace_bytes.argtypes = [vp]
    lib.hg_vocab_workspace_bytes.restype = sz
    lib.hg_vocab_sync.argtypes = [vp, st]
    lib.hg_vocab_embed.argtypes = [vp, vp, i, i, vp, f, vp, sz, st]
    lib.hg_vocab_embed_grad.argtypes = [vp, vp, i, i, vp, sz, vp, f, i, st]
    lib.hg_vocab_loss.argtypes = [vp, vp, sz, vp, vp, i, i, f, vp, vp, st]
    lib.hg_vocab_loss_grad.argtypes = [vp, vp, sz, vp, vp, i, vp, vp, i, f, vp, sz, vp, i, st]
    lib.hg_norm_create.argtypes = [i, i, i, vpp]
    lib.hg_norm_destroy.argtypes = [vp]
    lib.hg_norm_workspace_bytes.argtypes = [vp]
    lib.hg_norm_workspace_bytes.restype = sz
    lib.hg_norm_rows.argtypes = [vp, vp, sz, vp, sz, vp, sz, vp, f, i, vp, sz, i, vp, i, vp, st]
    lib.hg_norm_rows_grad.argtypes = [vp, vp, sz, vp, vp, vp, sz, vp, sz, i, vp, sz, vp, i, st]
    lib.hg_beam_create.argtypes = [i, i, i, i, i, vpp]
    lib.hg_beam_destroy.argtypes = [vp]
    lib.hg_beam_workspace_bytes.argtypes = [vp]
    lib.hg_beam_workspace_bytes.restype = sz
    lib.hg_beam_select.argtypes = [vp, vp, sz, vp, sz, vp, vp, i, i, vp, vp, i, vp, vp, st]
    lib.hg_beam_reorder.argtypes = [vp, vp, i, i, vp, i, st]
    lib.hg_strerror.argtypes = [i]
    lib.hg_strerror.restype = ctypes.c_char_p
    for name in ("hg_create", "hg_create_ex", "hg_destroy", "hg_gather", "hg_gather_host",
                 "hg_sync", "hg_rearm",
                 "hg_parity", "hg_mailbox", "hg_launch_shape", "hg_debug_skip_push",
                 "hg_stock_gather", "hg_gather_fused", "hg_gather_stats", "hg_timeline",
                 "hg_probe", "hg_vocab_create", "hg_vocab_destroy", "hg_vocab_sync",
                 "hg_vocab_embed", "hg_vocab_embed_grad", "hg_vocab_loss", "hg_vocab_loss_grad",
                 "hg_norm_create", "hg_norm_destroy", "hg_norm_rows", "hg_norm_rows_grad",
                 "hg_beam_create", "hg_beam_destroy", "hg_beam_select", "hg_beam_reorder"):
        getattr(lib, name).restype = i
    _LIB = lib
    return lib


def strerror(status: int) -> str:
    try:
        return load().hg_strerror(status).decode()
    except RuntimeError:
        return f"status {status}"


def _check(status: int, where: str) -> None:
    if status != HG_OK:
        raise HGError(status, where)


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr_array(tensors: Sequence[torch.Tensor]):
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


class Handle:
    """Owner of one hg_handle; freed by hg_destroy on close() or collection."""

    def __init__(self, ptr: int, tp: int, shard_cols: int, cap: int, rows):
        self.ptr = ptr
        self.tp, self.shard_cols, self.cap = tp, shard_cols, cap
        self.rows = frozenset(rows) if rows else frozenset(range(1, cap + 1))

    @property
    def V(self) -> int:
        return self.tp * self.shard_cols

    def close(self) -> None:
        if self.ptr:
            _check(load().hg_destroy(self.ptr), "hg_destroy")
            self.ptr = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def hg_create(tp: int, shard_cols: int, cap: int, rows: Sequence[int] | None = None, *,
              poll_timeout_ns: int = 0, elems_per_lane: int = 0, ctas: int = 0,
              prefetch: int = 0, cooperative: bool = False,
              device_parity: bool = False, autotune: bool = False,
              timeline_calls: int = 0) -> Handle:
    lib = load()
    rows = list(rows or [])
    arr = (ctypes.c_int * max(1, len(rows)))(*rows)
    out = ctypes.c_void_p()
    if poll_timeout_ns or elems_per_lane or ctas or prefetch or cooperative or device_parity \
            or autotune or timeline_calls:
        opt = _Options(poll_timeout_ns, elems_per_lane, ctas, prefetch, int(bool(cooperative)),
                       int(bool(device_parity)), int(bool(autotune)), int(timeline_calls))
        st = lib.hg_create_ex(tp, shard_cols, cap, arr, len(rows), ctypes.byref(opt),
                              ctypes.byref(out))
    else:
        st = lib.hg_create(tp, shard_cols, cap, arr, len(rows), ctypes.byref(out))
    _check(st, "hg_create")
    return Handle(out.value, tp, shard_cols, cap, rows)


def hg_destroy(h: Handle) -> None:
    h.close()


def _check_tensors(ts: Sequence[torch.Tensor], n: int, cols: int, M: int, what: str,
                   host: bool = False) -> None:
    if len(ts) != n:
        raise ValueError(f"{what}: expected {n} tensors, got {len(ts)}")
    for t in ts:
        if host:
            if not t.is_cuda and not t.is_pinned():
                raise ValueError(f"{what}: host tensors must be in page-locked memory")
        elif not t.is_cuda:
            raise ValueError(f"{what}: tensors must be on a CUDA device")
        if t.dtype not in (torch.bfloat16, torch.int16):
            raise ValueError(f"{what}: dtype must be bfloat16 (or its int16 bits), got {t.dtype}")
        if tuple(t.shape) != (M, cols) or not t.is_contiguous():
            raise ValueError(f"{what}: need contiguous [{M}, {cols}], got {tuple(t.shape)}")


def GatherCall(h: Handle, shards: Sequence[torch.Tensor], outs: Sequence[torch.Tensor], M: int,
               stream=None):
    """Marshalled arguments of one hg_gather call, reusable across calls with
    the same buffers: returns a callable that makes the call (raising HGError
    on a failed status). The callable is a small CPython object (the _hgcall
    extension) that calls the C entry point directly, so per-call host work
    is the C call itself. When any tensor is in (page-locked) host memory the
    call is hg_gather_host: the kernel reads and writes host memory directly
    over the host-device link."""
    host = any(not t.is_cuda for t in list(shards) + list(outs))
    _check_tensors(shards, h.tp, h.shard_cols, M, "shards", host)
    _check_tensors(outs, h.tp, h.V, M, "outs", host)
    entry = load().hg_gather_host if host else load().hg_gather
    fn = ctypes.cast(entry, ctypes.c_void_p).value
    return _pycall().Call(fn, h, [t.data_ptr() for t in shards], [t.data_ptr() for t in outs],
                          M, _stream_ptr(stream), (list(shards), list(outs)), _raise_gather)


def _raise_gather(status: int) -> None:
    raise HGError(status, "hg_gather")


_PYCALL = None


def _pycall():
    """The _hgcall extension (built in-tree next to libhg.so); raises if absent."""
    global _PYCALL
    if _PYCALL is None:
        import importlib
        if not os.path.exists(_build.PYCALL):
            raise RuntimeError(f"{_build.PYCALL} is missing: build it with "
                               "tp_vocab_logits_gb300._build.build()")
        _PYCALL = importlib.import_module("tp_vocab_logits_gb300._hgcall")
    return _PYCALL


def hg_gather(h: Handle, shards: Sequence[torch.Tensor], outs: Sequence[torch.Tensor],
              M: int | None = None, stream=None) -> None:
    """One gather: shards[r] is rank r's [M, W] bf16 logits, outs[d] rank d's
    [M, V] bf16 output (both lists of device tensors)."""
    M = shards[0].shape[0] if M is None else M
    GatherCall(h, shards, outs, M, stream)()


def hg_gather_host(h: Handle, shards: Sequence[torch.Tensor], outs: Sequence[torch.Tensor],
                   M: int | None = None, stream=None) -> None:
    """One gather whose shards and outputs are page-locked host tensors
    (``tensor.pin_memory()``) or device tensors: the kernel reads and writes
    host memory directly."""
    M = shards[0].shape[0] if M is None else M
    GatherCall(h, shards, outs, M, stream)()


def hg_gather_fused(h: Handle, hidden: Sequence[torch.Tensor], weight: Sequence[torch.Tensor],
                    outs: Sequence[torch.Tensor], M: int | None = None,
                    logits: Sequence[torch.Tensor] | None = None, stream=None) -> None:
    """LM head + gather in one launch: hidden[r] is rank r's [M, K] bf16 input,
    weight[r] its [W, K] bf16 lm_head weight (nn.Linear layout), outs[d] rank
    d's [M, V] output; logits, if given, receives each rank's [M, W] bf16
    logits."""
    M = hidden[0].shape[0] if M is None else M
    K = hidden[0].shape[1]
    _check_tensors(hidden, h.tp, K, M, "hidden")
    _check_tensors(weight, h.tp, K, h.shard_cols, "weight")
    _check_tensors(outs, h.tp, h.V, M, "outs")
    lp = None
    if logits is not None:
        _check_tensors(logits, h.tp, h.shard_cols, M, "logits")
        lp = _ptr_array(logits)
    st = load().hg_gather_fused(h.ptr, _ptr_array(hidden), _ptr_array(weight), lp,
                                _ptr_array(outs), M, K, _stream_ptr(stream))
    _check(st, "hg_gather_fused")


def new_row_stats(M: int, device="cuda") -> torch.Tensor:
    """Device buffer for M hg_row_stats records (int32 [M, 4])."""
    return torch.zeros((M, 4), dtype=torch.int32, device=device)


def unpack_row_stats(stats: torch.Tensor) -> dict:
    """max_logit, argmax, sum_exp, logsumexp columns of an hg_row_stats buffer."""
    f = stats.view(torch.float32)
    return {"max_logit": f[:, 0], "argmax": stats[:, 1], "sum_exp": f[:, 2], "logsumexp": f[:, 3]}


def hg_gather_stats(h: Handle, shards: Sequence[torch.Tensor], outs: Sequence[torch.Tensor],
                    stats: torch.Tensor, M: int | None = None, stream=None) -> None:
    """hg_gather plus per-row sampler statistics written into `stats`
    (a buffer from new_row_stats(M))."""
    M = shards[0].shape[0] if M is None else M
    _check_tensors(shards, h.tp, h.shard_cols, M, "shards")
    _check_tensors(outs, h.tp, h.V, M, "outs")
    if not stats.is_cuda or stats.dtype != torch.int32 or tuple(stats.shape) != (M, 4) \
            or not stats.is_contiguous():
        raise ValueError("stats: need a contiguous int32 CUDA tensor [M, 4] (new_row_stats)")
    _check(load().hg_gather_stats(h.ptr, _ptr_array(shards), _ptr_array(outs), M,
                                  stats.data_ptr(), _stream_ptr(stream)), "hg_gather_stats")


def hg_sync(h: Handle, stream=None) -> None:
    _check(load().hg_sync(h.ptr, _stream_ptr(stream)), "hg_sync")


def hg_rearm(h: Handle, stream=None) -> None:
    _check(load().hg_rearm(h.ptr, _stream_ptr(stream)), "hg_rearm")


def hg_parity(h: Handle) -> int:
    return int(load().hg_parity(h.ptr))


def hg_mailbox(h: Handle, rank: int) -> tuple:
    """(device pointer, bytes) of rank's [2, cap, V] bf16 mailbox."""
    p = ctypes.c_void_p()
    n = ctypes.c_size_t()
    _check(load().hg_mailbox(h.ptr, rank, ctypes.byref(p), ctypes.byref(n)), "hg_mailbox")
    return int(p.value), int(n.value)


class _DeviceView:
    """View of library-owned device memory for torch.as_tensor (only read)."""

    def __init__(self, ptr: int, shape: tuple, typestr: str):
        self.__cuda_array_interface__ = {"shape": shape, "typestr": typestr,
                                         "data": (ptr, False), "version": 3, "strides": None}


def mailbox_words(h: Handle, rank: int) -> torch.Tensor:
    """Copy of rank's mailbox as int32 words [2, cap, V / 2] (device tensor).
    Read it only while no gather of the handle is in flight."""
    ptr, nbytes = hg_mailbox(h, rank)
    shape = (2, h.cap, h.V // 2)
    assert nbytes == 4 * shape[0] * shape[1] * shape[2]
    view = torch.as_tensor(_DeviceView(ptr, shape, "<i4"), device="cuda")
    return view.clone()


def hg_launch_shape(h: Handle, M: int) -> dict:
    """Launch shape of row count M: ctas, threads, elems_per_lane, prefetch."""
    c, t, e, p = ctypes.c_int(), ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(load().hg_launch_shape(h.ptr, M, ctypes.byref(c), ctypes.byref(t), ctypes.byref(e),
                                  ctypes.byref(p)), "hg_launch_shape")
    return {"ctas": c.value, "threads": t.value, "elems_per_lane": e.value,
            "prefetch": bool(p.value)}


TIMELINE_SLOTS = 18  # HG_TIMELINE_SLOTS: entry, after the wait, one end time per warp


def hg_timeline(h: Handle) -> tuple:
    """(records, next): a copy of the handle's timeline as an int64 device
    tensor [calls, ctas, TIMELINE_SLOTS] of %globaltimer nanoseconds (slot 0
    entry, 1 after the wait, 2 + d when warp d finished), and the index of the
    record the next call writes. Read it only while no gather is in flight."""
    p = ctypes.c_void_p()
    calls, ctas, nxt = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(load().hg_timeline(h.ptr, ctypes.byref(p), ctypes.byref(calls), ctypes.byref(ctas),
                              ctypes.byref(nxt)), "hg_timeline")
    shape = (calls.value, ctas.value, TIMELINE_SLOTS)
    view = torch.as_tensor(_DeviceView(int(p.value), shape, "<i8"), device="cuda")
    return view.clone(), nxt.value


def hg_probe_scratch_bytes(ctas: int, threads: int) -> int:
    return int(load().hg_probe_scratch_bytes(ctas, threads))


def hg_probe(kind: int, ctas: int, threads: int, scratch: torch.Tensor | None = None,
             stream=None) -> None:
    """Measurement kernels launched as the gather is (see include/hg.h):
    kind 0 empty dependent launch, 1 one-vector push/poll/copy/re-arm
    handoff, 2 arm the handoff's scratch (a device tensor of at least
    hg_probe_scratch_bytes(ctas, threads) bytes)."""
    ptr = None
    if scratch is not None:
        if not scratch.is_cuda or scratch.numel() * scratch.element_size() < \
                hg_probe_scratch_bytes(ctas, threads):
            raise ValueError("scratch: need a CUDA tensor of hg_probe_scratch_bytes bytes")
        ptr = scratch.data_ptr()
    _check(load().hg_probe(kind, ctas, threads, ptr, _stream_ptr(stream)), "hg_probe")


def hg_debug_skip_push(h: Handle, rank: int) -> None:
    _check(load().hg_debug_skip_push(h.ptr, rank), "hg_debug_skip_push")


def hg_stock_gather(shards: Sequence[torch.Tensor], outs: Sequence[torch.Tensor],
                    M: int | None = None, stream=None) -> None:
    tp = len(shards)
    M = shards[0].shape[0] if M is None else M
    W = shards[0].shape[1]
    _check_tensors(shards, tp, W, M, "shards")
    _check_tensors(outs, tp, tp * W, M, "outs")
    _check(load().hg_stock_gather(tp, W, _ptr_array(shards), _ptr_array(outs), M,
                                  _stream_ptr(stream)), "hg_stock_gather")


HG_STATIC_MAILBOX_BYTES = 24 * 1024 * 1024


def hg_gather_static(shards: Sequence[torch.Tensor], outs: Sequence[torch.Tensor],
                     M: int | None = None, status_out: torch.Tensor | None = None,
                     stream=None) -> None:
    """The gather without any allocation (libhg's hg_gather_static), for callers
    that cannot allocate device memory; its mailbox is a fixed array inside the
    library, shared by every call. shards/outs as for hg_gather; status_out, if
    given, is a one-element int32 device tensor set to 0 (ok) or 1 (a poll gave
    up) in stream order."""
    fn = load().hg_gather_static
    fn.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_void_p),
                   ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_void_p,
                   ctypes.c_void_p]
    fn.restype = ctypes.c_int
    tp = len(shards)
    M = shards[0].shape[0] if M is None else M
    W = shards[0].shape[1]
    need = tp * M * tp * W * 2
    if need > HG_STATIC_MAILBOX_BYTES:
        raise ValueError(f"hg_gather_static: tp={tp}, M={M}, shard_cols={W} needs {need} "
                         f"bytes of mailbox, the fixed maximum is {HG_STATIC_MAILBOX_BYTES}")
    _check_tensors(shards, tp, W, M, "shards")
    _check_tensors(outs, tp, tp * W, M, "outs")
    st_ptr = None
    if status_out is not None:
        if not status_out.is_cuda or status_out.dtype != torch.int32 or status_out.numel() < 1:
            raise ValueError("status_out: need an int32 CUDA tensor with one element")
        st_ptr = status_out.data_ptr()
    _check(fn(tp, W, _ptr_array(shards), _ptr_array(outs), M, st_ptr, _stream_ptr(stream)),
           "hg_gather_static")


_VOCAB_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # HG_BF16, ...
_VOCAB_OPS = {"embed": 1, "embed_grad": 2, "loss": 4, "loss_grad": 8}  # HG_VOCAB_*


class VocabHandle:
    """Owner of one hg_vocab (the workspace of the vocabulary operators); freed
    by hg_vocab_destroy on close() or collection."""

    def __init__(self, ptr: int, tp: int, shard_cols: int, vocab: int, hidden: int, max_rows: int,
                 dtype: torch.dtype, device: int = 0):
        self.ptr = ptr
        self.tp, self.shard_cols, self.vocab = tp, shard_cols, vocab
        self.hidden, self.max_rows, self.dtype = hidden, max_rows, dtype
        self.device = torch.device("cuda", device)
        self._describe()

    def _describe(self) -> None:
        self.desc = struct.pack("Pqqqq", self.ptr, self.tp, self.shard_cols, self.hidden,
                                self.device.index)  # for _hgcall

    @property
    def workspace_bytes(self) -> int:
        return int(load().hg_vocab_workspace_bytes(self.ptr))

    def close(self) -> None:
        if self.ptr:
            ptr, self.ptr = self.ptr, 0
            self._describe()
            _check(load().hg_vocab_destroy(ptr), "hg_vocab_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def hg_vocab_create(tp: int, shard_cols: int, hidden: int, max_rows: int, *, vocab: int = 0,
                    dtype: torch.dtype = torch.bfloat16,
                    ops: Sequence[str] = ("embed", "embed_grad", "loss", "loss_grad"),
                    piece_bytes: int = 0) -> VocabHandle:
    """Workspace of the vocabulary operators on a [tp * shard_cols, hidden]
    matrix in tp shards, for calls of up to max_rows rows. vocab: the real
    vocabulary where the last shards are padded (0: all of it). ops: which of
    "embed", "embed_grad", "loss", "loss_grad" will be called (each needs its
    own workspace). piece_bytes: see include/hg.h. The handle is of the current
    device; calls take that device's tensors, and want it current."""
    if dtype not in _VOCAB_TYPES:
        raise ValueError("hg_vocab_create: dtype must be bfloat16, float16 or float32, got "
                         f"{dtype}")
    bits = 0
    for op in ops:
        if op not in _VOCAB_OPS:
            raise ValueError(f"hg_vocab_create: unknown operator {op!r}")
        bits |= _VOCAB_OPS[op]
    out = ctypes.c_void_p()
    _check(load().hg_vocab_create(tp, shard_cols, vocab, hidden, max_rows, _VOCAB_TYPES[dtype],
                                  bits, piece_bytes, ctypes.byref(out)), "hg_vocab_create")
    return VocabHandle(out.value, tp, shard_cols, vocab or tp * shard_cols, hidden, max_rows, dtype,
                       torch.cuda.current_device())


def hg_vocab_destroy(h: VocabHandle) -> None:
    h.close()


def hg_vocab_sync(h: VocabHandle, stream=None) -> None:
    _check(load().hg_vocab_sync(h.ptr, _stream_ptr(stream)), "hg_vocab_sync")


# The calls below check their tensors and reach the library in _hgcall (in
# Python the checks cost more than the launch). Where a check fails there it
# answers None, and the checks here, which are the same, say which.
_VOCAB_CALL = None


def _vocab_call():
    global _VOCAB_CALL
    if _VOCAB_CALL is None:
        lib, mod = load(), _pycall()
        mod.bind_vocab(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.hg_vocab_embed, lib.hg_vocab_embed_grad, lib.hg_vocab_loss,
            lib.hg_vocab_loss_grad)], torch.int32, torch.int64, torch.float32,
            getattr(torch._C, "_cuda_getCurrentRawStream", _current_raw_stream))
        _VOCAB_CALL = mod
    return _VOCAB_CALL


def _current_raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _vocab_refuse(where: str, *checks) -> None:
    """Run the checks that _hgcall found wanting; one of them raises."""
    for check in checks:
        check()
    raise ValueError(f"{where}: invalid arguments")


def _vocab_device(h: VocabHandle, t: torch.Tensor, what: str) -> None:
    if t.is_cuda and t.get_device() != h.device.index:
        raise ValueError(f"{what}: need a tensor on {h.device}, got one on {t.device}")


def _vocab_ids(h: VocabHandle, t: torch.Tensor, what: str) -> None:
    _vocab_device(h, t, what)
    if not t.is_cuda or t.dtype not in (torch.int32, torch.int64) or t.dim() != 1 \
            or not t.is_contiguous():
        raise ValueError(f"{what}: need a contiguous 1-D int32 or int64 CUDA tensor")


def _vocab_rows(h: VocabHandle, t: torch.Tensor, n: int, what: str) -> None:
    """A token-side [n, hidden] matrix (rows contiguous)."""
    _vocab_device(h, t, what)
    if not t.is_cuda or t.dtype != h.dtype:
        raise ValueError(f"{what}: need a CUDA tensor of {h.dtype}, got {t.dtype} on {t.device}")
    if t.shape != (n, h.hidden) or (h.hidden > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: need [{n}, {h.hidden}] with contiguous rows, got "
                         f"{tuple(t.shape)} with strides {t.stride()}")
    if n > 1 and t.stride(0) < h.hidden:
        raise ValueError(f"{what}: rows overlap (row stride {t.stride(0)})")


def _vocab_shards(h: VocabHandle, ts: Sequence[torch.Tensor], what: str) -> None:
    if not isinstance(ts, (list, tuple)):
        raise ValueError(f"{what}: need a list of {h.tp} shards")
    if len(ts) != h.tp:
        raise ValueError(f"{what}: expected {h.tp} shards, got {len(ts)}")
    for t in ts:
        _vocab_device(h, t, what)
        if not t.is_cuda or t.dtype != h.dtype:
            raise ValueError(f"{what}: need CUDA tensors of {h.dtype}, got {t.dtype} on {t.device}")
        if t.shape != (h.shard_cols, h.hidden) or not t.is_contiguous():
            raise ValueError(f"{what}: need contiguous [{h.shard_cols}, {h.hidden}], got "
                             f"{tuple(t.shape)}")


def _vocab_floats(h: VocabHandle, t: torch.Tensor, n: int, what: str) -> None:
    _vocab_device(h, t, what)
    if not t.is_cuda or t.dtype != torch.float32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what}: need a contiguous float32 CUDA tensor [{n}]")


def hg_vocab_embed(h: VocabHandle, tokens: torch.Tensor, table: Sequence[torch.Tensor],
                   out: torch.Tensor, scale: float = 1.0, stream=None) -> None:
    """out[n] = scale * table[tokens[n]]; a token outside [0, vocab) gives zeros."""
    st = _vocab_call().vocab_embed(h.desc, h.dtype, tokens, table, out, scale,
                                   None if stream is None else _stream_ptr(stream))
    if st is None:
        _vocab_refuse("hg_vocab_embed", lambda: _vocab_ids(h, tokens, "tokens"),
                      lambda: _vocab_shards(h, table, "table"),
                      lambda: _vocab_rows(h, out, tokens.shape[0], "out"))
    _check(st, "hg_vocab_embed")


def hg_vocab_embed_grad(h: VocabHandle, tokens: torch.Tensor, grad_out: torch.Tensor,
                        grad_table: Sequence[torch.Tensor], scale: float = 1.0,
                        accumulate: bool = False, stream=None) -> None:
    """grad_table[v] = scale * sum of grad_out[n] over tokens[n] = v (every row
    written), or added to grad_table where accumulate."""
    st = _vocab_call().vocab_embed_grad(h.desc, h.dtype, tokens, grad_out, grad_table, scale,
                                        accumulate,
                                        None if stream is None else _stream_ptr(stream))
    if st is None:
        _vocab_refuse("hg_vocab_embed_grad", lambda: _vocab_ids(h, tokens, "tokens"),
                      lambda: _vocab_rows(h, grad_out, tokens.shape[0], "grad_out"),
                      lambda: _vocab_shards(h, grad_table, "grad_table"))
    _check(st, "hg_vocab_embed_grad")


def hg_vocab_loss(h: VocabHandle, hidden: torch.Tensor, weight: Sequence[torch.Tensor],
                  targets: torch.Tensor, loss: torch.Tensor, lse: torch.Tensor,
                  logit_scale: float = 1.0, stream=None) -> None:
    """Per-row softmax cross entropy of logit_scale * hidden @ weight.T and its
    logsumexp, without storing logits. A negative target masks its row."""
    st = _vocab_call().vocab_loss(h.desc, h.dtype, hidden, weight, targets, loss, lse, logit_scale,
                                  None if stream is None else _stream_ptr(stream))
    if st is None:
        _vocab_refuse("hg_vocab_loss", lambda: _vocab_ids(h, targets, "targets"),
                      lambda: _vocab_rows(h, hidden, targets.shape[0], "hidden"),
                      lambda: _vocab_shards(h, weight, "weight"),
                      lambda: _vocab_floats(h, loss, targets.shape[0], "loss"),
                      lambda: _vocab_floats(h, lse, targets.shape[0], "lse"))
    _check(st, "hg_vocab_loss")


def hg_vocab_loss_grad(h: VocabHandle, hidden: torch.Tensor, weight: Sequence[torch.Tensor],
                       targets: torch.Tensor, lse: torch.Tensor, grad_loss: torch.Tensor,
                       grad_hidden: torch.Tensor | None,
                       grad_weight: Sequence[torch.Tensor] | None, logit_scale: float = 1.0,
                       accumulate: bool = False, stream=None) -> None:
    """Gradient of hg_vocab_loss from its logsumexp and the upstream gradient of
    each row's loss, to grad_hidden and grad_weight (either may be None);
    accumulate adds to what grad_weight holds."""
    st = _vocab_call().vocab_loss_grad(h.desc, h.dtype, hidden, weight, targets, lse, grad_loss,
                                       grad_hidden, grad_weight, logit_scale, accumulate,
                                       None if stream is None else _stream_ptr(stream))
    if st is None:
        _vocab_refuse("hg_vocab_loss_grad", lambda: _vocab_ids(h, targets, "targets"),
                      lambda: _vocab_rows(h, hidden, targets.shape[0], "hidden"),
                      lambda: _vocab_shards(h, weight, "weight"),
                      lambda: _vocab_floats(h, lse, targets.shape[0], "lse"),
                      lambda: _vocab_floats(h, grad_loss, targets.shape[0], "grad_loss"),
                      lambda: grad_hidden is None or _vocab_rows(h, grad_hidden, targets.shape[0],
                                                                 "grad_hidden"),
                      lambda: grad_weight is None or _vocab_shards(h, grad_weight, "grad_weight"))
    _check(st, "hg_vocab_loss_grad")


class _StepHandle:
    """What the handles of the norm and the beam search share: the pointer, the device, and
    the record that _hgcall reads."""

    _kind = ""

    def __init__(self, ptr: int, dtype: torch.dtype, device: int):
        self.ptr, self.dtype = ptr, dtype
        self.device = torch.device("cuda", device)
        self._describe()

    def _sizes(self) -> tuple:
        raise NotImplementedError

    def _describe(self) -> None:
        self.desc = struct.pack("Pqqqq", self.ptr, *self._sizes(), self.device.index)

    @property
    def workspace_bytes(self) -> int:
        return int(getattr(load(), f"{self._kind}_workspace_bytes")(self.ptr))

    def close(self) -> None:
        if self.ptr:
            ptr, self.ptr = self.ptr, 0
            self._describe()
            _check(getattr(load(), f"{self._kind}_destroy")(ptr), f"{self._kind}_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class NormHandle(_StepHandle):
    """Owner of one hg_norm; freed by hg_norm_destroy on close() or collection."""

    _kind = "hg_norm"

    def __init__(self, ptr: int, hidden: int, max_rows: int, dtype: torch.dtype, device: int = 0):
        self.hidden, self.max_rows = hidden, max_rows
        super().__init__(ptr, dtype, device)

    def _sizes(self) -> tuple:
        return _VOCAB_TYPES[self.dtype], 0, self.hidden


class BeamHandle(_StepHandle):
    """Owner of one hg_beam; freed by hg_beam_destroy on close() or collection."""

    _kind = "hg_beam"

    def __init__(self, ptr: int, max_items: int, beams: int, vocab: int, picks: int,
                 dtype: torch.dtype, device: int = 0):
        self.max_items, self.beams, self.vocab, self.picks = max_items, beams, vocab, picks
        super().__init__(ptr, dtype, device)

    def _sizes(self) -> tuple:
        return self.beams, self.picks, self.vocab


_STEP_CALL = None


def _step_call():
    global _STEP_CALL
    if _STEP_CALL is None:
        lib, mod = load(), _pycall()
        mod.bind_steps(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.hg_norm_rows, lib.hg_norm_rows_grad, lib.hg_beam_select, lib.hg_beam_reorder)],
            torch.int32, torch.int64, torch.float32, torch.float8_e4m3fn, torch.bool, torch.uint8,
            getattr(torch._C, "_cuda_getCurrentRawStream", _current_raw_stream))
        _STEP_CALL = mod
    return _STEP_CALL


def _step_dtype(dtype: torch.dtype, where: str) -> int:
    if dtype not in _VOCAB_TYPES:
        raise ValueError(f"{where}: dtype must be bfloat16, float16 or float32, got {dtype}")
    return _VOCAB_TYPES[dtype]


def _step_tensor(h: _StepHandle, t: torch.Tensor, types: Sequence[torch.dtype], what: str) -> None:
    _vocab_device(h, t, what)
    if not t.is_cuda or t.dtype not in types:
        raise ValueError(f"{what}: need a CUDA tensor of {' or '.join(map(str, types))}, got "
                         f"{t.dtype} on {t.device}")


def _step_table(h: _StepHandle, t: torch.Tensor, types: Sequence[torch.dtype], shape: tuple,
                what: str) -> None:
    _step_tensor(h, t, types, what)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{what}: need a contiguous {list(shape)}, got {tuple(t.shape)} with "
                         f"strides {t.stride()}")


def _step_rows(h: _StepHandle, t: torch.Tensor, dtype: torch.dtype, n: int, width: int,
               what: str) -> None:
    """An [n, width] matrix, rows contiguous."""
    _step_tensor(h, t, (dtype,), what)
    if tuple(t.shape) != (n, width) or (width > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: need [{n}, {width}] with contiguous rows, got "
                         f"{tuple(t.shape)} with strides {t.stride()}")
    if n > 1 and t.stride(0) < width:
        raise ValueError(f"{what}: rows overlap (row stride {t.stride(0)})")


def _step_count(t: torch.Tensor, what: str) -> int:
    if t.dim() != 2:
        raise ValueError(f"{what}: need a matrix, got {tuple(t.shape)}")
    return t.shape[0]


def hg_norm_create(hidden: int, max_rows: int, *, dtype: torch.dtype = torch.bfloat16) -> NormHandle:
    """The norm of rows of `hidden` elements of dtype, for calls of up to max_rows
    rows. The handle is of the current device; calls take that device's tensors, and
    want it current."""
    code = _step_dtype(dtype, "hg_norm_create")
    out = ctypes.c_void_p()
    _check(load().hg_norm_create(hidden, max_rows, code, ctypes.byref(out)), "hg_norm_create")
    return NormHandle(out.value, hidden, max_rows, dtype, torch.cuda.current_device())


def hg_norm_destroy(h: NormHandle) -> None:
    h.close()


def _norm_scales(h: NormHandle, t: torch.Tensor, n: int) -> None:
    blocks = -(-h.hidden // 128)
    if t.dim() == 2 and t.shape[1] == 1:
        blocks = 1
    _step_table(h, t, (torch.float32,), (n, blocks), "scales")


def hg_norm_rows(h: NormHandle, x: torch.Tensor, gain: torch.Tensor, out: torch.Tensor,
                 residual: torch.Tensor | None = None, sum_out: torch.Tensor | None = None,
                 rstd: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                 eps: float = 1e-6, stream=None) -> None:
    """s = x + residual (written to sum_out), out = s * rstd * gain with rstd = 1 /
    sqrt(mean of s^2 + eps) per row. With scales, float32 [N, 1] (one per row) or
    [N, ceil(hidden / 128)] (one per 128 columns), out is float8_e4m3fn and its values
    are out * scales."""
    st = _step_call().norm_rows(h.desc, h.dtype, x, gain, out, residual, sum_out, rstd, scales, eps,
                                None if stream is None else _stream_ptr(stream))
    if st is None:
        n = _step_count(x, "x")
        out_type = h.dtype if scales is None else torch.float8_e4m3fn
        _vocab_refuse(
            "hg_norm_rows", lambda: _step_rows(h, x, h.dtype, n, h.hidden, "x"),
            lambda: _step_table(h, gain, (h.dtype,), (h.hidden,), "gain"),
            lambda: _step_rows(h, out, out_type, n, h.hidden, "out"),
            lambda: residual is None or _step_rows(h, residual, h.dtype, n, h.hidden, "residual"),
            lambda: sum_out is None or _step_rows(h, sum_out, h.dtype, n, h.hidden, "sum_out"),
            lambda: rstd is None or _step_table(h, rstd, (torch.float32,), (n,), "rstd"),
            lambda: scales is None or _norm_scales(h, scales, n))
    _check(st, "hg_norm_rows")


def hg_norm_rows_grad(h: NormHandle, s: torch.Tensor, gain: torch.Tensor, rstd: torch.Tensor,
                      grad_out: torch.Tensor, grad_x: torch.Tensor | None,
                      grad_gain: torch.Tensor | None, grad_sum: torch.Tensor | None = None,
                      accumulate: bool = False, stream=None) -> None:
    """Gradient of hg_norm_rows from its s and rstd, to grad_x (of x and residual
    alike) and grad_gain (either may be None); grad_sum is what reaches s by the
    residual stream, accumulate adds to what grad_gain holds."""
    st = _step_call().norm_rows_grad(h.desc, h.dtype, s, gain, rstd, grad_out, grad_x, grad_gain,
                                     grad_sum, accumulate,
                                     None if stream is None else _stream_ptr(stream))
    if st is None:
        n = _step_count(s, "s")
        _vocab_refuse(
            "hg_norm_rows_grad", lambda: _step_rows(h, s, h.dtype, n, h.hidden, "s"),
            lambda: _step_table(h, gain, (h.dtype,), (h.hidden,), "gain"),
            lambda: _step_table(h, rstd, (torch.float32,), (n,), "rstd"),
            lambda: _step_rows(h, grad_out, h.dtype, n, h.hidden, "grad_out"),
            lambda: grad_x is None or _step_rows(h, grad_x, h.dtype, n, h.hidden, "grad_x"),
            lambda: grad_gain is None or _step_table(h, grad_gain, (h.dtype,), (h.hidden,),
                                                     "grad_gain"),
            lambda: grad_sum is None or _step_rows(h, grad_sum, h.dtype, n, h.hidden, "grad_sum"))
    _check(st, "hg_norm_rows_grad")


def hg_beam_create(max_items: int, beams: int, vocab: int, picks: int, *,
                   dtype: torch.dtype = torch.bfloat16) -> BeamHandle:
    """The workspace of a beam search of up to max_items items of `beams` beams, with
    `picks` continuations chosen per item, on logits of dtype. The handle is of the
    current device; calls take that device's tensors, and want it current."""
    code = _step_dtype(dtype, "hg_beam_create")
    out = ctypes.c_void_p()
    _check(load().hg_beam_create(max_items, beams, vocab, picks, code, ctypes.byref(out)),
           "hg_beam_create")
    return BeamHandle(out.value, max_items, beams, vocab, picks, dtype, torch.cuda.current_device())


def hg_beam_destroy(h: BeamHandle) -> None:
    h.close()


def _beam_lse(h: BeamHandle, t: torch.Tensor, rows: int) -> None:
    _step_tensor(h, t, (torch.float32,), "lse")
    if tuple(t.shape) != (rows,) or (rows > 1 and t.stride(0) < 1):
        raise ValueError(f"lse: need [{rows}], got {tuple(t.shape)} with strides {t.stride()}")


def _beam_end(h: BeamHandle, end: int) -> None:
    if not -1 <= end < h.vocab:
        raise ValueError(f"end: need a token in [0, {h.vocab}) or -1, got {end}")


def hg_beam_select(h: BeamHandle, logits: torch.Tensor, scores: torch.Tensor, tokens: torch.Tensor,
                   parents: torch.Tensor, picked: torch.Tensor, lse: torch.Tensor | None = None,
                   finished: torch.Tensor | None = None, end: int = -1,
                   picked_finished: torch.Tensor | None = None, stream=None) -> None:
    """The best continuations of each item, by scores [items, beams] + logits - lse:
    tokens, parents (int32 or int64), picked (their totals) and picked_finished (bool or
    uint8), all [items, picks]. logits: [items * beams, vocab]. lse: the logits'
    logsumexp (the column of unpack_row_stats, say), computed here where it is None.
    finished [items, beams] (bool or uint8): beams that go on with the token `end` alone."""
    st = _step_call().beam_select(h.desc, h.dtype, logits, scores, tokens, parents, picked, lse,
                                  finished, end, picked_finished,
                                  None if stream is None else _stream_ptr(stream))
    if st is None:
        n = _step_count(scores, "scores")
        ids, flags = (torch.int64, torch.int32), (torch.bool, torch.uint8)
        _vocab_refuse(
            "hg_beam_select",
            lambda: _step_table(h, scores, (torch.float32,), (n, h.beams), "scores"),
            lambda: _step_rows(h, logits, h.dtype, n * h.beams, h.vocab, "logits"),
            lambda: _step_table(h, tokens, ids, (n, h.picks), "tokens"),
            lambda: _step_table(h, parents, (tokens.dtype,), (n, h.picks), "parents"),
            lambda: _step_table(h, picked, (torch.float32,), (n, h.picks), "picked"),
            lambda: lse is None or _beam_lse(h, lse, n * h.beams),
            lambda: finished is None or _step_table(h, finished, flags, (n, h.beams), "finished"),
            lambda: picked_finished is None or _step_table(h, picked_finished, flags, (n, h.picks),
                                                           "picked_finished"),
            lambda: _beam_end(h, end))
    _check(st, "hg_beam_select")


def _beam_steps(t: torch.Tensor, dim: int) -> int:
    """Strides that step between the contiguous runs of a row."""
    steps = []
    others = [(t.stride(i), t.shape[i]) for i in range(t.dim()) if i != dim and t.shape[i] != 1]
    for stride, size in sorted(others, key=lambda d: -d[0]):
        if steps and steps[-1][0] == stride * size:
            steps[-1] = (stride, steps[-1][1] * size)
        else:
            steps.append((stride, size))
    return len(steps) - bool(steps and steps[-1][0] == 1)


def _beam_state(h: BeamHandle, state, rows: int) -> None:
    t, dim = state if isinstance(state, tuple) and len(state) == 2 else (state, 0)
    if not hasattr(t, "is_cuda") or not isinstance(dim, int):
        raise ValueError("states: need tensors, or pairs of a tensor and a dimension")
    _vocab_device(h, t, "states")
    if not t.is_cuda:
        raise ValueError(f"states: need CUDA tensors, got one on {t.device}")
    if not -t.dim() <= dim < t.dim() or t.shape[dim] != rows:
        raise ValueError(f"states: need {rows} rows in dimension {dim} of {tuple(t.shape)}")
    if t.numel() and _beam_steps(t, dim % t.dim()) > 2:
        raise ValueError(f"states: {tuple(t.shape)} with strides {t.stride()} has more than two "
                         "steps between its contiguous runs")


def hg_beam_reorder(h: BeamHandle, parents: torch.Tensor, states: Sequence, stream=None) -> None:
    """In place, row item * beams + j of every state takes what row item * beams +
    parents[item, j] held; a parent outside [0, beams) leaves its row. parents: int32 or
    int64 [items, beams]. states: tensors with their rows in dimension 0, or pairs of a
    tensor and the dimension of its rows; views of a larger cache are fine."""
    st = _step_call().beam_reorder(h.desc, parents, states,
                                   None if stream is None else _stream_ptr(stream))
    if st is None:
        n = _step_count(parents, "parents")
        _step_table(h, parents, (torch.int64, torch.int32), (n, h.beams), "parents")
        if not isinstance(states, (list, tuple)) or len(states) > HG_MAX_STATES:
            raise ValueError(f"states: need a list of at most {HG_MAX_STATES}")
        _vocab_refuse("hg_beam_reorder", *[lambda s=s: _beam_state(h, s, n * h.beams)
                                           for s in states])
    _check(st, "hg_beam_reorder")
