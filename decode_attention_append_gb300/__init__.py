"""GB300 (sm_103a) paged KV append + mixed-batch paged attention.

A thin ctypes binding over the C ABI of ``libdaa.so`` (declared in
``include/daa.h``).  It only marshals torch tensors into pointers and sizes:
every step of the computation runs in the library's CUDA kernels.  There is no
CPU or PyTorch fallback; if the library is missing the calls raise.

Entry points (same names as the C ABI, without the ``daa_`` prefix):

* ``kv_append(k_new, v_new, kv_pages, append_indptr, page_indices, kv_indptr,
  last_page_len)`` -- write each new token's K/V into its page slot.
* ``batch_attention(q, kv_pages, qo_indptr, kv_indptr, page_indices,
  last_page_len, causal, sm_scale, ...)`` -- attention for a batch mixing
  chunked-prefill requests (qo_len > 1, causal with the cache offset) and decode
  requests (qo_len = 1).
* ``batch_attention_tree(..., tree_mask, ...)`` -- the same attention with
  draft-tree masks over each request's new tokens (speculative-decoding
  verification of a tree of draft tokens).
* ``BatchAttention`` -- plans once from host copies of the page table and owns
  the workspace, for repeated calls over the same batch shape.
* ``PagePool`` -- the pages of many requests on the device; builds a step's page
  table there from the requests' lengths, and takes pages back.
* ``kv_append_q4``, ``kv_dequant_q4``, ``BatchAttentionQ4`` -- append, read-back
  and attention on a KV cache held in 4 bits (``new_q4_pool``).
* ``Rope``, ``apply_rope``, ``append_rope``, ``append_rope_q4`` -- rotary positions:
  query and key rows rotated, alone or on the way into either cache.

Tensors: bf16 ``q [nnz_qo, Hq, d]``, ``k_new/v_new [nnz_new, Hkv, d]``, page
pool ``kv_pages [num_pages, 2, Hkv, page_size, d]`` (K then V, HND inside a
page), int32 CSR arrays on the same CUDA device.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import functools
import importlib.util
import math
import os
import threading
import weakref
from dataclasses import dataclass

import numpy as np
import torch

from .rope import frequencies_of, rope_frequencies

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "libdaa.so")
_lib = None
_lock = threading.Lock()

DAA_OK = 0
STATUS = {0: "ok", -1: "invalid argument", -2: "shape", -3: "page range", -4: "unsupported",
          -5: "CUDA error", -6: "workspace", -7: "alignment"}
KERNEL_NAMES = {1: "kv_append", 2: "decode_splitkv", 3: "softmax_merge", 4: "prefill_tc", 5: "decode_tc",
                6: "short_tc", 7: "step_table", 8: "kv_append_q4", 9: "kv_dequant_q4", 10: "attention_q4",
                11: "rope", 12: "append_rope", 13: "append_rope_q4"}


class DaaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status})")
        self.status = status


class _Dims(ctypes.Structure):
    _fields_ = [("num_qo_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int64)]


class StepLayout(ctypes.Structure):
    """daa_step_layout: byte offsets of a host step's sections in its packed buffer."""
    _fields_ = [(n, ctypes.c_size_t) for n in ("qo_indptr", "kv_indptr", "page_indices", "last_page_len",
                                               "q", "k_new", "v_new", "total")]


class StepStreams(ctypes.Structure):
    """daa_step_streams: the streams and events of one host step."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("upload_stream", "compute_stream", "download_stream",
                                               "uploaded", "computed", "downloaded", "inputs_free",
                                               "out_free")]


class _Pool(ctypes.Structure):
    """daa_page_pool: device arrays of a page pool."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("seq_len", "held", "block_table", "free_pages", "counters")] + \
               [(n, ctypes.c_int32) for n in ("num_slots", "max_pages", "num_pages", "page_size")]


class PlanInfo(ctypes.Structure):
    """daa_plan_info: the record of a plan uploaded by ``batch_attention_plan``."""
    _fields_ = [("words", ctypes.c_int64 * 24)]


class _Rope(ctypes.Structure):
    """daa_rope: the frequencies of a rotation."""
    _fields_ = [("turns", ctypes.c_uint64 * 64), ("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("magnitude", ctypes.c_double)]


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libdaa.so (built by ``build.build()``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"libdaa.so not built at {_LIB_PATH}; run decode_attention_append_gb300.build.build()")
        lib = ctypes.CDLL(_LIB_PATH)
        vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        lib.daa_status_string.restype = ctypes.c_char_p
        lib.daa_status_string.argtypes = [i32]
        lib.daa_version.restype = i32
        lib.daa_kv_append.restype = i32
        lib.daa_kv_append.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, _Dims, vp]
        lib.daa_batch_attention_workspace_size.restype = sz
        lib.daa_batch_attention_workspace_size.argtypes = [vp, vp, vp, i32, _Dims, ctypes.POINTER(i32)]
        lib.daa_batch_attention.restype = i32
        lib.daa_batch_attention.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, f32, vp, vp,
                                            vp, sz, _Dims, vp]
        lib.daa_append_attention.restype = i32
        lib.daa_append_attention.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, f32,
                                             vp, vp, vp, sz, _Dims, vp]
        lib.daa_batch_attention_tree.restype = i32
        lib.daa_batch_attention_tree.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, f32,
                                                 vp, vp, vp, sz, _Dims, vp]
        lib.daa_batch_attention_noalloc.restype = i32
        lib.daa_batch_attention_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, f32,
                                                    vp, vp, _Dims, vp]
        lib.daa_batch_attention_shared_prefix_workspace_size.restype = sz
        lib.daa_batch_attention_shared_prefix_workspace_size.argtypes = [
            vp, vp, vp, i32, vp, vp, i32, _Dims, ctypes.POINTER(i32)]
        lib.daa_batch_attention_shared_prefix.restype = i32
        lib.daa_batch_attention_shared_prefix.argtypes = [
            vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, f32, vp, vp, vp, sz, _Dims, vp]
        lib.daa_append_attention_shared_prefix.restype = i32
        lib.daa_append_attention_shared_prefix.argtypes = [
            vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, f32, vp, vp, vp, sz,
            _Dims, vp]
        pinfo = ctypes.POINTER(PlanInfo)
        lib.daa_batch_attention_plan.restype = i32
        lib.daa_batch_attention_plan.argtypes = [vp, vp, vp, i32, vp, vp, i32, _Dims, vp, sz, pinfo, vp]
        lib.daa_batch_attention_run.restype = i32
        lib.daa_batch_attention_run.argtypes = [vp, vp, vp, vp, vp, vp, pinfo, i32, f32, vp, vp, vp, sz,
                                                _Dims, vp]
        lib.daa_append_attention_run.restype = i32
        lib.daa_append_attention_run.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, pinfo, i32, f32, vp, vp,
                                                 vp, sz, _Dims, vp]
        lib.daa_append_attention_host.restype = i32
        lib.daa_append_attention_host.argtypes = [vp, vp, ctypes.POINTER(StepLayout), i32, i32, f32, vp, vp,
                                                  vp, vp, sz, _Dims, ctypes.POINTER(StepStreams)]
        ppool = ctypes.POINTER(_Pool)
        lib.daa_step_table.restype = i32
        lib.daa_step_table.argtypes = [ppool, vp, vp, i32, i32, vp, vp, vp, i32, vp, vp, vp, i32, vp]
        lib.daa_release_pages.restype = i32
        lib.daa_release_pages.argtypes = [ppool, vp, i32, vp]
        lib.daa_kv_append_q4.restype = i32
        lib.daa_kv_append_q4.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, _Dims, vp]
        lib.daa_kv_dequant_q4.restype = i32
        lib.daa_kv_dequant_q4.argtypes = [vp, vp, vp, i32, vp, _Dims, vp]
        lib.daa_batch_attention_q4_workspace_size.restype = sz
        lib.daa_batch_attention_q4_workspace_size.argtypes = [vp, vp, vp, i32, _Dims, ctypes.POINTER(i32)]
        lib.daa_batch_attention_q4_plan.restype = i32
        lib.daa_batch_attention_q4_plan.argtypes = [vp, vp, vp, i32, _Dims, vp, sz, pinfo, vp]
        lib.daa_batch_attention_q4_run.restype = i32
        lib.daa_batch_attention_q4_run.argtypes = [vp, vp, vp, vp, pinfo, i32, f32, vp, vp, vp, sz, _Dims, vp]
        lib.daa_rope_init.restype = i32
        lib.daa_rope_init.argtypes = [vp, i32, i32, i32, vp, ctypes.c_double]
        lib.daa_apply_rope.restype = i32
        lib.daa_apply_rope.argtypes = [vp, vp, i32, i32, vp]
        lib.daa_append_rope.restype = i32
        lib.daa_append_rope.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, _Dims, vp]
        lib.daa_append_rope_q4.restype = i32
        lib.daa_append_rope_q4.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, _Dims, vp]
        lib.daa_set_prefill_append_fusion.restype = i32
        lib.daa_set_prefill_append_fusion.argtypes = [i32]
        lib.daa_prefill_append_fusion.restype = i32
        lib.daa_prefill_append_fusion.argtypes = []
        lib.daa_selftest_bounded_wait.restype = i32
        lib.daa_selftest_bounded_wait.argtypes = [ctypes.POINTER(i32)]
        lib.daa_device_error.restype = i32
        lib.daa_device_error.argtypes = [ctypes.POINTER(i32), i32]
        lib.daa_trace_enable.restype = i32
        lib.daa_trace_enable.argtypes = [i32]
        lib.daa_trace_disable.restype = i32
        lib.daa_trace_read.restype = i32
        lib.daa_trace_read.argtypes = [ctypes.POINTER(i32), ctypes.POINTER(f32), i32]
        _lib = lib
        return lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return ctypes.c_void_p(t.data_ptr())
    if isinstance(t, np.ndarray):
        return t.ctypes.data_as(ctypes.c_void_p)
    raise TypeError(type(t))


def _host_i32(a) -> np.ndarray:
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _dev_i32(t: torch.Tensor, name: str) -> torch.Tensor:
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.int32 and t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous int32 CUDA tensor")
    return t


def _dev_bf16(t: torch.Tensor, name: str) -> torch.Tensor:
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous bf16 CUDA tensor")
    return t


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _addr(t, name: str, dtype, dev: int) -> int:
    """The address of a contiguous tensor of `dtype` on CUDA device `dev`.  A few
    attribute reads: these checks are most of what a small call costs the host."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous {str(dtype).removeprefix('torch.')} CUDA tensor")
    raise ValueError(f"{name} must be on cuda:{dev}")


def _call(fn, what, dev: int, stream, *args):
    """fn(*args, stream) with device `dev` current; raises on an error status."""
    if stream is None:
        stream = _raw_stream(dev)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    else:
        stream = int(stream)
    if _current_device() == dev:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != DAA_OK:
        raise DaaError(st, what)


def _raw_stream(dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev)


def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _torch_stream(stream, dev: int):
    """A call's stream on CUDA device `dev` as torch's: a stream of torch's, or a
    cudaStream_t, alone or as an object's ``cuda_stream`` (0 and 1 are the handles of
    the default stream)."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return torch.cuda.default_stream(dev) if raw in (0, 1) else torch.cuda.ExternalStream(raw, device=dev)


def _use_stream(stream, dev: int):
    """torch's own work of a call on the stream that the call names."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(_torch_stream(stream, dev))


class _StreamUse:
    """Memory that torch allocated on one stream and calls use on others.  The
    first call on another stream waits for the allocating one, where the memory may
    still be in use as what it was before; and memory freed while a call is under
    way is not given away before that call has ended.  A stream of torch's is
    recorded with the allocator.  One of the caller's may be gone by the time the
    memory is freed: an event after each call stands for it, and the allocating
    stream waits for that.  Captured calls run when their graph is replayed: whoever
    replays it keeps the memory and the order."""

    def __init__(self, dev: int, *tensors):
        self.dev, self.tensors = dev, tensors
        self.home = torch.cuda.current_stream(dev) if dev >= 0 else None
        self.known, self.events = {self.home.cuda_stream if self.home else None}, {}

    def begin(self, stream):
        """Before a call on ``stream``; what it returns goes to ``end`` after it."""
        if self.home is None:  # host memory: the call itself will refuse it
            return None
        if stream is None:
            raw = _raw_stream(self.dev)
        else:
            raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if raw in self.known:
            return None
        s = torch.cuda.current_stream(self.dev) if stream is None else _torch_stream(stream, self.dev)
        if _capturing(s):
            return None
        if raw not in self.events:
            if not _capturing(self.home):  # s would become part of that capture
                s.wait_stream(self.home)
            if s.cuda_stream == 0 or s.stream_id != s.cuda_stream:  # not the caller's: those go by their handle
                for t in self.tensors:
                    t.record_stream(s)
                self.known.add(raw)
                return None
            if not self.events:
                weakref.finalize(self, _give_back, self.home, self.events, self.tensors).atexit = False
            self.events[raw] = torch.cuda.Event()
        return self.events[raw], s

    def end(self, used):
        if used is not None:
            used[0].record(used[1])


def _capturing(stream) -> bool:
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


_late: list = []  # memory dropped while its stream was being captured, which cannot wait then


def _give_back(stream, events, tensors):
    _late.append((stream, events, tensors))
    held, _late[:] = _late[:], []
    for item in held:
        if _capturing(item[0]):
            _late.append(item)
            continue
        for e in item[1].values():
            item[0].wait_event(e)


def _dims(kv_pages: torch.Tensor, num_qo_heads: int) -> _Dims:
    if kv_pages.dim() != 5 or kv_pages.shape[1] != 2:
        raise ValueError("kv_pages must be [num_pages, 2, Hkv, page_size, head_dim]")
    n, _, hkv, p, d = kv_pages.shape
    return _Dims(num_qo_heads, hkv, d, p, n)


def _check(st: int, what: str):
    if st != DAA_OK:
        raise DaaError(st, what)


def kv_append(k_new, v_new, kv_pages, append_indptr, page_indices, kv_indptr, last_page_len,
              stream=None) -> None:
    """Append new tokens' K/V into their pages (asynchronous on ``stream``)."""
    lib = load_library()
    _dev_bf16(k_new, "k_new"), _dev_bf16(v_new, "v_new"), _dev_bf16(kv_pages, "kv_pages")
    for n, t in (("append_indptr", append_indptr), ("page_indices", page_indices),
                 ("kv_indptr", kv_indptr), ("last_page_len", last_page_len)):
        _dev_i32(t, n)
    dims = _dims(kv_pages, kv_pages.shape[2])
    batch = append_indptr.numel() - 1
    _check(lib.daa_kv_append(_ptr(k_new), _ptr(v_new), _ptr(kv_pages), _ptr(append_indptr),
                             _ptr(page_indices), _ptr(kv_indptr), _ptr(last_page_len), batch,
                             k_new.shape[0], dims, _stream(stream)), "kv_append")


def batch_attention_workspace_size(h_qo_indptr, h_kv_indptr, h_last_page_len, num_qo_heads,
                                   num_kv_heads, head_dim, page_size, num_pages) -> int:
    lib = load_library()
    qo, kv, ll = _host_i32(h_qo_indptr), _host_i32(h_kv_indptr), _host_i32(h_last_page_len)
    st = ctypes.c_int32(0)
    n = lib.daa_batch_attention_workspace_size(_ptr(qo), _ptr(kv), _ptr(ll), len(qo) - 1,
                                               _Dims(num_qo_heads, num_kv_heads, head_dim,
                                                     page_size, num_pages), ctypes.byref(st))
    _check(st.value, "batch_attention_workspace_size")
    return int(n)


def _host_groups(prefix_groups):
    """(indptr, prefix_len) -> host int32 arrays and the group count."""
    ind, pl = (_host_i32(x) for x in prefix_groups)
    if len(ind) != len(pl) + 1:
        raise ValueError("prefix_groups: indptr must have one more entry than prefix_len")
    return ind, pl, len(pl)


def shared_prefix_workspace_size(h_qo_indptr, h_kv_indptr, h_last_page_len, prefix_groups,
                                 num_qo_heads, num_kv_heads, head_dim, page_size,
                                 num_pages) -> int:
    """Workspace bytes of ``batch_attention(..., prefix_groups=...)`` (and of
    ``append_attention`` with the same groups)."""
    lib = load_library()
    qo, kv, ll = _host_i32(h_qo_indptr), _host_i32(h_kv_indptr), _host_i32(h_last_page_len)
    gi, gl, ng = _host_groups(prefix_groups)
    st = ctypes.c_int32(0)
    n = lib.daa_batch_attention_shared_prefix_workspace_size(
        _ptr(qo), _ptr(kv), _ptr(ll), len(qo) - 1, _ptr(gi), _ptr(gl), ng,
        _Dims(num_qo_heads, num_kv_heads, head_dim, page_size, num_pages), ctypes.byref(st))
    _check(st.value, "shared_prefix_workspace_size")
    return int(n)


def _workspace_need(lib, hq, hk, hl, dims, groups, what):
    st = ctypes.c_int32(0)
    if groups is None:
        need = lib.daa_batch_attention_workspace_size(_ptr(hq), _ptr(hk), _ptr(hl), len(hq) - 1,
                                                      dims, ctypes.byref(st))
    else:
        gi, gl, ng = groups
        need = lib.daa_batch_attention_shared_prefix_workspace_size(
            _ptr(hq), _ptr(hk), _ptr(hl), len(hq) - 1, _ptr(gi), _ptr(gl), ng, dims,
            ctypes.byref(st))
    _check(st.value, what)
    return int(need)


def batch_attention(q, kv_pages, qo_indptr, kv_indptr, page_indices, last_page_len, causal=True,
                    sm_scale=None, out=None, lse=None, workspace=None, host_indptr=None,
                    stream=None, prefix_groups=None):
    """Mixed-batch paged attention.  Returns ``out`` (and fills ``lse`` if given).

    ``host_indptr`` = (h_qo_indptr, h_kv_indptr, h_last_page_len) host copies of
    the page table used for planning; when omitted they are copied from the
    device on the call's stream (a synchronisation).  ``workspace`` (uint8 CUDA tensor) is allocated
    by torch here when omitted, like ``out`` for the call's stream; the library
    itself never allocates.

    ``prefix_groups`` = (indptr, prefix_len), host int arrays: group i is
    requests [indptr[i], indptr[i+1]) whose first prefix_len[i] keys sit in the
    same pages (a shared cached prefix).  The shared keys are then attended
    once for all the group's rows (``daa_batch_attention_shared_prefix``); the
    result is the same.
    """
    lib = load_library()
    _dev_bf16(q, "q"), _dev_bf16(kv_pages, "kv_pages")
    for n, t in (("qo_indptr", qo_indptr), ("kv_indptr", kv_indptr), ("page_indices", page_indices),
                 ("last_page_len", last_page_len)):
        _dev_i32(t, n)
    Hq, d = q.shape[1], q.shape[2]
    dims = _dims(kv_pages, Hq)
    if sm_scale is None:
        sm_scale = 1.0 / float(d) ** 0.5
    if host_indptr is None:
        host_indptr = (qo_indptr, kv_indptr, last_page_len)
    with _use_stream(stream, q.get_device()):
        hq, hk, hl = (_host_i32(x) for x in host_indptr)
    batch = len(hq) - 1
    if out is None:
        with _use_stream(stream, q.get_device()):
            out = torch.empty_like(q)
    _dev_bf16(out, "out")
    if lse is not None and not (lse.is_cuda and lse.dtype == torch.float32 and lse.is_contiguous()):
        raise TypeError("lse must be a contiguous fp32 CUDA tensor")
    groups = None if prefix_groups is None else _host_groups(prefix_groups)
    need = _workspace_need(lib, hq, hk, hl, dims, groups, "batch_attention")
    if workspace is None and need > 0:
        with _use_stream(stream, q.get_device()):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if groups is None:
        st = lib.daa_batch_attention(_ptr(q), _ptr(kv_pages), _ptr(qo_indptr), _ptr(kv_indptr),
                                     _ptr(page_indices), _ptr(last_page_len), _ptr(hq), _ptr(hk),
                                     _ptr(hl), batch, int(bool(causal)), float(sm_scale), _ptr(out),
                                     _ptr(lse), _ptr(workspace), ws_bytes, dims, _stream(stream))
    else:
        gi, gl, ng = groups
        st = lib.daa_batch_attention_shared_prefix(
            _ptr(q), _ptr(kv_pages), _ptr(qo_indptr), _ptr(kv_indptr), _ptr(page_indices),
            _ptr(last_page_len), _ptr(hq), _ptr(hk), _ptr(hl), batch, _ptr(gi), _ptr(gl), ng,
            int(bool(causal)), float(sm_scale), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
            dims, _stream(stream))
    _check(st, "batch_attention")
    return out


def batch_attention_tree(q, kv_pages, qo_indptr, kv_indptr, page_indices, last_page_len, tree_mask,
                         sm_scale=None, out=None, lse=None, workspace=None, host_indptr=None,
                         stream=None):
    """Causal mixed-batch attention in which new token i of a request sees,
    among its request's new tokens, itself and the earlier ones selected by
    its mask row (for a draft tree numbered parents-first: its ancestors).

    ``tree_mask``: contiguous int32 or uint32 CUDA tensor [nnz_qo, words], one
    row per query row; bit t (word t // 32, bit t % 32) selects new token t.
    Every request needs qo_len <= 32 * words.  Other arguments as
    ``batch_attention``."""
    lib = load_library()
    _dev_bf16(q, "q"), _dev_bf16(kv_pages, "kv_pages")
    for n, t in (("qo_indptr", qo_indptr), ("kv_indptr", kv_indptr), ("page_indices", page_indices),
                 ("last_page_len", last_page_len)):
        _dev_i32(t, n)
    if not (isinstance(tree_mask, torch.Tensor) and tree_mask.is_cuda and tree_mask.dim() == 2
            and tree_mask.element_size() == 4 and tree_mask.is_contiguous()
            and not tree_mask.is_floating_point() and tree_mask.shape[0] == q.shape[0]):
        raise TypeError("tree_mask must be a contiguous [nnz_qo, words] int32/uint32 CUDA tensor")
    Hq, d = q.shape[1], q.shape[2]
    dims = _dims(kv_pages, Hq)
    if sm_scale is None:
        sm_scale = 1.0 / float(d) ** 0.5
    if host_indptr is None:
        host_indptr = (qo_indptr, kv_indptr, last_page_len)
    with _use_stream(stream, q.get_device()):
        hq, hk, hl = (_host_i32(x) for x in host_indptr)
    batch = len(hq) - 1
    if out is None:
        with _use_stream(stream, q.get_device()):
            out = torch.empty_like(q)
    _dev_bf16(out, "out")
    if lse is not None and not (lse.is_cuda and lse.dtype == torch.float32 and lse.is_contiguous()):
        raise TypeError("lse must be a contiguous fp32 CUDA tensor")
    if workspace is None:
        st = ctypes.c_int32(0)
        need = lib.daa_batch_attention_workspace_size(_ptr(hq), _ptr(hk), _ptr(hl), batch, dims,
                                                      ctypes.byref(st))
        _check(st.value, "batch_attention_tree")
        if need > 0:
            with _use_stream(stream, q.get_device()):
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.daa_batch_attention_tree(_ptr(q), _ptr(kv_pages), _ptr(qo_indptr), _ptr(kv_indptr),
                                        _ptr(page_indices), _ptr(last_page_len), _ptr(hq), _ptr(hk),
                                        _ptr(hl), batch, _ptr(tree_mask), int(tree_mask.shape[1]),
                                        float(sm_scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                        ws_bytes, dims, _stream(stream)),
           "batch_attention_tree")
    return out


def append_attention(k_new, v_new, q, kv_pages, qo_indptr, kv_indptr, page_indices, last_page_len,
                     causal=True, sm_scale=None, out=None, lse=None, workspace=None,
                     host_indptr=None, stream=None, prefix_groups=None):
    """``kv_append`` of this step's new K/V (rows laid out like ``q``) followed
    by ``batch_attention``, in one call: same results, with the attention
    kernels launched behind the append so that the work that does not read the
    appended rows overlaps it.  Arguments as ``batch_attention`` (including
    ``prefix_groups``)."""
    lib = load_library()
    _dev_bf16(k_new, "k_new"), _dev_bf16(v_new, "v_new")
    _dev_bf16(q, "q"), _dev_bf16(kv_pages, "kv_pages")
    for n, t in (("qo_indptr", qo_indptr), ("kv_indptr", kv_indptr), ("page_indices", page_indices),
                 ("last_page_len", last_page_len)):
        _dev_i32(t, n)
    Hq, d = q.shape[1], q.shape[2]
    dims = _dims(kv_pages, Hq)
    if k_new.shape != (q.shape[0], dims.num_kv_heads, d) or v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must be [nnz_qo, Hkv, head_dim]")
    if sm_scale is None:
        sm_scale = 1.0 / float(d) ** 0.5
    if host_indptr is None:
        host_indptr = (qo_indptr, kv_indptr, last_page_len)
    with _use_stream(stream, q.get_device()):
        hq, hk, hl = (_host_i32(x) for x in host_indptr)
    batch = len(hq) - 1
    if out is None:
        with _use_stream(stream, q.get_device()):
            out = torch.empty_like(q)
    _dev_bf16(out, "out")
    if lse is not None and not (lse.is_cuda and lse.dtype == torch.float32 and lse.is_contiguous()):
        raise TypeError("lse must be a contiguous fp32 CUDA tensor")
    groups = None if prefix_groups is None else _host_groups(prefix_groups)
    if workspace is None:
        need = _workspace_need(lib, hq, hk, hl, dims, groups, "append_attention")
        if need > 0:
            with _use_stream(stream, q.get_device()):
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if groups is None:
        st = lib.daa_append_attention(_ptr(k_new), _ptr(v_new), _ptr(q), _ptr(kv_pages),
                                      _ptr(qo_indptr), _ptr(kv_indptr), _ptr(page_indices),
                                      _ptr(last_page_len), _ptr(hq), _ptr(hk), _ptr(hl), batch,
                                      int(bool(causal)), float(sm_scale), _ptr(out), _ptr(lse),
                                      _ptr(workspace), ws_bytes, dims, _stream(stream))
    else:
        gi, gl, ng = groups
        st = lib.daa_append_attention_shared_prefix(
            _ptr(k_new), _ptr(v_new), _ptr(q), _ptr(kv_pages), _ptr(qo_indptr), _ptr(kv_indptr),
            _ptr(page_indices), _ptr(last_page_len), _ptr(hq), _ptr(hk), _ptr(hl), batch,
            _ptr(gi), _ptr(gl), ng, int(bool(causal)), float(sm_scale), _ptr(out), _ptr(lse),
            _ptr(workspace), ws_bytes, dims, _stream(stream))
    _check(st, "append_attention")
    return out


def batch_attention_noalloc(q, kv_pages, qo_indptr, kv_indptr, page_indices, last_page_len,
                            host_indptr, causal=True, sm_scale=None, out=None, lse=None,
                            stream=None):
    """``batch_attention`` without a workspace: the library's fixed device
    scratch array is used instead (see daa_batch_attention_noalloc in daa.h for
    its size limit and for why calls must not overlap on the GPU)."""
    lib = load_library()
    _dev_bf16(q, "q"), _dev_bf16(kv_pages, "kv_pages")
    for n, t in (("qo_indptr", qo_indptr), ("kv_indptr", kv_indptr), ("page_indices", page_indices),
                 ("last_page_len", last_page_len)):
        _dev_i32(t, n)
    if q.dim() != 3:
        raise ValueError("q must be [nnz_qo, Hq, head_dim]")
    Hq, d = q.shape[1], q.shape[2]
    dims = _dims(kv_pages, Hq)
    if sm_scale is None:
        sm_scale = 1.0 / float(d) ** 0.5
    hq, hk, hl = (_host_i32(x) for x in host_indptr)
    if out is None:
        with _use_stream(stream, q.get_device()):
            out = torch.empty_like(q)
    _dev_bf16(out, "out")
    if out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    if lse is not None:
        if not (isinstance(lse, torch.Tensor) and lse.is_cuda and lse.dtype == torch.float32
                and lse.is_contiguous()):
            raise TypeError("lse must be a contiguous fp32 CUDA tensor")
        if tuple(lse.shape) != (q.shape[0], Hq):
            raise ValueError("lse must be [nnz_qo, Hq]")
    _check(lib.daa_batch_attention_noalloc(_ptr(q), _ptr(kv_pages), _ptr(qo_indptr), _ptr(kv_indptr),
                                           _ptr(page_indices), _ptr(last_page_len), _ptr(hq), _ptr(hk),
                                           _ptr(hl), len(hq) - 1, int(bool(causal)), float(sm_scale),
                                           _ptr(out), _ptr(lse), dims, _stream(stream)),
           "batch_attention_noalloc")
    return out


def batch_attention_plan(h_qo_indptr, h_kv_indptr, h_last_page_len, num_qo_heads, kv_pages,
                         workspace, prefix_groups=None, stream=None) -> PlanInfo:
    """Plan a batch once (host) and copy the plan into ``workspace``; the
    returned record is what ``batch_attention_run`` / ``append_attention_run``
    take.  ``workspace`` must hold at least the size query's bytes (with the
    same ``prefix_groups``)."""
    lib = load_library()
    _dev_bf16(kv_pages, "kv_pages")
    hq, hk, hl = (_host_i32(x) for x in (h_qo_indptr, h_kv_indptr, h_last_page_len))
    gi, gl, ng = _host_groups(prefix_groups) if prefix_groups is not None else (None, None, 0)
    dims = _dims(kv_pages, num_qo_heads)
    info = PlanInfo()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.daa_batch_attention_plan(_ptr(hq), _ptr(hk), _ptr(hl), len(hq) - 1, _ptr(gi), _ptr(gl),
                                        ng, dims, _ptr(workspace), ws_bytes, ctypes.byref(info),
                                        _stream(stream)), "batch_attention_plan")
    return info


def _run_args(q, kv_pages, qo_indptr, kv_indptr, page_indices, last_page_len, out, lse, stream):
    _dev_bf16(q, "q"), _dev_bf16(kv_pages, "kv_pages")
    for n, t in (("qo_indptr", qo_indptr), ("kv_indptr", kv_indptr), ("page_indices", page_indices),
                 ("last_page_len", last_page_len)):
        _dev_i32(t, n)
    if out is None:
        with _use_stream(stream, q.get_device()):
            out = torch.empty_like(q)
    _dev_bf16(out, "out")
    if lse is not None and not (lse.is_cuda and lse.dtype == torch.float32 and lse.is_contiguous()):
        raise TypeError("lse must be a contiguous fp32 CUDA tensor")
    return out


def batch_attention_run(q, kv_pages, qo_indptr, kv_indptr, page_indices, last_page_len, info,
                        workspace, causal=True, sm_scale=None, out=None, lse=None, stream=None):
    """Attention on a plan made by ``batch_attention_plan`` (kernels only)."""
    lib = load_library()
    out = _run_args(q, kv_pages, qo_indptr, kv_indptr, page_indices, last_page_len, out, lse, stream)
    if sm_scale is None:
        sm_scale = 1.0 / float(q.shape[2]) ** 0.5
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.daa_batch_attention_run(_ptr(q), _ptr(kv_pages), _ptr(qo_indptr), _ptr(kv_indptr),
                                       _ptr(page_indices), _ptr(last_page_len), ctypes.byref(info),
                                       int(bool(causal)), float(sm_scale), _ptr(out), _ptr(lse),
                                       _ptr(workspace), ws_bytes, _dims(kv_pages, q.shape[1]),
                                       _stream(stream)), "batch_attention_run")
    return out


def append_attention_run(k_new, v_new, q, kv_pages, qo_indptr, kv_indptr, page_indices,
                         last_page_len, info, workspace, causal=True, sm_scale=None, out=None,
                         lse=None, stream=None):
    """``append_attention`` on a plan made by ``batch_attention_plan``."""
    lib = load_library()
    _dev_bf16(k_new, "k_new"), _dev_bf16(v_new, "v_new")
    out = _run_args(q, kv_pages, qo_indptr, kv_indptr, page_indices, last_page_len, out, lse, stream)
    if sm_scale is None:
        sm_scale = 1.0 / float(q.shape[2]) ** 0.5
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.daa_append_attention_run(_ptr(k_new), _ptr(v_new), _ptr(q), _ptr(kv_pages),
                                        _ptr(qo_indptr), _ptr(kv_indptr), _ptr(page_indices),
                                        _ptr(last_page_len), ctypes.byref(info), int(bool(causal)),
                                        float(sm_scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                        ws_bytes, _dims(kv_pages, q.shape[1]), _stream(stream)),
           "append_attention_run")
    return out


@dataclass
class PageTable:
    """Device int32 CSR page table plus its host mirror (numpy).  A table built
    by ``PagePool.step`` also has its new tokens' places in the pool
    (``slot_map``, int64) and their positions (int32)."""
    qo_indptr: torch.Tensor
    kv_indptr: torch.Tensor
    page_indices: torch.Tensor
    last_page_len: torch.Tensor
    h_qo_indptr: np.ndarray
    h_kv_indptr: np.ndarray
    h_last_page_len: np.ndarray
    slot_map: torch.Tensor | None = None
    positions: torch.Tensor | None = None

    @classmethod
    def from_host(cls, qo_indptr, kv_indptr, page_indices, last_page_len, device="cuda"):
        hq, hk, hp, hl = (_host_i32(x) for x in (qo_indptr, kv_indptr, page_indices, last_page_len))
        dev = lambda a: torch.from_numpy(a).to(device)  # noqa: E731
        return cls(dev(hq), dev(hk), dev(hp), dev(hl), hq, hk, hl)


class BatchAttention:
    """Plan-once / run-many wrapper for one batch shape (FlashInfer-style).  Calls of
    one object share its workspace and must be ordered on the GPU.  The object may be
    dropped while one is under way; a graph that holds one needs it until its last
    replay has ended."""

    def __init__(self, table: PageTable, num_qo_heads: int, kv_pages: torch.Tensor, causal=True,
                 sm_scale=None, prefix_groups=None):
        self.t = table
        self.kv_pages = kv_pages
        self.causal = causal
        self.Hq = num_qo_heads
        self.sm_scale = sm_scale if sm_scale is not None else 1.0 / float(kv_pages.shape[4]) ** 0.5
        self.prefix_groups = prefix_groups
        n, _, hkv, p, d = kv_pages.shape
        if prefix_groups is None:
            need = batch_attention_workspace_size(table.h_qo_indptr, table.h_kv_indptr,
                                                  table.h_last_page_len, num_qo_heads, hkv, d, p, n)
        else:
            need = shared_prefix_workspace_size(table.h_qo_indptr, table.h_kv_indptr,
                                                table.h_last_page_len, prefix_groups,
                                                num_qo_heads, hkv, d, p, n)
        self.workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=kv_pages.device)
        self._use = _StreamUse(self.workspace.get_device(), self.workspace)
        self.info = None  # set by plan(): run() and step() then launch the kernels only

    def plan(self, stream=None):
        """Upload the batch's plan once; later run() / step() calls (e.g. one per
        layer) reuse it until the next plan() or a tree-mask run."""
        t = self.t
        used = self._use.begin(stream)
        try:
            self.info = batch_attention_plan(t.h_qo_indptr, t.h_kv_indptr, t.h_last_page_len, self.Hq,
                                             self.kv_pages, self.workspace,
                                             prefix_groups=self.prefix_groups, stream=stream)
        finally:
            self._use.end(used)
        return self.info

    def append(self, k_new, v_new, stream=None):
        t = self.t
        kv_append(k_new, v_new, self.kv_pages, t.qo_indptr, t.page_indices, t.kv_indptr,
                  t.last_page_len, stream=stream)

    def append_rope(self, q, k_new, v_new, rope, positions=None, q_out=None, q_norm=None, k_norm=None, eps=1e-6,
                    stream=None):
        """``append_rope`` on this table and pool; returns the rotated q for ``run``."""
        t = self.t
        return append_rope(q, k_new, v_new, self.kv_pages, t.qo_indptr, t.page_indices, t.kv_indptr, t.last_page_len,
                           rope, positions, q_out, q_norm, k_norm, eps, stream)

    def step_rope(self, q, k_new, v_new, rope, positions=None, q_norm=None, k_norm=None, eps=1e-6, out=None, lse=None,
                  stream=None, tree_mask=None):
        """append_rope, then run: a step on the projections' rows as they are."""
        q = self.append_rope(q, k_new, v_new, rope, positions, None, q_norm, k_norm, eps, stream)
        return self.run(q, out=out, lse=lse, stream=stream, tree_mask=tree_mask)

    def step(self, k_new, v_new, q, out=None, lse=None, stream=None):
        """append + run in one call (``append_attention``, or ``append_attention_run``
        on the stored plan)."""
        used = self._use.begin(stream)
        try:
            return self._step(k_new, v_new, q, out, lse, stream)
        finally:
            self._use.end(used)

    def _step(self, k_new, v_new, q, out, lse, stream):
        t = self.t
        if self.info is not None:
            return append_attention_run(k_new, v_new, q, self.kv_pages, t.qo_indptr, t.kv_indptr,
                                        t.page_indices, t.last_page_len, self.info, self.workspace,
                                        self.causal, self.sm_scale, out=out, lse=lse, stream=stream)
        return append_attention(k_new, v_new, q, self.kv_pages, t.qo_indptr, t.kv_indptr,
                                t.page_indices, t.last_page_len, self.causal, self.sm_scale,
                                out=out, lse=lse, workspace=self.workspace,
                                host_indptr=(t.h_qo_indptr, t.h_kv_indptr, t.h_last_page_len),
                                stream=stream, prefix_groups=self.prefix_groups)

    def run(self, q, out=None, lse=None, stream=None, tree_mask=None):
        """Attention over the batch; with ``tree_mask``, under draft-tree masks
        (``batch_attention_tree``; the batch must be causal)."""
        used = self._use.begin(stream)
        try:
            return self._run(q, out, lse, stream, tree_mask)
        finally:
            self._use.end(used)

    def _run(self, q, out, lse, stream, tree_mask):
        t = self.t
        if tree_mask is None and self.info is not None:
            return batch_attention_run(q, self.kv_pages, t.qo_indptr, t.kv_indptr, t.page_indices,
                                       t.last_page_len, self.info, self.workspace, self.causal,
                                       self.sm_scale, out=out, lse=lse, stream=stream)
        if tree_mask is not None:
            self.info = None  # the tree call plans into the workspace itself
            if self.prefix_groups is not None:
                raise ValueError("tree masks and prefix groups are not combined")
            if not self.causal:
                raise ValueError("a tree mask refines the causal rule")
            return batch_attention_tree(q, self.kv_pages, t.qo_indptr, t.kv_indptr, t.page_indices,
                                        t.last_page_len, tree_mask, self.sm_scale, out=out, lse=lse,
                                        workspace=self.workspace,
                                        host_indptr=(t.h_qo_indptr, t.h_kv_indptr,
                                                     t.h_last_page_len),
                                        stream=stream)
        return batch_attention(q, self.kv_pages, t.qo_indptr, t.kv_indptr, t.page_indices,
                               t.last_page_len, self.causal, self.sm_scale, out=out, lse=lse,
                               workspace=self.workspace,
                               host_indptr=(t.h_qo_indptr, t.h_kv_indptr, t.h_last_page_len),
                               stream=stream, prefix_groups=self.prefix_groups)


class HostStep:
    """Serving steps fed from pinned host memory, one library call each
    (``daa_append_attention_host``): upload the packed inputs, append +
    attention, read the output back.  Two sets of device buffers alternate, so
    step i + 1's upload and step i - 1's read-back overlap step i's kernels.

    ``sections``: the step's host tensors by name -- qo_indptr, kv_indptr,
    page_indices, last_page_len (int32) and q, k_new, v_new (bf16) -- packed
    once into one pinned buffer (``pack``; refill it with ``update``).  The
    page table must not change shape between steps (the workspace is sized for
    it).  ``step(i)`` enqueues step i on the current stream (compute) and two
    side streams; ``out(i)`` is step i's pinned output once ``done(i)`` has
    completed."""

    NAMES = ("qo_indptr", "kv_indptr", "page_indices", "last_page_len", "q", "k_new", "v_new")

    def __init__(self, sections, kv_pages, num_qo_heads, causal=True, sm_scale=None, workspace=None):
        lib = load_library()
        self.lib = lib
        dev = kv_pages.device
        self.kv_pages = kv_pages
        offs, at = {}, 0
        for n in self.NAMES:
            t = sections[n]
            offs[n] = at
            at += (t.numel() * t.element_size() + 255) // 256 * 256
        self.layout = StepLayout(*(offs[n] for n in self.NAMES), at)
        self.offsets = offs
        self.pack = torch.empty(at, dtype=torch.uint8, pin_memory=True)
        self.update(sections)
        hq, hk, hl = (sections[n].numpy() for n in ("qo_indptr", "kv_indptr", "last_page_len"))
        self.batch = len(hq) - 1
        q = sections["q"]
        self.dims = _dims(kv_pages, num_qo_heads)
        self.causal = int(bool(causal))
        self.sm_scale = float(sm_scale if sm_scale is not None else 1.0 / float(q.shape[2]) ** 0.5)
        if workspace is None:
            need = _workspace_need(lib, _host_i32(hq), _host_i32(hk), _host_i32(hl), self.dims, None,
                                   "HostStep")
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        self.workspace = workspace
        self.d_inputs = [torch.empty(at, dtype=torch.uint8, device=dev) for _ in range(2)]
        self.d_out = [torch.empty(q.shape, dtype=torch.bfloat16, device=dev) for _ in range(2)]
        self.h_out = [torch.empty(q.shape, dtype=torch.bfloat16, pin_memory=True) for _ in range(2)]
        self.up = torch.cuda.Stream(device=dev)
        self.down = torch.cuda.Stream(device=dev)
        self.events = [[torch.cuda.Event() for _ in range(3)] for _ in range(2)]
        cur = torch.cuda.current_stream(dev)
        for evs in self.events:  # events are created on first record
            for e in evs:
                e.record(cur)
        torch.cuda.synchronize(dev)
        self._args = []
        for k in range(2):
            up_ev, comp_ev, down_ev = (e.cuda_event for e in self.events[k])
            ss = StepStreams(self.up.cuda_stream, cur.cuda_stream, self.down.cuda_stream, up_ev, comp_ev,
                             down_ev, comp_ev, down_ev)
            self._args.append((ctypes.c_void_p(self.pack.data_ptr()),
                               ctypes.c_void_p(self.d_inputs[k].data_ptr()), ctypes.byref(self.layout),
                               self.batch, self.causal, ctypes.c_float(self.sm_scale),
                               ctypes.c_void_p(kv_pages.data_ptr()), ctypes.c_void_p(self.d_out[k].data_ptr()),
                               ctypes.c_void_p(self.h_out[k].data_ptr()),
                               ctypes.c_void_p(self.workspace.data_ptr()),
                               self.workspace.numel(), self.dims, ctypes.byref(ss), ss))
        self._stream = cur

    def update(self, sections):
        """Copy the step's host tensors into the pinned pack (wait for the
        previous step's ``uploaded`` event before calling this)."""
        for n in self.NAMES:
            t = sections[n].contiguous()
            nb = t.numel() * t.element_size()
            self.pack[self.offsets[n]:self.offsets[n] + nb].copy_(t.reshape(-1).view(torch.uint8))

    def step(self, i):
        """Enqueue step i (slot i % 2)."""
        a = self._args[i & 1]
        _check(self.lib.daa_append_attention_host(*a[:-1]), "append_attention_host")

    def done(self, i):
        """The event after which step i's output is in ``out(i)``."""
        return self.events[i & 1][2]

    def out(self, i):
        return self.h_out[i & 1]


class PagePool:
    """The pages of many requests, on the device: a block-table row of page ids
    per slot, a stack of free pages, and a kernel that builds a step's page table
    from lengths (``daa_step_table``).  The host keeps the lengths, never the page
    ids.

    ``step`` is the call of a serving loop: it checks the lengths on the host,
    raises before anything is launched when they do not fit, and returns a
    ``PageTable``.  ``build`` is the kernel alone, on device arrays.  Calls on one
    pool must be ordered on the GPU (one stream, or events between streams).  A pool
    may be dropped while a call on its arrays is under way, but not while a graph
    that holds one is still to be replayed."""

    PAGE_SIZE = 16

    def __init__(self, num_pages, num_slots, max_pages, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        # the lowest ids come off the stack first
        free = torch.arange(num_pages - 1, -1, -1, **i32)
        counters = torch.tensor([num_pages, 0], **i32)
        self._init(torch.zeros(num_slots, **i32), torch.zeros(num_slots, **i32),
                   torch.full((num_slots, max_pages), -1, **i32), free, counters)
        self._use = _StreamUse(self.dev, self.seq_len, self.held, self.block_table, free, counters)
        self.h_len, self.h_held, self.h_free = (np.zeros(num_slots, np.int64), np.zeros(num_slots, np.int64),
                                                int(num_pages))

    @classmethod
    def from_tensors(cls, seq_len, held, block_table, free_pages, counters):
        """A pool on the caller's tensors (see ``daa_page_pool``).  Its host
        copies of the lengths are read from the device by the first ``step``,
        ``set_lengths`` or ``release``, on that call's stream."""
        self = cls.__new__(cls)
        self._init(seq_len, held, block_table, free_pages, counters)
        self.h_len = self.h_held = self.h_free = None
        return self

    def _init(self, seq_len, held, block_table, free_pages, counters):
        tensors = (("seq_len", seq_len), ("held", held), ("block_table", block_table),
                   ("free_pages", free_pages), ("counters", counters))
        self.dev = seq_len.get_device() if isinstance(seq_len, torch.Tensor) else -1
        if self.dev < 0:
            raise TypeError("seq_len must be a contiguous int32 CUDA tensor")
        ptrs = [_addr(t, n, torch.int32, self.dev) for n, t in tensors]
        if seq_len.dim() != 1 or held.shape != seq_len.shape or block_table.dim() != 2 or \
                block_table.shape[0] != seq_len.shape[0] or free_pages.dim() != 1 or counters.shape != (2,):
            raise ValueError("a pool has seq_len [slots], held [slots], block_table [slots, max_pages], "
                             "free_pages [num_pages] and counters [2]")
        self.seq_len, self.held, self.block_table = seq_len, held, block_table
        self.free_pages, self.counters, self.device = free_pages, counters, seq_len.device
        self._pool = _Pool(*ptrs, seq_len.shape[0], block_table.shape[1], free_pages.shape[0], self.PAGE_SIZE)
        self._pool_ref = ctypes.byref(self._pool)
        self._use = None  # the caller's arrays: theirs to keep and to order

    def _mirror(self, stream):
        """The host copies, read once behind what the call's stream holds (it may be
        what fills the arrays)."""
        if self.h_len is None:
            with torch.cuda.device(self.dev), _use_stream(stream, self.dev):
                n, held, free = (x.cpu().numpy() for x in (self.seq_len, self.held, self.counters))
            self.h_len, self.h_held, self.h_free = n.astype(np.int64), held.astype(np.int64), int(free[0])

    def build(self, slots, new_len, qo_indptr, kv_indptr, page_indices, last_page_len, slot_map=None,
              positions=None, advance=False, stream=None):
        """``daa_step_table`` on device arrays: fills the given tensors (their
        sizes are the capacities) and takes the pages the step needs.  What the
        kernel refuses gives an empty step and sets the device error word.  The
        host copies of the lengths are not updated: a pool is driven either by
        ``build`` or by ``step``."""
        i32, dev = torch.int32, self.dev
        args = (_addr(slots, "slots", i32, dev), _addr(new_len, "new_len", i32, dev),
                _addr(qo_indptr, "qo_indptr", i32, dev), _addr(kv_indptr, "kv_indptr", i32, dev),
                _addr(page_indices, "page_indices", i32, dev), _addr(last_page_len, "last_page_len", i32, dev))
        batch = slots.numel()
        if new_len.numel() != batch or qo_indptr.numel() != batch + 1 or kv_indptr.numel() != batch + 1 \
                or last_page_len.numel() != batch:
            raise ValueError("slots, new_len and last_page_len have one entry per request, "
                             "qo_indptr and kv_indptr one more")
        rows, p_map, p_pos = 2 ** 31 - 1, None, None  # without either nothing is written per row
        if slot_map is not None:
            p_map, rows = _addr(slot_map, "slot_map", torch.int64, dev), slot_map.numel()
        if positions is not None:
            p_pos, rows = _addr(positions, "positions", i32, dev), min(rows, positions.numel())
        used = self._use and self._use.begin(stream)
        try:
            _call(load_library().daa_step_table, "step_table", dev, stream, self._pool_ref, args[0], args[1], batch,
                  1 if advance else 0, args[2], args[3], args[4], page_indices.numel(), args[5], p_map, p_pos, rows)
        finally:
            if used:
                self._use.end(used)

    def step(self, slots, new_lens, advance=True, stream=None) -> PageTable:
        """The page table of a step that brings ``new_lens[i]`` tokens to slot
        ``slots[i]`` (host sequences).  With ``advance`` the lengths grow by them;
        otherwise call ``set_lengths`` once it is known how many were kept."""
        self._mirror(stream)
        sl, nl = (np.asarray(x, np.int64).reshape(-1) for x in (slots, new_lens))
        self._check_slots(sl)
        if len(nl) != len(sl) or (nl < 0).any():
            raise ValueError("new_lens must have one entry >= 0 per slot")
        kv = self.h_len[sl] + nl
        pages = -(-kv // self.PAGE_SIZE)
        if len(kv) and pages.max() > self.block_table.shape[1]:
            raise DaaError(-2, "PagePool.step: a request is longer than its block-table row")
        take = int(np.maximum(pages - self.h_held[sl], 0).sum())
        if take > self.h_free:
            raise DaaError(-3, f"PagePool.step: {take} pages needed, {self.h_free} free")
        csr = lambda n: np.concatenate([[0], np.cumsum(n)])  # noqa: E731
        hq, hk = csr(nl), csr(pages)
        if max(hq[-1], hk[-1]) > 2 ** 31 - 1:
            raise DaaError(-2, "PagePool.step: the step's rows and pages must fit 32 bits")
        hl = np.where(pages > 0, kv - (pages - 1) * self.PAGE_SIZE, 0)
        i32 = dict(dtype=torch.int32, device=self.device)
        with torch.cuda.device(self.dev), _use_stream(stream, self.dev):
            up = torch.from_numpy(np.stack([sl, nl]).astype(np.int32)).to(self.device)
            n = len(sl)
            t = PageTable(torch.empty(n + 1, **i32), torch.empty(n + 1, **i32),
                          torch.empty(int(hk[-1]), **i32), torch.empty(n, **i32), _host_i32(hq),
                          _host_i32(hk), _host_i32(hl),
                          torch.empty(int(hq[-1]), dtype=torch.int64, device=self.device),
                          torch.empty(int(hq[-1]), **i32))
            self.build(up[0], up[1], t.qo_indptr, t.kv_indptr, t.page_indices, t.last_page_len,
                       t.slot_map, t.positions, advance, stream)
        self.h_held[sl] = np.maximum(self.h_held[sl], pages)
        self.h_free -= take
        if advance:
            self.h_len[sl] = kv
        return t

    def set_lengths(self, slots, lens, stream=None):
        """Set the cached lengths of slots (the tokens kept of a step that did
        not advance, or a request cut back).  Pages stay with their slots."""
        self._mirror(stream)
        sl, ln = (np.asarray(x, np.int64).reshape(-1) for x in (slots, lens))
        self._check_slots(sl)
        if len(ln) != len(sl) or (ln < 0).any() or (-(-ln // self.PAGE_SIZE) > self.h_held[sl]).any():
            raise ValueError("lens must have one entry per slot, within the pages the slot holds")
        with torch.cuda.device(self.dev), _use_stream(stream, self.dev):
            at = torch.from_numpy(sl).to(self.device)
            to = torch.from_numpy(ln.astype(np.int32)).to(self.device)
            used = self._use and self._use.begin(stream)
            try:
                self.seq_len.index_copy_(0, at, to)
            finally:
                if used:
                    self._use.end(used)
        self.h_len[sl] = ln

    def release(self, slots, stream=None):
        """Give the pages of slots back (``daa_release_pages``); their lengths become 0."""
        self._mirror(stream)
        sl = np.asarray(slots, np.int64).reshape(-1)
        self._check_slots(sl)
        with torch.cuda.device(self.dev), _use_stream(stream, self.dev):
            dev = torch.from_numpy(sl.astype(np.int32)).to(self.device)
            used = self._use and self._use.begin(stream)
            try:
                _call(load_library().daa_release_pages, "release_pages", self.dev, stream, self._pool_ref,
                      dev.data_ptr(), len(sl))
            finally:
                if used:
                    self._use.end(used)
        self.h_free += int(self.h_held[sl].sum())
        self.h_len[sl] = self.h_held[sl] = 0

    def _check_slots(self, sl):
        if len(sl) and (sl.min() < 0 or sl.max() >= len(self.h_len) or len(np.unique(sl)) < len(sl)):
            raise ValueError("slots must be distinct and within the pool")


def new_q4_pool(num_pages, num_kv_heads, head_dim, device="cuda") -> torch.Tensor:
    """An empty (zero) 4-bit page pool: uint8 [num_pages, Hkv, 2, 9 * head_dim]."""
    return torch.zeros(num_pages, num_kv_heads, 2, 9 * head_dim, dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=64)
def _q4_dims_of(shape, num_qo_heads) -> _Dims:
    if len(shape) != 4 or shape[2] != 2 or shape[3] % 9 != 0:
        raise ValueError("kv_pages must be [num_pages, Hkv, 2, 9 * head_dim]")
    n, hkv, _, b = shape
    return _Dims(hkv if num_qo_heads is None else num_qo_heads, hkv, b // 9, 16, n)


def _q4_pool(kv_pages, kv_exp, num_qo_heads=None):
    """(device index, pool address, exponents' address or None, dims) of a 4-bit pool."""
    dev = kv_pages.get_device() if isinstance(kv_pages, torch.Tensor) else -1
    pool = _addr(kv_pages, "kv_pages", torch.uint8, dev)
    if dev < 0:
        raise TypeError("kv_pages must be a contiguous uint8 CUDA tensor")
    dims = _q4_dims_of(kv_pages.shape, num_qo_heads)
    if kv_exp is None:
        return dev, pool, None, dims
    exp = _addr(kv_exp, "kv_exp", torch.int32, dev)
    if kv_exp.shape != (2, dims.num_kv_heads):
        raise ValueError("kv_exp must be [2, Hkv]")
    return dev, pool, exp, dims


def kv_append_q4(k_new, v_new, kv_pages, append_indptr, page_indices, kv_indptr, last_page_len,
                 kv_exp=None, stream=None) -> None:
    """``kv_append`` into a 4-bit pool: the new tokens' K/V are quantised (e2m1
    with an e4m3 scale for every 16 dims, and the head's exponent ``kv_exp``
    [2, Hkv]) and written into their page slots."""
    dev, pool, exp, dims = _q4_pool(kv_pages, kv_exp)
    i32, bf16 = torch.int32, torch.bfloat16
    k, v = _addr(k_new, "k_new", bf16, dev), _addr(v_new, "v_new", bf16, dev)
    table = (_addr(append_indptr, "append_indptr", i32, dev), _addr(page_indices, "page_indices", i32, dev),
             _addr(kv_indptr, "kv_indptr", i32, dev), _addr(last_page_len, "last_page_len", i32, dev))
    rows = k_new.shape[0] if k_new.dim() == 3 else 0
    if k_new.shape != (rows, dims.num_kv_heads, dims.head_dim) or v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must be [nnz_new, Hkv, head_dim]")
    batch = append_indptr.numel() - 1
    if kv_indptr.numel() != batch + 1 or last_page_len.numel() != batch:
        raise ValueError("append_indptr and kv_indptr have batch + 1 entries, last_page_len batch")
    _call(load_library().daa_kv_append_q4, "kv_append_q4", dev, stream, k, v, pool, exp, *table, batch, rows, dims)


def kv_dequant_q4(kv_pages, page_ids, kv_exp=None, out=None, stream=None):
    """Pages of a 4-bit pool as bf16 pages [n, 2, Hkv, 16, head_dim], exactly."""
    dev, pool, exp, dims = _q4_pool(kv_pages, kv_exp)
    ids, n = _addr(page_ids, "page_ids", torch.int32, dev), page_ids.numel()
    shape = (n, 2, dims.num_kv_heads, dims.page_size, dims.head_dim)
    if out is None:
        with _use_stream(stream, dev):
            out = torch.empty(shape, dtype=torch.bfloat16, device=kv_pages.device)
    o = _addr(out, "out", torch.bfloat16, dev)
    if out.shape != shape:
        raise ValueError("out must be [n_pages, 2, Hkv, 16, head_dim]")
    _call(load_library().daa_kv_dequant_q4, "kv_dequant_q4", dev, stream, pool, exp, ids, n, o, dims)
    return out


def batch_attention_q4_workspace_size(h_qo_indptr, h_kv_indptr, h_last_page_len, num_qo_heads,
                                      num_kv_heads, head_dim, page_size, num_pages) -> int:
    lib = load_library()
    qo, kv, ll = _host_i32(h_qo_indptr), _host_i32(h_kv_indptr), _host_i32(h_last_page_len)
    st = ctypes.c_int32(0)
    n = lib.daa_batch_attention_q4_workspace_size(_ptr(qo), _ptr(kv), _ptr(ll), len(qo) - 1,
                                                  _Dims(num_qo_heads, num_kv_heads, head_dim,
                                                        page_size, num_pages), ctypes.byref(st))
    _check(st.value, "batch_attention_q4_workspace_size")
    return int(n)


class BatchAttentionQ4:
    """``BatchAttention`` over a 4-bit pool (``new_q4_pool``): plan once from the
    table's host copies, then append, run or step on it.  ``run`` plans first when
    ``plan`` has not been called.  Runs of one object share its workspace and must
    be ordered on the GPU; append and run can be captured into a CUDA graph, plan
    cannot.  The object may be dropped while a run is under way; a graph that holds
    one needs it until its last replay has ended."""

    def __init__(self, table: PageTable, num_qo_heads: int, kv_pages: torch.Tensor, causal=True,
                 sm_scale=None, kv_exp=None):
        self.t = table
        self.kv_pages, self.kv_exp = kv_pages, kv_exp
        self.dev, _, _, self.dims = _q4_pool(kv_pages, kv_exp, num_qo_heads)
        for n in ("qo_indptr", "kv_indptr", "page_indices", "last_page_len"):
            _addr(getattr(table, n), n, torch.int32, self.dev)
        batch = len(table.h_qo_indptr) - 1
        if len(table.h_kv_indptr) != batch + 1 or len(table.h_last_page_len) != batch or \
                table.page_indices.numel() < int(table.h_kv_indptr[-1]):
            raise ValueError("the table's host arrays have batch + 1, batch + 1 and batch entries, and "
                             "page_indices has an entry for every page of them")
        self.causal = int(bool(causal))
        self.sm_scale = float(sm_scale if sm_scale is not None else 1.0 / float(self.dims.head_dim) ** 0.5)
        d = self.dims
        need = batch_attention_q4_workspace_size(table.h_qo_indptr, table.h_kv_indptr,
                                                 table.h_last_page_len, d.num_qo_heads, d.num_kv_heads,
                                                 d.head_dim, d.page_size, d.num_pages)
        self.shape = (int(table.h_qo_indptr[-1]), d.num_qo_heads, d.head_dim)
        self.workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=kv_pages.device)
        self._use = _StreamUse(self.dev, self.workspace)
        self.info = None

    def plan(self, stream=None):
        """Upload the batch's plan; later runs (one per layer) reuse it."""
        t, info = self.t, PlanInfo()
        used = self._use.begin(stream)
        try:
            _call(load_library().daa_batch_attention_q4_plan, "batch_attention_q4_plan", self.dev, stream,
                  _ptr(t.h_qo_indptr), _ptr(t.h_kv_indptr), _ptr(t.h_last_page_len), len(t.h_qo_indptr) - 1,
                  self.dims, self.workspace.data_ptr(), self.workspace.numel(), ctypes.byref(info))
        finally:
            self._use.end(used)
        self.info = info
        return info

    def append(self, k_new, v_new, stream=None):
        t = self.t
        kv_append_q4(k_new, v_new, self.kv_pages, t.qo_indptr, t.page_indices, t.kv_indptr,
                     t.last_page_len, kv_exp=self.kv_exp, stream=stream)

    def append_rope(self, q, k_new, v_new, rope, positions=None, q_out=None, q_norm=None, k_norm=None, eps=1e-6,
                    stream=None):
        """``append_rope_q4`` on this table and pool; returns the rotated q for ``run``."""
        t = self.t
        return append_rope_q4(q, k_new, v_new, self.kv_pages, t.qo_indptr, t.page_indices, t.kv_indptr,
                              t.last_page_len, rope, positions, self.kv_exp, q_out, q_norm, k_norm, eps, stream)

    def step_rope(self, q, k_new, v_new, rope, positions=None, q_norm=None, k_norm=None, eps=1e-6, out=None, lse=None,
                  stream=None):
        """append_rope, then run: a step on the projections' rows as they are."""
        q = self.append_rope(q, k_new, v_new, rope, positions, None, q_norm, k_norm, eps, stream)
        return self.run(q, out=out, lse=lse, stream=stream)

    def run(self, q, out=None, lse=None, stream=None):
        """Attention of q [nnz_qo, Hq, head_dim]; returns ``out`` and fills ``lse``."""
        d, dev, bf16 = self.dims, self.dev, torch.bfloat16
        pq = _addr(q, "q", bf16, dev)
        if q.shape != self.shape:
            raise ValueError("q must be [nnz_qo, Hq, head_dim] of the planned table")
        if out is None:
            with _use_stream(stream, dev):
                out = torch.empty_like(q)
        po = _addr(out, "out", bf16, dev)
        if out.shape != self.shape:
            raise ValueError("out must have the shape of q")
        pl = None
        if lse is not None:
            pl = _addr(lse, "lse", torch.float32, dev)
            if lse.shape != self.shape[:2]:
                raise ValueError("lse must be [nnz_qo, Hq]")
        if self.info is None:
            self.plan(stream)
        exp = None if self.kv_exp is None else self.kv_exp.data_ptr()
        used = self._use.begin(stream)
        try:
            _call(load_library().daa_batch_attention_q4_run, "batch_attention_q4", dev, stream, pq,
                  self.kv_pages.data_ptr(), exp, self.t.page_indices.data_ptr(), self.info, self.causal,
                  self.sm_scale, po, pl, self.workspace.data_ptr(), self.workspace.numel(), d)
        finally:
            self._use.end(used)
        return out

    def step(self, k_new, v_new, q, out=None, lse=None, stream=None):
        """append, then run."""
        self.append(k_new, v_new, stream)
        return self.run(q, out=out, lse=lse, stream=stream)


class Rope:
    """A rotation of heads by their tokens' positions (``daa_rope``): pair i of the
    first ``rotary_dim`` dims (all of ``head_dim`` without one; a multiple of 16) turns
    by position * ``frequencies[i]`` and is multiplied by ``magnitude``.  Pairs are dims
    (i, i + rotary_dim / 2), or (2i, 2i + 1) when ``interleaved``.  The frequencies are
    those of ``base`` and ``scaling`` (``rope_frequencies``), or given as
    ``frequencies`` (radians a token, rotary_dim / 2 of them).  Host data, fixed once it
    is made, for every device and layer."""

    def __init__(self, head_dim, base=10000.0, rotary_dim=None, interleaved=False, scaling=None, frequencies=None,
                 magnitude=None):
        self.head_dim = int(head_dim)
        self.rotary_dim = self.head_dim if rotary_dim is None else int(rotary_dim)
        self.interleaved = bool(interleaved)
        if frequencies is None:
            f, m = frequencies_of(self.rotary_dim, base, scaling)
        elif scaling is not None:
            raise ValueError("a scaling changes the base's frequencies: give one of scaling and frequencies")
        else:
            f, m = [float(x) for x in frequencies], 1.0
        if len(f) != self.rotary_dim // 2 or not all(map(math.isfinite, f)):
            raise ValueError("frequencies must be rotary_dim / 2 finite numbers")
        self._frequencies = array.array("d", f)
        self.magnitude = float(m if magnitude is None else magnitude)
        self._rope = _Rope()
        _check(load_library().daa_rope_init(ctypes.byref(self._rope), self.head_dim, self.rotary_dim,
                                            int(self.interleaved), self._frequencies.buffer_info()[0],
                                            self.magnitude), "Rope")

    @property
    def frequencies(self) -> np.ndarray:
        """Radians a token of each pair (a copy)."""
        return np.array(self._frequencies)


_native = None


def _load_native():
    """The module that hands tensors to the calls with rotation (built by ``build.build()``)."""
    global _native
    load_library()
    with _lock:
        if _native is None:
            path = os.path.join(_HERE, "_build", "_binding.so")
            if not os.path.exists(path):
                why = ""
                if os.path.exists(error := os.path.join(_HERE, "_build", "_binding.error")):
                    with open(error) as f:
                        why = f" (the last build of it: {f.read()})"
                raise ImportError(f"_binding.so not built at {path}; run decode_attention_append_gb300.build.build(){why}")
            spec = importlib.util.spec_from_file_location("_binding", path)
            mod = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(mod)
            _native = mod
    return _native


def _rows_like(x, name, stream):
    """New contiguous rows of the shape of x, for the call's stream."""
    if not (isinstance(x, torch.Tensor) and x.is_cuda):
        raise TypeError(f"{name} must be a bf16 CUDA tensor")
    with _use_stream(stream, x.get_device()):
        return torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)


def _handle(stream):
    return stream if stream is None else stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _rope_addr(rope):
    if not isinstance(rope, Rope):
        raise TypeError("rope must be a Rope")
    return ctypes.addressof(rope._rope)


def apply_rope(q, k, positions, rope, q_out=None, k_out=None, q_norm=None, k_norm=None, eps=1e-6, stream=None):
    """q [rows, Hq, head_dim] and k [rows, Hkv, head_dim] (or None) rotated by ``positions``
    (int32 [rows]): (q_out, k_out), new contiguous tensors unless given; q_out=q is in
    place.  Rows may have any strides of whole 16 bytes (views of a projection's
    output).  With ``q_norm`` / ``k_norm`` (bf16 [head_dim]) heads are divided by their root
    mean square (with ``eps``) and multiplied by these first.  No autograd: the
    gradients of the inputs are this call on those of the outputs at negated
    positions (without norms)."""
    if q_out is None:
        q_out = _rows_like(q, "q", stream)
    if k_out is None and k is not None:
        k_out = _rows_like(k, "k", stream)
    st = (_native or _load_native()).apply_rope(q, k, positions, _rope_addr(rope), q_out, k_out, q_norm, k_norm, eps,
                                                _handle(stream))
    if st != DAA_OK:
        raise DaaError(st, "apply_rope")
    return q_out, k_out


def append_rope(q, k_new, v_new, kv_pages, append_indptr, page_indices, kv_indptr, last_page_len, rope,
                positions=None, q_out=None, q_norm=None, k_norm=None, eps=1e-6, stream=None):
    """``kv_append`` of rotated keys: k_new [nnz_new, Hkv, head_dim] rotated and written with
    v_new into their page slots, and q [nnz_new, Hq, head_dim] (or None) rotated into
    ``q_out`` (a new contiguous tensor without one), which is returned.  A token's
    position is its place in its request; ``positions`` (int32 [nnz_new]) gives others,
    as the depths of draft trees.  Rows behind the last request (nnz_new more than
    append_indptr[batch]) are padding: nothing is written for them.  Strides, norms and
    in-place as ``apply_rope``."""
    if q_out is None and q is not None:
        q_out = _rows_like(q, "q", stream)
    st = (_native or _load_native()).append_rope(q, k_new, v_new, kv_pages, None, append_indptr, page_indices,
                                                 kv_indptr, last_page_len, _rope_addr(rope), positions, q_out, q_norm,
                                                 k_norm, eps, _handle(stream))
    if st != DAA_OK:
        raise DaaError(st, "append_rope")
    return q_out


def append_rope_q4(q, k_new, v_new, kv_pages, append_indptr, page_indices, kv_indptr, last_page_len, rope,
                   positions=None, kv_exp=None, q_out=None, q_norm=None, k_norm=None, eps=1e-6, stream=None):
    """``append_rope`` into a 4-bit pool: the rotated keys and v_new are quantised as
    ``kv_append_q4`` does.  These keys are rotated to the nearest fp32 value, and rounded
    to bf16 from that, so that a code does not hang on the order of fp32 operations."""
    if q_out is None and q is not None:
        q_out = _rows_like(q, "q", stream)
    st = (_native or _load_native()).append_rope_q4(q, k_new, v_new, kv_pages, kv_exp, append_indptr, page_indices,
                                                    kv_indptr, last_page_len, _rope_addr(rope), positions, q_out,
                                                    q_norm, k_norm, eps, _handle(stream))
    if st != DAA_OK:
        raise DaaError(st, "append_rope_q4")
    return q_out


def set_prefill_append_fusion(enable: bool) -> None:
    """Fused calls (``append_attention``, ``BatchAttention.step``): whether the
    prefill kernels read long chunks' own key tiles from k_new / v_new and write
    them into their pages themselves (True, the default) or the append kernel
    writes every row (False).  Results are identical."""
    _check(load_library().daa_set_prefill_append_fusion(int(bool(enable))),
           "set_prefill_append_fusion")


def prefill_append_fusion() -> bool:
    return bool(load_library().daa_prefill_append_fusion())


def device_error(reset: bool = True) -> int:
    """The library's device error word (0 = none); synchronises the device."""
    lib = load_library()
    code = ctypes.c_int32(0)
    _check(lib.daa_device_error(ctypes.byref(code), int(reset)), "device_error")
    return int(code.value)


def selftest_bounded_wait() -> bool:
    """Run the library's bounded wait on a barrier nothing completes; True when
    it gave up by its time limit (the device error word then holds 2)."""
    lib = load_library()
    flag = ctypes.c_int32(-1)
    _check(lib.daa_selftest_bounded_wait(ctypes.byref(flag)), "selftest_bounded_wait")
    return flag.value == 1


def trace_enable(capacity: int = 4096) -> None:
    _check(load_library().daa_trace_enable(capacity), "trace_enable")


def trace_disable() -> None:
    _check(load_library().daa_trace_disable(), "trace_disable")


def trace_read(max_records: int = 65536):
    """[(kernel name, milliseconds)] of the launches recorded since the last read."""
    lib = load_library()
    ids = (ctypes.c_int32 * max_records)()
    ms = (ctypes.c_float * max_records)()
    n = lib.daa_trace_read(ids, ms, max_records)
    return [(KERNEL_NAMES.get(ids[i], str(ids[i])), float(ms[i])) for i in range(n)]
