"""Exact causal grouped-query attention over paged K/V on GB300 (sm_103a).

Python binding of ``libatlas_attn.so`` (C ABI in ``include/*.h``).
This module only marshals arguments: it checks tensor shapes and dtypes,
allocates outputs and workspace with torch, and passes raw device pointers and
the current torch stream to the library.  Every step of the computation runs in
the library's CUDA kernels; there is no CPU or torch fallback, and the import
fails loudly when the library has not been built.

Functions (same names as the C entry points):
  decode(...)   one query row per sequence            -> atlas_attn_decode
  suffix(...)   the last q_len positions as queries   -> atlas_attn_suffix
  prefill(...)  causal self-attention of a prompt     -> atlas_attn_prefill
  cross(...)    decoder rows over an encoder's states -> atlas_attn_cross
  shared(...)   rows of sequences that share prefixes -> atlas_attn_shared
  kv_append(...)  new tokens' K/V into their pages    -> atlas_kv_append
  kv_append_rope(...)  the same, with rotary positions of several axes applied to the
                new keys and the step's queries       -> atlas_kv_append_rope
  kv_append_norm_rope(...)  that, after a norm of each head's queries and keys
                                                      -> atlas_kv_append_norm_rope
  kv_weights(...)  attention weight each cached key received -> atlas_kv_weights
  kv_select(...)   the keys that stay under a budget  -> atlas_kv_select
  kv_compact(...)  pages with only those keys left    -> atlas_kv_compact
  kv_resize(...)   page tables and slots from the sequences' lengths -> atlas_kv_resize
  workspace_size(kind, ...)                            -> atlas_attn_workspace_size
  run_host(kind, ...)  host tensors in, host tensor out (copies on the stream)
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import struct
from typing import Optional

import torch

from . import _build

__all__ = ["AtlasError", "decode", "suffix", "prefill", "cross", "shared", "kv_append",
           "kv_append_rope", "kv_append_norm_rope", "kv_weights", "kv_select", "kv_compact", "kv_resize",
           "workspace_size", "run_host",
           "library_path", "DEV_BAD_PAGE", "DEV_BAD_SEQLEN", "DEV_TIMEOUT", "DEV_NO_PAGES",
           "DEBUG_WITHHOLD_STAGE", "KIND_DECODE", "KIND_SUFFIX", "KIND_PREFILL",
           "KIND_CROSS", "rope_sections", "shared_workspace_size"]

KIND_DECODE, KIND_SUFFIX, KIND_PREFILL, KIND_CROSS = 0, 1, 2, 3
_KINDS = {"decode": KIND_DECODE, "suffix": KIND_SUFFIX, "prefill": KIND_PREFILL,
          "cross": KIND_CROSS}
DEV_BAD_PAGE, DEV_BAD_SEQLEN, DEV_TIMEOUT, DEV_NO_PAGES = 1, 2, 4, 8
DEBUG_WITHHOLD_STAGE = 1
DEBUG_TC_DIRECT = 2
DEBUG_SHARED_SPLIT, DEBUG_SHARED_TC, DEBUG_SHARED_WHOLE = 4, 8, 16
_F32, _BF16 = 0, 1
_DTYPES = {torch.float32: _F32, torch.bfloat16: _BF16}
STATUS_NAMES = {0: "ATLAS_OK", 1: "ATLAS_ERR_INVALID_ARG", 2: "ATLAS_ERR_UNSUPPORTED",
                3: "ATLAS_ERR_WORKSPACE", 4: "ATLAS_ERR_CUDA", 5: "ATLAS_ERR_DEVICE"}


class AtlasError(RuntimeError):
    """A non-OK status from the library."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class _Launch(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("q_len", ctypes.c_int32),
                ("q_dtype", ctypes.c_int), ("kv_dtype", ctypes.c_int),
                ("out_dtype", ctypes.c_int), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("status_word", ctypes.c_void_p),
                ("stream", ctypes.c_void_p), ("split_tokens", ctypes.c_int32),
                ("debug_flags", ctypes.c_uint32), ("events", ctypes.c_void_p),
                ("window", ctypes.c_int32), ("softcap", ctypes.c_float),
                ("sinks", ctypes.c_void_p), ("q_lens", ctypes.c_void_p),
                ("chunk_range", ctypes.c_void_p), ("phase", ctypes.c_int32),
                ("sm_count", ctypes.c_int32)]

PHASE_ALL, PHASE_CHUNKS, PHASE_MERGE = 0, 1, 2


class _Shared(ctypes.Structure):
    _fields_ = [("prefix_table", ctypes.c_void_p), ("prefix_lens", ctypes.c_void_p),
                ("group_starts", ctypes.c_void_p), ("n_groups", ctypes.c_int32),
                ("max_prefix_pages", ctypes.c_int32)]


class _PoolConfig(ctypes.Structure):
    _fields_ = [("hot_slots", ctypes.c_int32), ("scratch_slots", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("host_pages", ctypes.c_int32)]


class _PoolRequest(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("host_page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("chunk_tokens", ctypes.c_int32), ("keep_recent_tokens", ctypes.c_int32),
                ("admit", ctypes.c_int32)]


class PoolStats(ctypes.Structure):
    """What one plan of a HotPagePool did (atlas_pool_stats)."""
    _fields_ = [("passes", ctypes.c_int32), ("pages", ctypes.c_int64), ("hits", ctypes.c_int64),
                ("admitted", ctypes.c_int64), ("evicted", ctypes.c_int64),
                ("scratch_loads", ctypes.c_int64), ("copies", ctypes.c_int64)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class _Append(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int), ("status_word", ctypes.c_void_p),
                ("stream", ctypes.c_void_p)]


class _Rope(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int), ("n_q_heads", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("q_strides", ctypes.c_int64 * 3), ("k_strides", ctypes.c_int64 * 3),
                ("v_strides", ctypes.c_int64 * 3), ("positions", ctypes.c_void_p),
                ("n_axes", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("pair_axis", ctypes.c_void_p),
                ("inv_freq", ctypes.c_void_p), ("theta", ctypes.c_double),
                ("status_word", ctypes.c_void_p), ("stream", ctypes.c_void_p)]


class _Norm(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("weight_dtype", ctypes.c_int), ("per_head", ctypes.c_int32),
                ("weight_offset", ctypes.c_float), ("eps", ctypes.c_float)]


class _Weights(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("q_len", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("weights", ctypes.c_void_p),
                ("row_tokens", ctypes.c_int32), ("accumulate", ctypes.c_int32),
                ("q_lens", ctypes.c_void_p), ("window", ctypes.c_int32),
                ("softcap", ctypes.c_float), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("status_word", ctypes.c_void_p),
                ("stream", ctypes.c_void_p), ("sm_count", ctypes.c_int32)]


class _Select(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("row_tokens", ctypes.c_int32),
                ("budget", ctypes.c_int32), ("keep_first", ctypes.c_int32),
                ("keep_recent", ctypes.c_int32), ("kept_row_tokens", ctypes.c_int32),
                ("kept", ctypes.c_void_p),
                ("new_lens", ctypes.c_void_p), ("kept_weights", ctypes.c_void_p),
                ("status_word", ctypes.c_void_p), ("stream", ctypes.c_void_p)]


class _Compact(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_kept", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int), ("new_page_table", ctypes.c_void_p),
                ("new_max_pages", ctypes.c_int32), ("status_word", ctypes.c_void_p),
                ("stream", ctypes.c_void_p)]


class _Resize(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("n_new", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("status_word", ctypes.c_void_p), ("stream", ctypes.c_void_p)]


# The structures of calls whose time on the host counts, packed in one step (ctypes sets field by
# field); native alignment lays them out as the declarations above.
_pack_launch = struct.Struct("iiiiiiiPPPQPPiIPifPPPii").pack
_pack_shared = struct.Struct("PPPii").pack
_pack_rope = struct.Struct("iiiiiiPPqqqqqqqqqPiiiPPdPP").pack
_pack_norm = struct.Struct("PPiiff").pack
_pack_resize = struct.Struct("iiiiPPPP").pack
_lib = _fast = None


class _Fast:
    """Entry points that take packed structures."""

    def __init__(self, lib):
        pointers, ints = [ctypes.c_void_p] * 7, [ctypes.c_int32] * 3
        for name, args, result in (
                ("atlas_attn_shared", pointers[:5] + [ctypes.c_int32] * 4 + [ctypes.c_float] + pointers[:2],
                 ctypes.c_int),
                ("atlas_attn_shared_workspace_size", [ctypes.c_int32] * 4 + pointers[:2], ctypes.c_size_t),
                ("atlas_kv_append_rope", pointers + ints + pointers[:1], ctypes.c_int),
                ("atlas_kv_append_norm_rope", pointers + ints + pointers[:2], ctypes.c_int),
                ("atlas_kv_resize", pointers[:5] + ints[:1] + pointers[:1], ctypes.c_int)):
            fn = lib[name]  # (a function object of its own)
            fn.argtypes, fn.restype = args, result
            setattr(self, name[6:], fn)


def library_path() -> str:
    return _build.LIB


def load_library(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libatlas_attn.so; raises if it has not been built (no fallback)."""
    global _lib, _fast
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB):
        if not build_if_missing:
            raise ImportError(f"{_build.LIB} is missing: build it with "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
        _build.build()
    lib = ctypes.CDLL(_build.LIB)
    args = [ctypes.c_void_p] * 5 + [ctypes.c_int32] * 4 + [ctypes.c_float,
                                                           ctypes.POINTER(_Launch)]
    for name in ("atlas_attn_decode", "atlas_attn_suffix", "atlas_attn_prefill",
                 "atlas_attn_cross"):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.atlas_attn_shared.argtypes = args[:-1] + [ctypes.POINTER(_Shared), ctypes.POINTER(_Launch)]
    lib.atlas_attn_shared.restype = ctypes.c_int
    lib.atlas_attn_shared_workspace_size.argtypes = [ctypes.c_int32] * 4 + [
        ctypes.POINTER(_Shared), ctypes.POINTER(_Launch)]
    lib.atlas_attn_shared_workspace_size.restype = ctypes.c_size_t
    lib.atlas_attn_workspace_size.argtypes = [ctypes.c_int] + [ctypes.c_int32] * 4 + [
        ctypes.POINTER(_Launch)]
    lib.atlas_attn_workspace_size.restype = ctypes.c_size_t
    lib.atlas_kv_append.argtypes = [ctypes.c_void_p] * 7 + [ctypes.c_int32] * 3 + [
        ctypes.POINTER(_Append)]
    lib.atlas_kv_append.restype = ctypes.c_int
    lib.atlas_kv_append_rope.argtypes = [ctypes.c_void_p] * 7 + [ctypes.c_int32] * 3 + [
        ctypes.POINTER(_Rope)]
    lib.atlas_kv_append_rope.restype = ctypes.c_int
    lib.atlas_kv_append_norm_rope.argtypes = [ctypes.c_void_p] * 7 + [ctypes.c_int32] * 3 + [
        ctypes.POINTER(_Rope), ctypes.POINTER(_Norm)]
    lib.atlas_kv_append_norm_rope.restype = ctypes.c_int
    lib.atlas_kv_weights.argtypes = [ctypes.c_void_p] * 5 + [ctypes.c_int32] * 4 + [
        ctypes.c_float, ctypes.POINTER(_Weights)]
    lib.atlas_kv_weights.restype = ctypes.c_int
    lib.atlas_kv_weights_workspace_size.argtypes = [ctypes.c_int32] * 4 + [
        ctypes.POINTER(_Weights)]
    lib.atlas_kv_weights_workspace_size.restype = ctypes.c_size_t
    lib.atlas_kv_select.argtypes = [ctypes.c_void_p] * 2 + [ctypes.c_int32,
                                                            ctypes.POINTER(_Select)]
    lib.atlas_kv_select.restype = ctypes.c_int
    lib.atlas_kv_compact.argtypes = [ctypes.c_void_p] * 5 + [ctypes.c_int32] * 3 + [
        ctypes.POINTER(_Compact)]
    lib.atlas_kv_compact.restype = ctypes.c_int
    lib.atlas_kv_resize.argtypes = [ctypes.c_void_p] * 5 + [ctypes.c_int32, ctypes.POINTER(_Resize)]
    lib.atlas_kv_resize.restype = ctypes.c_int
    lib.atlas_attn_status_string.argtypes = [ctypes.c_int]
    lib.atlas_attn_status_string.restype = ctypes.c_char_p
    lib.atlas_attn_split_tokens.argtypes = [ctypes.c_int] + [ctypes.c_int32] * 4 + [
        ctypes.POINTER(_Launch)]
    lib.atlas_attn_split_tokens.restype = ctypes.c_int32
    lib.atlas_pool_create.argtypes = [ctypes.POINTER(_PoolConfig), ctypes.POINTER(ctypes.c_void_p)]
    lib.atlas_pool_create.restype = ctypes.c_int
    lib.atlas_pool_destroy.argtypes = [ctypes.c_void_p]
    lib.atlas_pool_destroy.restype = None
    lib.atlas_pool_plan.argtypes = [ctypes.c_void_p, ctypes.POINTER(_PoolRequest),
                                    ctypes.POINTER(PoolStats)]
    lib.atlas_pool_plan.restype = ctypes.c_int
    lib.atlas_pool_pass.argtypes = [ctypes.c_void_p, ctypes.c_int32] + [ctypes.c_void_p] * 3 + [
        ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)]
    lib.atlas_pool_pass.restype = ctypes.c_int
    lib.atlas_pool_slot_of.argtypes = [ctypes.c_void_p, ctypes.c_int32]
    lib.atlas_pool_slot_of.restype = ctypes.c_int32
    lib.atlas_pool_invalidate.argtypes = [ctypes.c_void_p, ctypes.c_int32]
    lib.atlas_pool_invalidate.restype = None
    lib.atlas_pool_fill.argtypes = [ctypes.c_void_p] * 5 + [ctypes.c_int32, ctypes.c_int64,
                                                            ctypes.c_int32, ctypes.c_int32,
                                                            ctypes.c_void_p, ctypes.c_void_p]
    lib.atlas_pool_fill.restype = ctypes.c_int
    _lib, _fast = lib, _Fast(lib)
    return lib


def status_string(status: int) -> str:
    return load_library().atlas_attn_status_string(status).decode()


def _address(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _launch(q, k_pages, page_table, out_dtype, out=None, lse=None, workspace=None,
            status=None, stream=None, split_tokens=0, debug_flags=0, events=None,
            window=0, softcap=0.0, sinks=None, q_lens=None, chunk_range=None,
            phase=PHASE_ALL, sm_count=0) -> _Launch:
    L = _Launch()
    L.batch, L.q_len = q.shape[0], q.shape[2]
    L.max_pages_per_seq = page_table.shape[1]
    L.num_pages = k_pages.shape[0]
    L.q_dtype = _DTYPES.get(q.dtype, -1)
    L.kv_dtype = _DTYPES.get(k_pages.dtype, -1)
    L.out_dtype = _DTYPES.get(out_dtype, -1)
    L.out = _ptr(out)
    L.lse = _ptr(lse)
    L.workspace = _ptr(workspace)
    L.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    L.status_word = _ptr(status)
    L.stream = stream
    L.split_tokens = split_tokens
    L.debug_flags = debug_flags
    L.events = events
    L.window = window
    L.softcap = softcap
    L.sinks = _ptr(sinks)
    L.q_lens = _ptr(q_lens)
    L.chunk_range = _ptr(chunk_range)
    L.phase = phase
    L.sm_count = sm_count
    return L


def workspace_size(kind: str, q_shape, n_q_heads, n_kv_heads, head_dim, page_tokens,
                   max_pages_per_seq, num_pages, dtype=torch.bfloat16,
                   out_dtype=None, split_tokens=0, window=0, phase=PHASE_ALL) -> int:
    """Workspace bytes a call needs (from shapes, split size, window and phase only)."""
    L = _Launch()
    L.window, L.phase = window, phase
    L.batch, L.q_len = q_shape[0], q_shape[2]
    L.max_pages_per_seq, L.num_pages = max_pages_per_seq, num_pages
    L.q_dtype = L.kv_dtype = _DTYPES.get(dtype, -1)
    L.out_dtype = _DTYPES.get(out_dtype or dtype, -1)
    L.split_tokens = split_tokens
    n = load_library().atlas_attn_workspace_size(_KINDS[kind], n_q_heads, n_kv_heads, head_dim,
                                                 page_tokens, ctypes.byref(L))
    if n == ctypes.c_size_t(-1).value:
        raise AtlasError(1, "invalid arguments for workspace_size")
    return n


def _call(kind: str, q, k_pages, v_pages, page_table, seq_lens, n_q_heads, n_kv_heads,
          head_dim, page_tokens, scale, *, out=None, out_dtype=None, lse=None,
          workspace=None, status=None, split_tokens=0, debug_flags=0, events=None,
          window=0, softcap=0.0, sinks=None, q_lens=None, chunk_range=None,
          phase=PHASE_ALL, sm_count=0):
    """``events``: optional ctypes array of three cudaEvent_t handles (see
    EventTimer) recorded around the main kernel and the merge.  ``window``,
    ``softcap`` and ``sinks`` (float32 CUDA tensor [n_q_heads]) select the score /
    mask variants; the defaults give plain causal attention.  ``q_lens`` (int32
    CUDA tensor [B]) makes the batch ragged: sequence b has q_lens[b] query rows.
    ``phase`` and ``chunk_range`` (int32 CUDA tensor [B][2]) spread one call over
    several launches sharing ``workspace`` (atlas_launch.phase).  ``sm_count`` > 0
    plans for that many SMs instead of the device's (atlas_launch.sm_count)."""
    for name, t in (("q", q), ("k_pages", k_pages), ("v_pages", v_pages),
                    ("page_table", page_table), ("seq_lens", seq_lens)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if page_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("page_table and seq_lens must be int32")
    if q.dim() != 4 or k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("q must be [B][Hq][q_len][D] and pools [num_pages][Hkv][P][D]")
    out_dtype = out_dtype or (out.dtype if out is not None else q.dtype)
    if out is None and phase != PHASE_CHUNKS:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    if chunk_range is not None and (not chunk_range.is_cuda or chunk_range.dtype != torch.int32
                                    or chunk_range.numel() != 2 * q.shape[0]
                                    or not chunk_range.is_contiguous()):
        raise ValueError("chunk_range must be a contiguous int32 CUDA tensor [batch][2]")
    if status is not None and (status.dtype != torch.int32 or status.numel() < 1):
        raise ValueError("status must be an int32 device tensor")
    if sinks is not None and (not sinks.is_cuda or sinks.dtype != torch.float32 or
                              sinks.numel() != n_q_heads or not sinks.is_contiguous()):
        raise ValueError("sinks must be a contiguous float32 CUDA tensor [n_q_heads]")
    if q_lens is not None and (not q_lens.is_cuda or q_lens.dtype != torch.int32 or
                               q_lens.numel() != q.shape[0]):
        raise ValueError("q_lens must be an int32 CUDA tensor [batch]")
    return _enqueue(kind, q, k_pages, v_pages, page_table, seq_lens, n_q_heads, n_kv_heads,
                    head_dim, page_tokens, scale, out, out_dtype, lse, workspace, status,
                    split_tokens, debug_flags, events, window, softcap, sinks, q_lens,
                    chunk_range, phase, sm_count)


def _enqueue(kind, q, k_pages, v_pages, page_table, seq_lens, n_q_heads, n_kv_heads, head_dim,
             page_tokens, scale, out, out_dtype, lse, workspace, status, split_tokens=0,
             debug_flags=0, events=None, window=0, softcap=0.0, sinks=None, q_lens=None,
             chunk_range=None, phase=PHASE_ALL, sm_count=0):
    """An attention call whose tensors have been checked."""
    lib = load_library()
    stream = _stream(q.device)
    L = _launch(q, k_pages, page_table, out_dtype, out, lse, None, status, stream,
                split_tokens, debug_flags,
                None if events is None else ctypes.cast(events, ctypes.c_void_p).value,
                window, softcap, sinks, q_lens, chunk_range, phase, sm_count)
    need = lib.atlas_attn_workspace_size(_KINDS[kind], n_q_heads, n_kv_heads, head_dim,
                                         page_tokens, ctypes.byref(L))
    if workspace is None and 0 < need < ctypes.c_size_t(-1).value:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    L.workspace = _ptr(workspace)
    L.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    fn = getattr(lib, f"atlas_attn_{kind}")
    rc = fn(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
            seq_lens.data_ptr(), n_q_heads, n_kv_heads, head_dim, page_tokens, float(scale),
            ctypes.byref(L))
    if rc != 0:
        raise AtlasError(rc, status_string(rc))
    return out


def split_tokens_of(kind: str, q_shape, n_q_heads, n_kv_heads, head_dim, page_tokens,
                    max_pages_per_seq, num_pages, dtype=torch.bfloat16, out_dtype=None,
                    split_tokens=0, window=0, phase=PHASE_ALL) -> int:
    """Keys per split-KV chunk of such a call (0: no chunks), atlas_attn_split_tokens."""
    L = _Launch()
    L.window, L.phase = window, phase
    L.batch, L.q_len = q_shape[0], q_shape[2]
    L.max_pages_per_seq, L.num_pages = max_pages_per_seq, num_pages
    L.q_dtype = L.kv_dtype = _DTYPES.get(dtype, -1)
    L.out_dtype = _DTYPES.get(out_dtype or dtype, -1)
    L.split_tokens = split_tokens
    n = load_library().atlas_attn_split_tokens(_KINDS[kind], n_q_heads, n_kv_heads, head_dim,
                                               page_tokens, ctypes.byref(L))
    if n < 0:
        raise AtlasError(1, "invalid arguments for split_tokens_of")
    return n


def decode(q, k_pages, v_pages, page_table, seq_lens, n_q_heads, n_kv_heads, head_dim,
           page_tokens, scale, **kw):
    """One query row per sequence (q_len == 1).  Returns out [B][Hq][1][D]."""
    return _call("decode", q, k_pages, v_pages, page_table, seq_lens, n_q_heads, n_kv_heads,
                 head_dim, page_tokens, scale, **kw)


def suffix(q, k_pages, v_pages, page_table, seq_lens, n_q_heads, n_kv_heads, head_dim,
           page_tokens, scale, **kw):
    """Queries are the last q_len positions of each sequence's K/V."""
    return _call("suffix", q, k_pages, v_pages, page_table, seq_lens, n_q_heads, n_kv_heads,
                 head_dim, page_tokens, scale, **kw)


def prefill(q, k_pages, v_pages, page_table, seq_lens, n_q_heads, n_kv_heads, head_dim,
            page_tokens, scale, **kw):
    """Causal self-attention of whole prompts (seq_lens[b] == q_len for every b)."""
    return _call("prefill", q, k_pages, v_pages, page_table, seq_lens, n_q_heads, n_kv_heads,
                 head_dim, page_tokens, scale, **kw)


def cross(q, k_pages, v_pages, page_table, enc_lens, n_q_heads, n_kv_heads, head_dim,
          page_tokens, scale, *, out=None, out_dtype=None, lse=None, workspace=None, status=None,
          sinks=None, q_lens=None, **options):
    """Attention of q_len decoder rows to all enc_lens[b] encoder states of their
    sequence (no causal mask; enc_lens[b] == 0 gives rows of 0 and lse -inf).  The pools,
    table and lengths are the encoder's; q [B][Hq][q_len][D] and lse [B][Hq][q_len] the
    decoder's.  Other options are those of the causal calls."""
    device, dtype, shape = _cuda_device("q", q), q.dtype, q.shape
    pool = k_pages.shape
    if len(shape) != 4 or shape[1] != n_q_heads or shape[3] != head_dim or len(pool) != 4 or \
            pool[1:] != (n_kv_heads, page_tokens, head_dim) or v_pages.shape != pool:
        raise ValueError("q must be [B][Hq][q_len][D] and the pools [num_pages][Hkv][P][D], of the "
                         "sizes given")
    B, _, n, _ = shape
    if out is None:
        out_dtype = out_dtype or dtype
        out = torch.empty(shape, dtype=out_dtype, device=device)
    else:
        out_dtype = out_dtype or out.dtype
    _check(device, ("q", q, dtype), ("k_pages", k_pages, dtype), ("v_pages", v_pages, dtype),
           ("page_table", page_table, torch.int32), ("enc_lens", enc_lens, torch.int32),
           ("out", out, out_dtype), ("lse", lse, torch.float32), ("status", status, torch.int32),
           ("sinks", sinks, torch.float32), ("q_lens", q_lens, torch.int32),
           ("workspace", workspace, None if workspace is None else workspace.dtype))
    table = page_table.shape
    if len(table) != 2 or table[0] != B or enc_lens.numel() != B or out.shape != shape or \
            (lse is not None and lse.numel() != B * n_q_heads * n) or \
            (sinks is not None and sinks.numel() != n_q_heads) or \
            (q_lens is not None and q_lens.numel() != B) or \
            (status is not None and status.numel() < 1):
        raise ValueError("page_table must be [B][max_pages], enc_lens and q_lens [B], out like q, "
                         "lse [B][Hq][q_len], sinks [Hq], status one word")
    with _on(device):
        return _enqueue("cross", q, k_pages, v_pages, page_table, enc_lens, n_q_heads, n_kv_heads,
                        head_dim, page_tokens, scale, out, out_dtype, lse, workspace, status,
                        sinks=sinks, q_lens=q_lens, **options)


def shared(q, k_pages, v_pages, prefix_table, prefix_lens, group_starts, page_table, seq_lens,
           n_q_heads, n_kv_heads, head_dim, page_tokens, scale, *, out=None, out_dtype=None,
           lse=None, workspace=None, status=None, split_tokens=0, debug_flags=0, events=None,
           softcap=0.0, sinks=None, q_lens=None, sm_count=0):
    """Attention of the last q_len positions of each sequence to its own cache (page_table
    [B][max_pages], seq_lens [B]: as for suffix) and to all of its group's prefix: sequences
    group_starts[n] <= b < group_starts[n + 1] share the prefix_lens[n] keys of prefix_table[n]
    [n_groups][max_prefix_pages] (atlas_attn_shared).  Other options are those of the causal
    calls; ``workspace``: at least shared_workspace_size(...) bytes."""
    device, dtype, shape, pool = _cuda_device("q", q), q.dtype, q.shape, k_pages.shape
    if len(shape) != 4 or shape[1] != n_q_heads or shape[3] != head_dim or len(pool) != 4 or \
            pool[1:] != (n_kv_heads, page_tokens, head_dim) or v_pages.shape != pool:
        raise ValueError("q must be [B][Hq][q_len][D] and the pools [num_pages][Hkv][P][D], of the "
                         "sizes given")
    B, _, n, _ = shape
    if out is None:
        out_dtype = out_dtype or dtype
        out = torch.empty(shape, dtype=out_dtype, device=device)
    else:
        out_dtype = out_dtype or out.dtype
    i32, f32, index = torch.int32, torch.float32, device.index
    if not _fits(index, (q, dtype), (k_pages, dtype), (v_pages, dtype), (prefix_table, i32),
                 (prefix_lens, i32), (group_starts, i32), (page_table, i32), (seq_lens, i32),
                 (out, out_dtype), (lse, f32), (status, i32), (sinks, f32), (q_lens, i32),
                 (workspace, None if workspace is None else workspace.dtype)):
        _check(device, ("q", q, dtype), ("k_pages", k_pages, dtype), ("v_pages", v_pages, dtype),
               ("prefix_table", prefix_table, i32), ("prefix_lens", prefix_lens, i32),
               ("group_starts", group_starts, i32), ("page_table", page_table, i32),
               ("seq_lens", seq_lens, i32), ("out", out, out_dtype), ("lse", lse, f32),
               ("status", status, i32), ("sinks", sinks, f32), ("q_lens", q_lens, i32),
               ("workspace", workspace, None if workspace is None else workspace.dtype))
    table, prefixes = page_table.shape, prefix_table.shape
    if len(table) != 2 or table[0] != B or seq_lens.numel() != B or len(prefixes) != 2 or \
            prefix_lens.numel() != prefixes[0] or group_starts.numel() != prefixes[0] + 1 or \
            out.shape != shape or (lse is not None and lse.numel() != B * n_q_heads * n) or \
            (sinks is not None and sinks.numel() != n_q_heads) or \
            (q_lens is not None and q_lens.numel() != B) or \
            (status is not None and status.numel() < 1):
        raise ValueError("page_table must be [B][max_pages], prefix_table [n_groups][max_prefix_pages], "
                         "prefix_lens [n_groups], group_starts [n_groups + 1], seq_lens and q_lens "
                         "[B], out like q, lse [B][Hq][q_len], sinks [Hq], status one word")
    load_library()
    kind = _DTYPES.get(dtype, -1)
    S = _pack_shared(prefix_table.data_ptr(), prefix_lens.data_ptr(), group_starts.data_ptr(),
                     prefixes[0], prefixes[1])
    L = [B, table[1], pool[0], n, kind, kind, _DTYPES.get(out_dtype, -1), out.data_ptr(), _address(lse),
         0, 0, _address(status), _stream(device) or 0, split_tokens, debug_flags,
         0 if events is None else ctypes.cast(events, ctypes.c_void_p).value, 0, softcap,
         _address(sinks), _address(q_lens), 0, PHASE_ALL, sm_count]
    with _on(device):
        if workspace is None:
            need = _fast.attn_shared_workspace_size(n_q_heads, n_kv_heads, head_dim, page_tokens, S,
                                                    _pack_launch(*L))
            if need < ctypes.c_size_t(-1).value:
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
        if workspace is not None:
            L[9], L[10] = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        rc = _fast.attn_shared(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                               page_table.data_ptr(), seq_lens.data_ptr(), n_q_heads, n_kv_heads,
                               head_dim, page_tokens, scale, S, _pack_launch(*L))
    if rc != 0:
        raise AtlasError(rc, status_string(rc))
    return out


def shared_workspace_size(q_shape, n_q_heads, n_kv_heads, head_dim, page_tokens, max_pages_per_seq,
                          n_groups, max_prefix_pages, num_pages, dtype=torch.bfloat16,
                          out_dtype=None, split_tokens=0, debug_flags=0, sm_count=0) -> int:
    """Workspace bytes a shared() call needs: from shapes, the split size and the number of SMs that
    it is planned for (sm_count, as given to the call; 0: those of the current device)."""
    L = _Launch()
    L.batch, L.q_len = q_shape[0], q_shape[2]
    L.max_pages_per_seq, L.num_pages = max_pages_per_seq, num_pages
    L.q_dtype = L.kv_dtype = _DTYPES.get(dtype, -1)
    L.out_dtype = _DTYPES.get(out_dtype or dtype, -1)
    L.split_tokens, L.debug_flags, L.sm_count = split_tokens, debug_flags, sm_count
    S = _Shared(n_groups=n_groups, max_prefix_pages=max_prefix_pages)
    n = load_library().atlas_attn_shared_workspace_size(n_q_heads, n_kv_heads, head_dim, page_tokens,
                                                        ctypes.byref(S), ctypes.byref(L))
    if n == ctypes.c_size_t(-1).value:
        raise AtlasError(1, "invalid arguments for shared_workspace_size")
    return n


def run(problem, **kw):
    """Call the entry point named by ``problem.kind`` on an inputs.Problem on the GPU."""
    fn = {"decode": decode, "suffix": suffix, "prefill": prefill}[problem.kind]
    return fn(problem.q, problem.k_pages, problem.v_pages, problem.page_table,
              problem.seq_lens, problem.n_q_heads, problem.n_kv_heads, problem.head_dim,
              problem.page_tokens, problem.scale, **kw)


def kv_append(k_new, v_new, k_pages, v_pages, page_table, seq_lens, n_new=None,
              status=None):
    """Write the new tokens' K/V rows [B][Hkv][max_new][D] of each sequence into its
    pages at positions seq_lens[b] .. seq_lens[b] + n_new[b] - 1 (atlas_kv_append).
    The pools are updated in place; seq_lens is not advanced."""
    lib = load_library()
    for name, t in (("k_new", k_new), ("v_new", v_new), ("k_pages", k_pages),
                    ("v_pages", v_pages), ("page_table", page_table), ("seq_lens", seq_lens)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if k_new.shape != v_new.shape or k_new.dim() != 4 or k_pages.dim() != 4:
        raise ValueError("k_new/v_new must be [B][Hkv][max_new][D], pools [pages][Hkv][P][D]")
    if k_new.dtype != k_pages.dtype:
        raise ValueError("new rows and pools must share a dtype")
    A = _Append()
    A.batch, A.max_new = k_new.shape[0], k_new.shape[2]
    A.max_pages_per_seq, A.num_pages = page_table.shape[1], k_pages.shape[0]
    A.kv_dtype = _DTYPES.get(k_pages.dtype, -1)
    A.status_word = _ptr(status)
    A.stream = torch.cuda.current_stream(k_new.device).cuda_stream
    rc = lib.atlas_kv_append(k_new.data_ptr(), v_new.data_ptr(), k_pages.data_ptr(),
                             v_pages.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
                             _ptr(n_new), k_new.shape[1], k_new.shape[3], k_pages.shape[2],
                             ctypes.byref(A))
    if rc != 0:
        raise AtlasError(rc, status_string(rc))


_SAME_DEVICE = contextlib.nullcontext()


def _on(device):
    """The device guard of a call: work goes to the tensors' device, whichever is current."""
    if device.index == torch._C._cuda_getDevice():
        return _SAME_DEVICE
    return torch.cuda.device(device)


def _stream(device):
    """Handle of the current torch stream of a CUDA device (torch.cuda.current_stream
    builds a Stream object around it, several microseconds a call)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _check(device, *tensors):
    """Every given (name, tensor, dtype) is contiguous, of `device` and of that dtype."""
    for name, t, dtype in tensors:
        if t is None:
            continue
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}")
        if t.device != device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor on {device}")


def _fits(index, *tensors):
    """Whether _check would pass them: (tensor or None, dtype) each, on the device of that index."""
    for t, dtype in tensors:
        if t is not None and (t.dtype is not dtype or t.get_device() != index or not t.is_contiguous()):
            return False
    return True


def _cuda_device(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


@functools.lru_cache(maxsize=64)
def _host_array(ctype, values):
    return (ctype * len(values))(*values)


@functools.lru_cache(maxsize=64)
def _frequencies(theta, rot_dim):
    """theta^(-2 p / rot_dim) of every pair: a table of its arguments alone."""
    if not 0.0 < theta < float("inf") or not 2 <= rot_dim <= 4096:
        return None  # the library refuses these
    return _host_array(ctypes.c_double, tuple(theta ** (-2.0 * p / rot_dim)
                                              for p in range(rot_dim // 2)))


_DENSE = (0, 0, 0)


def _row_strides(name, t):
    """Element strides (batch, head, token) of a [B][H][n][D] view with contiguous rows;
    all zero for a contiguous one."""
    if t.is_contiguous():
        return _DENSE
    sb, sh, st, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must have contiguous rows of head_dim elements")
    nb, nh, nt, _ = t.shape
    sb, sh, st = sb if nb > 1 else 0, sh if nh > 1 else 0, st if nt > 1 else 0
    if not (sb or sh or st):  # the library reads all-zero strides as dense rows
        raise ValueError(f"{name} is one row broadcast to all: make it contiguous")
    return sb, sh, st


def kv_append_rope(q, k_new, v_new, k_pages, v_pages, page_table, seq_lens, positions, *,
                   theta=10000.0, inv_freq=None, rot_dim=None, pair_axis=None,
                   interleaved=False, n_new=None, q_out=None, status=None):
    """Rotate the step's queries and new keys by their positions, and write the keys and
    values into the cache (atlas_kv_append_rope).

    q [B][Hq][n][D] (or None), k_new and v_new [B][Hkv][n][D]: views with contiguous rows,
    e.g. slices of a fused projection [B][n][heads][D] transposed to [B][heads][n][D].
    positions int32 [n_axes][B][n] (or [B][n] for one axis).  rot_dim: rotated leading
    elements of a row (default all); pair_axis: rot_dim // 2 axis numbers, one per pair
    (default 0), see ``rope_sections``; inv_freq: rot_dim // 2 host floats, radians per
    position (default theta ** (-2 p / rot_dim)); interleaved: pairs (2p, 2p + 1) rather
    than (p, p + rot_dim / 2).  Returns the rotated queries [B][Hq][n][D] (q_out, which
    may be q itself when q is contiguous); None without q."""
    return _append_rope(q, k_new, v_new, k_pages, v_pages, page_table, seq_lens, positions, theta,
                        inv_freq, rot_dim, pair_axis, interleaved, n_new, q_out, status, None)


def kv_append_norm_rope(q, k_new, v_new, k_pages, v_pages, page_table, seq_lens, positions, *,
                        q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0, theta=10000.0,
                        inv_freq=None, rot_dim=None, pair_axis=None, interleaved=False, n_new=None,
                        q_out=None, status=None):
    """kv_append_rope with a root-mean-square norm of each head's queries and new keys before
    the rotation, in the same pass (atlas_kv_append_norm_rope): each row is divided by
    sqrt(mean of its squares + eps) and multiplied by its weights + weight_offset.  q_weight and
    k_weight: [D], or [Hq][D] and [Hkv][D] for weights of each head (both alike), of the pools'
    dtype or float32; None: ones."""
    return _append_rope(q, k_new, v_new, k_pages, v_pages, page_table, seq_lens, positions, theta,
                        inv_freq, rot_dim, pair_axis, interleaved, n_new, q_out, status,
                        (q_weight, k_weight, eps, weight_offset))


def _norm(device, dtype, q_weight, k_weight, eps, offset, Hq, Hkv, D):
    """The packed atlas_qk_norm of checked weights."""
    first = q_weight if q_weight is not None else k_weight
    if first is None:
        return _pack_norm(0, 0, _F32, 0, offset, eps)
    kind, per_head = first.dtype, first.dim() == 2
    if kind is not dtype and kind is not torch.float32:
        raise ValueError(f"q_weight and k_weight must be {dtype} or {torch.float32}")
    if not _fits(device.index, (q_weight, kind), (k_weight, kind)):
        _check(device, ("q_weight", q_weight, kind), ("k_weight", k_weight, kind))
    for name, w, heads in (("q_weight", q_weight, Hq), ("k_weight", k_weight, Hkv)):
        if w is not None and w.shape != ((heads, D) if per_head else (D,)) and \
                not (heads is None and w.dim() == 1 + per_head and w.shape[-1] == D):
            raise ValueError(f"{name} must be [head_dim], or [heads][head_dim] like the other")
    return _pack_norm(_address(q_weight), _address(k_weight), _DTYPES.get(kind, -1), per_head, offset, eps)


def _append_rope(q, k_new, v_new, k_pages, v_pages, page_table, seq_lens, positions, theta, inv_freq,
                 rot_dim, pair_axis, interleaved, n_new, q_out, status, norm):
    lib = load_library()
    shape, pool = k_new.shape, k_pages.shape
    if len(shape) != 4 or v_new.shape != shape or len(pool) != 4 or v_pages.shape != pool or \
            pool[1] != shape[1] or pool[3] != shape[3]:
        raise ValueError("k_new/v_new must be [B][Hkv][n][D], pools [pages][Hkv][P][D]")
    B, Hkv, n, D = shape
    device, dtype = _cuda_device("k_pages", k_pages), k_pages.dtype
    if positions.dim() == 2:
        positions = positions[None]
    if positions.shape[1:] != (B, n):
        raise ValueError("positions must be [n_axes][B][n]")
    index, i32 = device.index, torch.int32
    for name, t in (("k_new", k_new), ("v_new", v_new), ("q", q)):
        if t is not None and (t.dtype is not dtype or t.get_device() != index):
            raise ValueError(f"{name} must be a {dtype} tensor on {device}")
    if not _fits(index, (k_pages, dtype), (v_pages, dtype), (page_table, i32), (seq_lens, i32),
                 (positions, i32), (n_new, i32), (q_out, dtype), (status, i32)):
        _check(device, ("k_pages", k_pages, dtype), ("v_pages", v_pages, dtype),
               ("page_table", page_table, i32), ("seq_lens", seq_lens, i32),
               ("positions", positions, i32), ("n_new", n_new, i32), ("q_out", q_out, dtype),
               ("status", status, i32))
    table = page_table.shape
    if len(table) != 2 or table[0] != B or seq_lens.numel() != B or \
            (n_new is not None and n_new.numel() != B):
        raise ValueError("page_table must be [B][max_pages]; seq_lens and n_new [B]")
    rot_dim = D if rot_dim is None else rot_dim
    for name, x in (("pair_axis", pair_axis), ("inv_freq", inv_freq)):
        if x is not None and len(x) != rot_dim // 2:
            raise ValueError(f"{name} must have rot_dim / 2 entries")
    n_q_heads = q_at = q_out_at = 0
    q_strides = _DENSE
    if q is not None:
        rows = q.shape
        if len(rows) != 4 or rows[0] != B or rows[2:] != (n, D):
            raise ValueError("q must be [B][Hq][n][D] like k_new")
        if q_out is None:
            q_out = torch.empty(rows, dtype=dtype, device=device)
        elif q_out.shape != rows:
            raise ValueError("q_out must have q's shape")
        n_q_heads, q_at, q_out_at, q_strides = rows[1], q.data_ptr(), q_out.data_ptr(), _row_strides("q", q)
        if q_out_at == q_at and not q.is_contiguous():
            raise ValueError("q_out may be q itself only when q is contiguous")
    elif q_out is not None:
        raise ValueError("q_out needs q")
    # (the host arrays are held until the call is over)
    axes = None if pair_axis is None else _host_array(ctypes.c_int32, tuple(pair_axis))
    freq = _frequencies(theta, rot_dim) if inv_freq is None else \
        (ctypes.c_double * len(inv_freq))(*inv_freq)
    R = _pack_rope(B, table[1], pool[0], n, _DTYPES.get(dtype, -1), n_q_heads, q_at, q_out_at,
                   *q_strides, *_row_strides("k_new", k_new), *_row_strides("v_new", v_new),
                   positions.data_ptr(), positions.shape[0], rot_dim, bool(interleaved),
                   0 if axes is None else ctypes.addressof(axes),
                   0 if freq is None else ctypes.addressof(freq), theta, _address(status),
                   _stream(device) or 0)
    args = (k_new.data_ptr(), v_new.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
            page_table.data_ptr(), seq_lens.data_ptr(), _ptr(n_new), Hkv, D, pool[2], R)
    if norm is None:
        with _on(device):
            rc = _fast.kv_append_rope(*args)
    else:
        N = _norm(device, dtype, *norm, None if q is None else n_q_heads, Hkv, D)
        with _on(device):
            rc = _fast.kv_append_norm_rope(*args, N)
    if rc != 0:
        raise AtlasError(rc, status_string(rc))
    return q_out


def rope_sections(sizes, cycle=False):
    """The pair_axis of kv_append_rope for axes that turn sizes[a] pairs each: axis 0's
    pairs, then axis 1's, ... or (cycle) pair after pair to the next axis that has any left."""
    if not cycle:
        return tuple(a for a, size in enumerate(sizes) for _ in range(size))
    left, out = list(sizes), []
    while any(left):
        for a, size in enumerate(left):
            if size > 0:
                out.append(a)
                left[a] -= 1
    return tuple(out)


def kv_weights(q, k_pages, page_table, seq_lens, lse, n_q_heads, n_kv_heads, head_dim,
               page_tokens, scale, *, weights=None, accumulate=True, q_lens=None, window=0,
               softcap=0.0, workspace=None, status=None, sm_count=0):
    """Add the attention weight that each cached key received from the rows q
    [B][Hq][q_len][D] to weights [B][Hkv][row_tokens] (float32; new zeros of
    max_pages * P tokens when None), or overwrite with it (atlas_kv_weights).  lse
    [B][Hq][q_len]: what the attention call with the same rows and options returned.
    Returns weights."""
    lib = load_library()
    if q.dim() != 4 or k_pages.dim() != 4:
        raise ValueError("q must be [B][Hq][q_len][D] and the pool [num_pages][Hkv][P][D]")
    B = q.shape[0]
    if q.shape[1] != n_q_heads or q.shape[3] != head_dim or \
            k_pages.shape[1:] != (n_kv_heads, page_tokens, head_dim):
        raise ValueError("q and the pool must have the shapes the sizes given say")
    if weights is None:
        weights = torch.zeros((B, n_kv_heads, page_table.shape[1] * page_tokens), device=q.device)
    device = _cuda_device("q", q)
    _check(device, ("q", q, q.dtype), ("k_pages", k_pages, q.dtype),
           ("page_table", page_table, torch.int32), ("seq_lens", seq_lens, torch.int32),
           ("lse", lse, torch.float32), ("weights", weights, torch.float32),
           ("workspace", workspace, workspace.dtype if workspace is not None else None),
           ("q_lens", q_lens, torch.int32), ("status", status, torch.int32))
    if page_table.dim() != 2 or page_table.shape[0] != B or seq_lens.numel() != B or \
            lse.numel() != q.shape[0] * q.shape[1] * q.shape[2] or weights.dim() != 3 or \
            weights.shape[:2] != (B, n_kv_heads) or (q_lens is not None and q_lens.numel() != B):
        raise ValueError("page_table must be [B][max_pages], seq_lens and q_lens [B], lse "
                         "[B][Hq][q_len], weights [B][Hkv][row_tokens]")
    W = _Weights()
    W.batch, W.q_len, W.dtype = B, q.shape[2], _DTYPES.get(q.dtype, -1)
    W.max_pages_per_seq, W.num_pages = page_table.shape[1], k_pages.shape[0]
    W.weights, W.row_tokens, W.accumulate = weights.data_ptr(), weights.shape[2], int(bool(accumulate))
    W.q_lens, W.window, W.softcap, W.sm_count = _ptr(q_lens), window, softcap, sm_count
    W.status_word = _ptr(status)
    W.stream = _stream(device)
    with _on(device):
        need = lib.atlas_kv_weights_workspace_size(n_q_heads, n_kv_heads, head_dim, page_tokens,
                                                   ctypes.byref(W))
        if workspace is None and 0 < need < ctypes.c_size_t(-1).value:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        if workspace is not None:
            W.workspace = workspace.data_ptr()
            W.workspace_bytes = workspace.numel() * workspace.element_size()
        rc = lib.atlas_kv_weights(q.data_ptr(), k_pages.data_ptr(), page_table.data_ptr(),
                                  seq_lens.data_ptr(), lse.data_ptr(), n_q_heads, n_kv_heads,
                                  head_dim, page_tokens, float(scale), ctypes.byref(W))
    if rc != 0:
        raise AtlasError(rc, status_string(rc))
    return weights


def kv_select(weights, seq_lens, budget, *, keep_first=0, keep_recent=0, kept=None, new_lens=None,
              kept_weights=None, kept_row_tokens=None, status=None):
    """The keys of each (sequence, kv head) that stay under the budget: the first and the
    most recent ones, the others by weights [B][Hkv][row_tokens] (atlas_kv_select).
    Returns kept int32 [B][Hkv][budget] (ascending, then -1), new_lens int32 [B] and
    kept_weights [B][Hkv][kept_row_tokens], the totals of the kept keys, then 0: what
    kv_weights goes on adding to after kv_compact.  kept_row_tokens (default: budget, or the
    row length of kept_weights) must leave room for the keys to come: kv_weights skips a
    sequence longer than its rows and reports it in the status word alone.  Outputs given may
    not overlap weights, seq_lens (new_lens is not seq_lens) or one another."""
    lib = load_library()
    if weights.dim() != 3 or seq_lens.numel() != weights.shape[0]:
        raise ValueError("weights must be [B][Hkv][row_tokens] and seq_lens [B]")
    B, Hkv, T = weights.shape
    budget = int(budget)
    shape = (B, Hkv, max(budget, 0))
    dev = _cuda_device("weights", weights)
    if kept is None:
        kept = torch.empty(shape, dtype=torch.int32, device=dev)
    if kept_weights is None:
        row = shape[2] if kept_row_tokens is None else int(kept_row_tokens)
        kept_weights = torch.empty((B, Hkv, max(row, 0)), dtype=torch.float32, device=dev)
    if new_lens is None:
        new_lens = torch.empty(B, dtype=torch.int32, device=dev)
    _check(dev, ("weights", weights, torch.float32), ("seq_lens", seq_lens, torch.int32),
           ("kept", kept, torch.int32), ("kept_weights", kept_weights, torch.float32),
           ("new_lens", new_lens, torch.int32), ("status", status, torch.int32))
    room = kept_weights.shape
    if kept.shape != shape or len(room) != 3 or room[:2] != shape[:2] or room[2] < shape[2] or \
            kept_row_tokens not in (None, room[2]) or new_lens.numel() != B:
        raise ValueError("kept must be [B][Hkv][budget], kept_weights [B][Hkv][kept_row_tokens] "
                         "of at least budget, and new_lens [B]")
    S = _Select()
    S.batch, S.row_tokens, S.budget = B, T, budget
    S.keep_first, S.keep_recent, S.kept_row_tokens = keep_first, keep_recent, room[2]
    S.kept, S.new_lens, S.kept_weights = kept.data_ptr(), new_lens.data_ptr(), kept_weights.data_ptr()
    S.status_word = _ptr(status)
    S.stream = _stream(dev)
    with _on(dev):
        rc = lib.atlas_kv_select(weights.data_ptr(), seq_lens.data_ptr(), Hkv, ctypes.byref(S))
    if rc != 0:
        raise AtlasError(rc, status_string(rc))
    return kept, new_lens, kept_weights


def kv_compact(k_pages, v_pages, page_table, kept, new_lens, *, new_page_table=None, status=None):
    """Move the kept rows of both pools together (atlas_kv_compact): into the sequences'
    own pages (new_page_table None; kept ascending, pages not shared), or into the fresh
    pages of new_page_table [B][new_max_pages].  The pools are updated in place."""
    lib = load_library()
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("pools must be [num_pages][Hkv][P][D]")
    num_pages, Hkv, P, D = k_pages.shape
    device = _cuda_device("k_pages", k_pages)
    _check(device, ("k_pages", k_pages, k_pages.dtype), ("v_pages", v_pages, k_pages.dtype),
           ("page_table", page_table, torch.int32), ("kept", kept, torch.int32),
           ("new_lens", new_lens, torch.int32), ("new_page_table", new_page_table, torch.int32),
           ("status", status, torch.int32))
    if page_table.dim() != 2 or kept.dim() != 3 or \
            kept.shape[:2] != (page_table.shape[0], Hkv) or \
            new_lens.numel() != page_table.shape[0] or (new_page_table is not None and (
                new_page_table.dim() != 2 or new_page_table.shape[0] != page_table.shape[0])):
        raise ValueError("page tables must be [B][max_pages], kept [B][Hkv][max_kept], new_lens [B]")
    C = _Compact()
    C.batch, C.max_pages_per_seq = page_table.shape
    C.num_pages, C.max_kept, C.kv_dtype = num_pages, kept.shape[2], _DTYPES.get(k_pages.dtype, -1)
    if new_page_table is not None:
        C.new_page_table, C.new_max_pages = new_page_table.data_ptr(), new_page_table.shape[1]
    C.status_word = _ptr(status)
    C.stream = _stream(device)
    with _on(device):
        rc = lib.atlas_kv_compact(k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
                                  kept.data_ptr(), new_lens.data_ptr(), Hkv, D, P, ctypes.byref(C))
    if rc != 0:
        raise AtlasError(rc, status_string(rc))


def kv_resize(page_table, n_pages, seq_lens, free_pages, free_state, page_tokens, *, n_new=None,
              slots=None, max_new=None, status=None):
    """Give every sequence the pages that seq_lens [B] needs (atlas_kv_resize): those it lacks
    come from the ring free_pages [num_pages], free_state [2] = first entry and count, into
    page_table [B][max_pages] behind its n_pages [B]; those it has too many of go back to the
    ring.  All int32; page_table, n_pages, free_pages and free_state are updated in place.
    slots (or max_new, for a new one): [B][max_new], written with the places page * page_tokens
    + offset of each sequence's last n_new[b] tokens (None: max_new of them), then -1.  Returns
    slots (None without)."""
    load_library()
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B][max_pages]")
    B, width = page_table.shape
    device, i32 = _cuda_device("page_table", page_table), torch.int32
    if slots is None and max_new:
        slots = torch.empty((B, max_new), dtype=i32, device=device)
    if n_new is not None and slots is None:
        raise ValueError("n_new needs slots or max_new")
    if not _fits(device.index, (page_table, i32), (n_pages, i32), (seq_lens, i32), (free_pages, i32),
                 (free_state, i32), (n_new, i32), (slots, i32), (status, i32)):
        _check(device, ("page_table", page_table, i32), ("n_pages", n_pages, i32),
               ("seq_lens", seq_lens, i32), ("free_pages", free_pages, i32),
               ("free_state", free_state, i32), ("n_new", n_new, i32), ("slots", slots, i32),
               ("status", status, i32))
    if n_pages.numel() != B or seq_lens.numel() != B or free_state.numel() != 2 or \
            (n_new is not None and n_new.numel() != B) or (status is not None and status.numel() < 1) or \
            (slots is not None and (slots.dim() != 2 or slots.shape[0] != B or
                                    max_new not in (None, slots.shape[1]))):
        raise ValueError("n_pages, seq_lens and n_new must be [B], free_state [2], slots "
                         "[B][max_new], status one word")
    Z = _pack_resize(B, width, free_pages.numel(), 0 if slots is None else slots.shape[1],
                     _address(n_new), _address(slots), _address(status), _stream(device) or 0)
    with _on(device):
        rc = _fast.kv_resize(page_table.data_ptr(), n_pages.data_ptr(), seq_lens.data_ptr(),
                             free_pages.data_ptr(), free_state.data_ptr(), page_tokens, Z)
    if rc != 0:
        raise AtlasError(rc, status_string(rc))
    return slots


class EventTimer:
    """Three torch CUDA events whose handles the library records around its main
    kernel and its merge: main_ms() and merge_ms() read them after a sync."""

    def __init__(self):
        self.ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
        for e in self.ev:  # torch creates the CUDA event on its first record
            e.record()
        self.handles = (ctypes.c_void_p * 3)(*[e.cuda_event for e in self.ev])

    def main_ms(self) -> float:
        return self.ev[0].elapsed_time(self.ev[1])

    def merge_ms(self) -> float:
        return self.ev[1].elapsed_time(self.ev[2])


def run_host(kind: str, q, k_pages, v_pages, page_table, seq_lens, n_q_heads, n_kv_heads,
             head_dim, page_tokens, scale, *, device="cuda", out_dtype=None, host_out=None,
             **kw):
    """End-to-end call on host tensors (ideally pinned): copies the inputs to the
    device on the current stream, runs the kernels, and copies the result back.
    Returns the host output tensor (``host_out`` if given)."""
    dev = [t.to(device, non_blocking=True) for t in (q, k_pages, v_pages, page_table, seq_lens)]
    call = cross if kind == "cross" else functools.partial(_call, kind)
    out = call(*dev, n_q_heads, n_kv_heads, head_dim, page_tokens, scale, out_dtype=out_dtype, **kw)
    if host_out is None:
        host_out = torch.empty(out.shape, dtype=out.dtype, pin_memory=True)
    host_out.copy_(out, non_blocking=True)
    torch.cuda.current_stream(out.device).synchronize()
    return host_out


from .pool import HotPagePool  # noqa: E402  (the pool binding uses the names above)
