"""Python binding for libarena_compaction.so (gfx950).

Argument marshalling only: every step of the compaction runs in the HIP
kernels behind the C-ABI declared in include/arena_compaction.h.  PyTorch is
used for device memory and streams.  Importing this module fails loudly if
the library has not been built -- there is no CPU fallback.

Tables are torch tensors on the GPU: offset and size as int64 holding the
unsigned 64-bit values, live as uint8 (or None: every entry live), pinned as
uint8 (or None: nothing pinned).  Handles
and new offsets are int64 tensors holding unsigned values; an unmapped handle
reads back as -1 (UINT64_MAX).
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libarena_compaction.so")

DEFRAG_OK = 0
DEFRAG_EINVAL = -1
DEFRAG_EWORKSPACE = -2
DEFRAG_ENOPLAN = -3
DEFRAG_EHIP = -4
DEFRAG_ETIMEOUT = -5
DEFRAG_ENOFIT = -6
DEFRAG_ECAPACITY = -7
DEFRAG_ECORRUPT = -8
DEFRAG_ETOOBIG = -9
STATIC_SCRATCH_BYTES = 128 << 20   # DEFRAG_STATIC_SCRATCH_BYTES
REASONS = {0: "none", 1: "zero_size", 2: "misaligned", 3: "live_flag",
           4: "out_of_arena", 5: "overlap", 6: "argument", 7: "pinned_flag"}
U64_MAX = (1 << 64) - 1


class defrag_table(ctypes.Structure):
    _fields_ = [("offset_dev", ctypes.c_void_p), ("size_dev", ctypes.c_void_p),
                ("live_dev", ctypes.c_void_p), ("n", ctypes.c_uint64),
                ("pinned_dev", ctypes.c_void_p)]


class defrag_stats_t(ctypes.Structure):
    _fields_ = [(k, ctypes.c_uint64) for k in (
        "arena_bytes", "live_bytes", "free_bytes", "largest_hole", "hole_count",
        "live_blocks", "moved_blocks", "moved_bytes")] + [
        ("frag_free_over_largest_minus_1", ctypes.c_double),
        ("frag_one_minus_largest_over_free", ctypes.c_double),
        ("invalid_index", ctypes.c_uint64), ("invalid_reason", ctypes.c_int32),
        ("reserved", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {k: getattr(self, k) for k, _ in self._fields_ if k != "reserved"}


class defrag_tuning(ctypes.Structure):
    _fields_ = [("tile_bytes", ctypes.c_uint32), ("wg_per_cu", ctypes.c_uint32),
                ("nontemporal", ctypes.c_uint32), ("spin_limit_log2", ctypes.c_uint32),
                ("stall_every", ctypes.c_uint32), ("stall_sleeps", ctypes.c_uint32),
                ("stall_seed", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class defrag_move_report_t(ctypes.Structure):
    _fields_ = [("status", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("tiles", ctypes.c_uint64), ("late_tiles", ctypes.c_uint64),
                ("waited_tiles", ctypes.c_uint64), ("polls", ctypes.c_uint64)]


class defrag_plan_t(ctypes.Structure):
    _fields_ = [("magic", ctypes.c_uint64), ("epoch", ctypes.c_uint64),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64),
                ("n", ctypes.c_uint64), ("arena_bytes", ctypes.c_uint64),
                ("live_blocks", ctypes.c_uint64), ("pinned_blocks", ctypes.c_uint64),
                ("move_begin", ctypes.c_uint64), ("live_bytes", ctypes.c_uint64),
                ("n_tiles", ctypes.c_uint64), ("max_tiles", ctypes.c_uint64),
                ("max_blocks_per_tile", ctypes.c_uint64), ("whole_tiles", ctypes.c_uint64),
                ("request_bytes", ctypes.c_uint64), ("window_begin", ctypes.c_uint64),
                ("window_end", ctypes.c_uint64), ("window_hole", ctypes.c_uint64),
                ("state", ctypes.c_int32), ("device", ctypes.c_int32),
                ("tuning", defrag_tuning), ("stats", defrag_stats_t)]


class defrag_monitor_cfg(ctypes.Structure):
    _fields_ = [("warning_ratio", ctypes.c_double), ("critical_ratio", ctypes.c_double),
                ("frag_threshold", ctypes.c_double), ("next_request", ctypes.c_uint64),
                ("growth_bytes_per_s", ctypes.c_double)]


class defrag_monitor_report(ctypes.Structure):
    _fields_ = [("level", ctypes.c_int32), ("action", ctypes.c_int32),
                ("usage_ratio", ctypes.c_double),
                ("frag_free_over_largest_minus_1", ctypes.c_double),
                ("frag_one_minus_largest_over_free", ctypes.c_double),
                ("seconds_to_full", ctypes.c_double)]


class defrag_kv_cache(ctypes.Structure):
    _fields_ = [("arena_dev", ctypes.c_void_p), ("arena_bytes", ctypes.c_uint64),
                ("pages_dev", ctypes.c_void_p), ("page_stride", ctypes.c_uint64),
                ("lens_dev", ctypes.c_void_p), ("batch", ctypes.c_uint32),
                ("heads", ctypes.c_uint32), ("dim", ctypes.c_uint32), ("codes", ctypes.c_int32),
                ("n_invalid_dev", ctypes.c_void_p)]


class defrag_kv_append_args(ctypes.Structure):
    _fields_ = [("cache", ctypes.POINTER(defrag_kv_cache)), ("k_dev", ctypes.c_void_p),
                ("v_dev", ctypes.c_void_p), ("k_row", ctypes.c_int64), ("k_head", ctypes.c_int64),
                ("v_row", ctypes.c_int64), ("v_head", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("max_new", ctypes.c_uint32), ("tokens", ctypes.c_uint64),
                ("starts_dev", ctypes.c_void_p), ("weight_dev", ctypes.c_void_p),
                ("pos_dev", ctypes.c_void_p), ("first_pos_dev", ctypes.c_void_p),
                ("weight_stride", ctypes.c_uint64)]


class defrag_kv_attend_args(ctypes.Structure):
    _fields_ = [("cache", ctypes.POINTER(defrag_kv_cache)), ("q_dev", ctypes.c_void_p),
                ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("group", ctypes.c_uint32), ("tokens", ctypes.c_uint64),
                ("starts_dev", ctypes.c_void_p), ("max_new", ctypes.c_uint32),
                ("max_len", ctypes.c_uint32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_uint32), ("out_dev", ctypes.c_void_p),
                ("lse_dev", ctypes.c_void_p), ("weight_dev", ctypes.c_void_p),
                ("weight_stride", ctypes.c_uint64)]


class defrag_kv_evict_args(ctypes.Structure):
    _fields_ = [("cache", ctypes.POINTER(defrag_kv_cache)), ("budget", ctypes.c_uint32),
                ("max_len", ctypes.c_uint32), ("sink", ctypes.c_int32), ("recent", ctypes.c_int32),
                ("next_pos_dev", ctypes.c_void_p), ("weight_dev", ctypes.c_void_p),
                ("pos_dev", ctypes.c_void_p), ("weight_stride", ctypes.c_uint64),
                ("weight_out_dev", ctypes.c_void_p), ("pos_out_dev", ctypes.c_void_p),
                ("weight_out_stride", ctypes.c_uint64), ("lens_out_dev", ctypes.c_void_p)]


class defrag_kv_rotary_args(ctypes.Structure):
    _fields_ = [("append", ctypes.POINTER(defrag_kv_append_args)), ("freq_dev", ctypes.c_void_p),
                ("rotary_dim", ctypes.c_uint32), ("interleaved", ctypes.c_int32),
                ("token_pos_dev", ctypes.c_void_p), ("q_dev", ctypes.c_void_p),
                ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("out_dev", ctypes.c_void_p), ("out_row", ctypes.c_int64),
                ("out_head", ctypes.c_int64), ("q_heads", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class defrag_kv_terms(ctypes.Structure):
    _fields_ = [("mask_dev", ctypes.c_void_p), ("mask_words", ctypes.c_uint64),
                ("cap", ctypes.c_float), ("reserved", ctypes.c_uint32),
                ("slopes_dev", ctypes.c_void_p), ("pos_dev", ctypes.c_void_p),
                ("pos_stride", ctypes.c_uint64)]


class defrag_kv_accept_args(ctypes.Structure):
    _fields_ = [("cache", ctypes.POINTER(defrag_kv_cache)), ("tokens", ctypes.c_uint64),
                ("starts_dev", ctypes.c_void_p), ("max_new", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("path_dev", ctypes.c_void_p),
                ("path_stride", ctypes.c_uint64), ("kept_dev", ctypes.c_void_p),
                ("weight_dev", ctypes.c_void_p), ("pos_dev", ctypes.c_void_p),
                ("weight_stride", ctypes.c_uint64), ("lens_out_dev", ctypes.c_void_p)]


KV_PAGE_TOKENS = 64                # DEFRAG_KV_PAGE_TOKENS
KV_CODES = {torch.float8_e4m3fn: 0, torch.int8: 1}     # DEFRAG_KV_E4M3, DEFRAG_KV_INT8
KV_DTYPES = {torch.bfloat16: 0, torch.float16: 1}      # DEFRAG_KV_BF16, DEFRAG_KV_FP16

LEVELS = {0: "OK", 1: "WARNING", 2: "CRITICAL"}
ACTIONS = {0: "none", 1: "targeted", 2: "full", 3: "no_room"}


class defrag_compact_args(ctypes.Structure):
    _fields_ = [("table", ctypes.POINTER(defrag_table)), ("arena_bytes", ctypes.c_uint64),
                ("arena_dev", ctypes.c_void_p), ("request_bytes", ctypes.c_uint64),
                ("tuning", ctypes.POINTER(defrag_tuning)), ("ws_dev", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_size_t), ("new_offset_dev", ctypes.c_void_p),
                ("h_in_dev", ctypes.c_void_p), ("h_out_dev", ctypes.c_void_p),
                ("n_handles", ctypes.c_uint64), ("n_invalid_dev", ctypes.c_void_p),
                ("offset_out_dev", ctypes.c_void_p), ("size_out_dev", ctypes.c_void_p),
                ("live_out_dev", ctypes.c_void_p), ("pinned_out_dev", ctypes.c_void_p)]


# defrag_tile_t: one mover tile of a plan (defrag_plan_tiles)
TILE_DTYPE = np.dtype([("dst_begin", "<u8"), ("dst_end", "<u8"), ("shift_first", "<u8"),
                       ("first_block", "<u4"), ("last_block", "<u4"),
                       ("dep_lo", "<u4"), ("dep_hi", "<u4")])
assert TILE_DTYPE.itemsize == 40


class DefragError(RuntimeError):
    def __init__(self, code: int, what: str, stats: Optional[defrag_stats_t] = None):
        self.code = code
        self.invalid_index = None
        self.invalid_reason = None
        msg = f"{what}: {strerror(code)} ({code})"
        if stats is not None and stats.invalid_reason:
            self.invalid_index = int(stats.invalid_index)
            self.invalid_reason = int(stats.invalid_reason)
            msg += f"; entry {self.invalid_index}: {REASONS.get(self.invalid_reason, '?')}"
        super().__init__(msg)


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; "
            "g.build()'); there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    P, U, S = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_size_t
    L.defrag_workspace_bytes.argtypes = [U, U, U, ctypes.c_uint32]
    L.defrag_workspace_bytes.restype = S
    L.defrag_stats.argtypes = [ctypes.POINTER(defrag_table), U, P, S, P,
                               ctypes.POINTER(defrag_stats_t)]
    L.defrag_plan.argtypes = [ctypes.POINTER(defrag_table), U, ctypes.POINTER(defrag_tuning),
                              P, S, P, P, ctypes.POINTER(defrag_plan_t)]
    L.defrag_plan_targeted.argtypes = [ctypes.POINTER(defrag_table), U, U,
                                       ctypes.POINTER(defrag_tuning), P, S, P, P,
                                       ctypes.POINTER(defrag_plan_t)]
    L.defrag_first_fit.argtypes = [ctypes.POINTER(defrag_table), U, U, P, S, P,
                                   ctypes.POINTER(ctypes.c_uint64),
                                   ctypes.POINTER(defrag_stats_t)]
    L.defrag_move.argtypes = [P, U, ctypes.POINTER(defrag_plan_t), P, S, P]
    L.defrag_move_status.argtypes = [ctypes.POINTER(defrag_plan_t), P, P]
    L.defrag_move_report.argtypes = [ctypes.POINTER(defrag_plan_t), P, P,
                                     ctypes.POINTER(defrag_move_report_t)]
    L.defrag_plan_tiles.argtypes = [ctypes.POINTER(defrag_plan_t), P, S, P, U, P]
    L.defrag_remap.argtypes = [ctypes.POINTER(defrag_plan_t), P, S, P, P, U, P, P]
    L.defrag_commit.argtypes = [ctypes.POINTER(defrag_plan_t), P, S, P, P, P, P, P]
    L.defrag_compact.argtypes = [ctypes.POINTER(defrag_compact_args), P,
                                 ctypes.POINTER(defrag_plan_t), ctypes.POINTER(defrag_stats_t)]
    L.defrag_compact_static.argtypes = [ctypes.POINTER(defrag_compact_args), P,
                                        ctypes.POINTER(defrag_plan_t),
                                        ctypes.POINTER(defrag_stats_t)]
    L.defrag_monitor.argtypes = [ctypes.POINTER(defrag_stats_t), ctypes.POINTER(defrag_monitor_cfg),
                                 ctypes.POINTER(defrag_monitor_report)]
    L.defrag_kv_page_bytes.argtypes = [ctypes.c_uint32, ctypes.c_uint32]
    L.defrag_kv_append.argtypes = [ctypes.POINTER(defrag_kv_append_args), P]
    L.defrag_kv_attend_workspace_bytes.argtypes = [ctypes.POINTER(defrag_kv_attend_args)]
    L.defrag_kv_attend.argtypes = [ctypes.POINTER(defrag_kv_attend_args), P, S, P]
    L.defrag_kv_evict_workspace_bytes.argtypes = [ctypes.POINTER(defrag_kv_evict_args)]
    L.defrag_kv_evict.argtypes = [ctypes.POINTER(defrag_kv_evict_args), P, S, P]
    L.defrag_kv_append_rotary.argtypes = [ctypes.POINTER(defrag_kv_rotary_args), P]
    L.defrag_kv_attend_terms_workspace_bytes.argtypes = [ctypes.POINTER(defrag_kv_attend_args),
                                                         ctypes.POINTER(defrag_kv_terms)]
    L.defrag_kv_attend_terms.argtypes = [ctypes.POINTER(defrag_kv_attend_args),
                                         ctypes.POINTER(defrag_kv_terms), P, S, P]
    L.defrag_kv_accept.argtypes = [ctypes.POINTER(defrag_kv_accept_args), P]
    for f in ("defrag_kv_page_bytes", "defrag_kv_attend_workspace_bytes",
              "defrag_kv_attend_terms_workspace_bytes", "defrag_kv_evict_workspace_bytes"):
        getattr(L, f).restype = S
    L.defrag_strerror.argtypes = [ctypes.c_int]
    L.defrag_strerror.restype = ctypes.c_char_p
    for f in ("defrag_stats", "defrag_first_fit", "defrag_plan", "defrag_plan_targeted",
              "defrag_move", "defrag_monitor", "defrag_compact", "defrag_compact_static",
              "defrag_move_status", "defrag_move_report", "defrag_plan_tiles",
              "defrag_remap", "defrag_commit", "defrag_kv_append", "defrag_kv_attend",
              "defrag_kv_evict", "defrag_kv_append_rotary", "defrag_kv_attend_terms",
              "defrag_kv_accept"):
        getattr(L, f).restype = ctypes.c_int
    return L


lib = _load()

EXPORTS = ("defrag_workspace_bytes", "defrag_stats", "defrag_first_fit", "defrag_plan",
           "defrag_plan_targeted",
           "defrag_move",
           "defrag_move_status", "defrag_move_report", "defrag_plan_tiles", "defrag_remap",
           "defrag_commit",
           "defrag_compact", "defrag_compact_static", "defrag_monitor",
           "defrag_kv_page_bytes", "defrag_kv_append", "defrag_kv_attend_workspace_bytes",
           "defrag_kv_attend", "defrag_kv_evict_workspace_bytes", "defrag_kv_evict",
           "defrag_kv_append_rotary", "defrag_kv_attend_terms_workspace_bytes",
           "defrag_kv_attend_terms", "defrag_kv_accept", "defrag_strerror")


def strerror(code: int) -> str:
    return lib.defrag_strerror(int(code)).decode()


def _ptr(t: Optional[torch.Tensor]):
    """The device address of t (an int: every pointer argument and field is
    declared c_void_p, which takes one as it is)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        raise ValueError("device arguments must be contiguous GPU tensors")
    return t.data_ptr()


def _need(t: Optional[torch.Tensor], dtype: torch.dtype, n: int, what: str) -> None:
    """Raise unless t is None or a tensor of dtype with at least n elements
    (the kernels write or read that many; a shorter buffer would be overrun)."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise ValueError(f"{what}: expected a {dtype} tensor")
    if t.numel() < n:
        raise ValueError(f"{what}: {t.numel()} elements, {n} needed")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_table(offset: torch.Tensor, size: torch.Tensor, live: Optional[torch.Tensor],
               pinned: Optional[torch.Tensor] = None) -> defrag_table:
    n = offset.numel()
    _need(offset, torch.int64, 0, "offset")
    _need(size, torch.int64, n, "size")
    _need(live, torch.uint8, n, "live")
    _need(pinned, torch.uint8, n, "pinned")
    return defrag_table(_ptr(offset) if n else None, _ptr(size) if n else None,
                        _ptr(live) if (live is not None and n) else None, n,
                        _ptr(pinned) if (pinned is not None and n) else None)


def defrag_workspace_bytes(n: int, arena_bytes: int, tile_bytes: int = 0,
                           max_pinned: int = 0) -> int:
    return int(lib.defrag_workspace_bytes(n, max_pinned, arena_bytes, tile_bytes))


def workspace(n: int, arena_bytes: int, tile_bytes: int = 0, device=None,
              max_pinned: int = 0) -> torch.Tensor:
    """Allocate a workspace tensor (torch allocations are 256-byte aligned)."""
    nb = defrag_workspace_bytes(n, arena_bytes, tile_bytes, max_pinned)
    if nb == 0:
        raise DefragError(DEFRAG_EINVAL, "defrag_workspace_bytes")
    return torch.empty(nb, dtype=torch.uint8, device=device or "cuda")


def defrag_stats(offset, size, live, arena_bytes: int, ws: torch.Tensor,
                 stream=None, pinned=None) -> defrag_stats_t:
    t = make_table(offset, size, live, pinned)
    out = defrag_stats_t()
    rc = lib.defrag_stats(ctypes.byref(t), arena_bytes, _ptr(ws), ws.numel(), _stream(stream),
                          ctypes.byref(out))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_stats", out)
    return out


def defrag_first_fit(offset, size, live, arena_bytes: int, request_bytes: int,
                     ws: torch.Tensor, stream=None, pinned=None):
    """(offset, stats): the offset first fit gives the request, or None when
    no hole holds it (DEFRAG_ENOFIT)."""
    t = make_table(offset, size, live, pinned)
    out = ctypes.c_uint64()
    st = defrag_stats_t()
    rc = lib.defrag_first_fit(ctypes.byref(t), arena_bytes, request_bytes, _ptr(ws), ws.numel(),
                              _stream(stream), ctypes.byref(out), ctypes.byref(st))
    if rc == DEFRAG_ENOFIT:
        return None, st
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_first_fit", st)
    return int(out.value), st


def defrag_plan(offset, size, live, arena_bytes: int, ws: torch.Tensor,
                new_offset: Optional[torch.Tensor] = None,
                tuning: Optional[defrag_tuning] = None, stream=None,
                pinned: Optional[torch.Tensor] = None) -> defrag_plan_t:
    _need(new_offset, torch.int64, offset.numel(), "new_offset")
    t = make_table(offset, size, live, pinned)
    plan = defrag_plan_t()
    rc = lib.defrag_plan(ctypes.byref(t), arena_bytes,
                         ctypes.byref(tuning) if tuning is not None else None,
                         _ptr(ws), ws.numel(), _stream(stream),
                         _ptr(new_offset) if new_offset is not None and new_offset.numel() else None,
                         ctypes.byref(plan))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_plan", plan.stats)
    return plan


def defrag_plan_targeted(offset, size, live, arena_bytes: int, request_bytes: int,
                         ws: torch.Tensor, new_offset: Optional[torch.Tensor] = None,
                         tuning: Optional[defrag_tuning] = None, stream=None,
                         pinned: Optional[torch.Tensor] = None) -> defrag_plan_t:
    """Raises DefragError with code DEFRAG_ENOFIT when no window fits."""
    _need(new_offset, torch.int64, offset.numel(), "new_offset")
    t = make_table(offset, size, live, pinned)
    plan = defrag_plan_t()
    rc = lib.defrag_plan_targeted(ctypes.byref(t), arena_bytes, request_bytes,
                                  ctypes.byref(tuning) if tuning is not None else None,
                                  _ptr(ws), ws.numel(), _stream(stream),
                                  _ptr(new_offset) if new_offset is not None and new_offset.numel()
                                  else None, ctypes.byref(plan))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_plan_targeted", plan.stats)
    return plan


def defrag_move(arena: torch.Tensor, plan: defrag_plan_t, ws: torch.Tensor, stream=None) -> None:
    _need(arena, torch.uint8, 0, "arena")
    rc = lib.defrag_move(_ptr(arena) if arena.numel() else None, arena.numel(),
                         ctypes.byref(plan), _ptr(ws), ws.numel(), _stream(stream))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_move")


def defrag_move_status(plan: defrag_plan_t, ws: torch.Tensor, stream=None) -> int:
    return int(lib.defrag_move_status(ctypes.byref(plan), _ptr(ws), _stream(stream)))


def defrag_move_report(plan: defrag_plan_t, ws: torch.Tensor, stream=None) -> defrag_move_report_t:
    """The move's outcome (status) and the mover's wait counters."""
    out = defrag_move_report_t()
    rc = lib.defrag_move_report(ctypes.byref(plan), _ptr(ws), _stream(stream), ctypes.byref(out))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_move_report")
    return out


def defrag_plan_tiles(plan: defrag_plan_t, ws: torch.Tensor, stream=None) -> np.ndarray:
    """The plan's mover tiles as a structured array of TILE_DTYPE."""
    n = int(plan.n_tiles)
    out = np.zeros(n, dtype=TILE_DTYPE)
    rc = lib.defrag_plan_tiles(ctypes.byref(plan), _ptr(ws), ws.numel(),
                               ctypes.c_void_p(out.ctypes.data) if n else None, n,
                               _stream(stream))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_plan_tiles")
    return out


def defrag_remap(plan: defrag_plan_t, ws: torch.Tensor, h_in: torch.Tensor,
                 h_out: Optional[torch.Tensor] = None,
                 n_invalid: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    _need(h_in, torch.int64, 0, "h_in")
    if h_out is None:
        h_out = torch.empty_like(h_in)
    H = h_in.numel()
    _need(h_out, torch.int64, H, "h_out")
    _need(n_invalid, torch.int64, 1, "n_invalid")
    rc = lib.defrag_remap(ctypes.byref(plan), _ptr(ws), ws.numel(),
                          _ptr(h_in) if H else None, _ptr(h_out) if H else None, H,
                          _ptr(n_invalid), _stream(stream))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_remap")
    return h_out


def defrag_commit(plan: defrag_plan_t, ws: torch.Tensor, offset_out=None, size_out=None,
                  live_out=None, stream=None, pinned_out=None) -> None:
    m = int(plan.live_blocks)
    _need(offset_out, torch.int64, m, "offset_out")
    _need(size_out, torch.int64, m, "size_out")
    _need(live_out, torch.uint8, m, "live_out")
    _need(pinned_out, torch.uint8, m, "pinned_out")
    rc = lib.defrag_commit(ctypes.byref(plan), _ptr(ws), ws.numel(), _ptr(offset_out),
                           _ptr(size_out), _ptr(live_out), _ptr(pinned_out), _stream(stream))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_commit")


def _compact_args(offset, size, live, arena_bytes, arena, ws, request_bytes, new_offset, handles,
                  h_out, n_invalid, offset_out, size_out, live_out, pinned_out, tuning, pinned):
    """The defrag_compact_args of a call, its argument checks, and the
    buffers it points at (kept alive with it)."""
    _need(arena, torch.uint8, 0, "arena")
    _need(new_offset, torch.int64, offset.numel(), "new_offset")
    H = 0 if handles is None else handles.numel()
    if handles is not None:
        _need(handles, torch.int64, 0, "handles")
        if h_out is None:
            h_out = torch.empty_like(handles)
        _need(h_out, torch.int64, H, "h_out")
    _need(n_invalid, torch.int64, 1, "n_invalid")
    for o, dt, name in ((offset_out, torch.int64, "offset_out"), (size_out, torch.int64, "size_out"),
                        (live_out, torch.uint8, "live_out"), (pinned_out, torch.uint8, "pinned_out")):
        _need(o, dt, 0, name)
    t = make_table(offset, size, live, pinned)
    a = defrag_compact_args(
        ctypes.pointer(t), arena_bytes, _ptr(arena) if arena.numel() else None, request_bytes,
        ctypes.pointer(tuning) if tuning is not None else None,
        _ptr(ws) if ws is not None else None, ws.numel() if ws is not None else 0,
        _ptr(new_offset) if new_offset is not None and new_offset.numel() else None,
        _ptr(handles) if H else None, _ptr(h_out) if H else None, H, _ptr(n_invalid),
        _ptr(offset_out) if offset_out is not None and offset_out.numel() else None,
        _ptr(size_out) if size_out is not None and size_out.numel() else None,
        _ptr(live_out) if live_out is not None and live_out.numel() else None,
        _ptr(pinned_out) if pinned_out is not None and pinned_out.numel() else None)
    return a, (t, h_out)


def defrag_compact(offset, size, live, arena_bytes: int, arena: torch.Tensor, ws: torch.Tensor,
                   request_bytes: int = 0, new_offset: Optional[torch.Tensor] = None,
                   handles: Optional[torch.Tensor] = None, h_out: Optional[torch.Tensor] = None,
                   n_invalid: Optional[torch.Tensor] = None, offset_out=None, size_out=None,
                   live_out=None, pinned_out=None, tuning: Optional[defrag_tuning] = None,
                   stream=None, pinned=None, after: Optional[bool] = None):
    """Plan, move, remap, commit and the post-check in one C-ABI call.
    after (default: whenever offset_out and size_out are given) asks for the
    post-move statistics.  Returns (plan, post-move stats or None).
    offset_out, size_out, live_out and pinned_out need one element per live
    block, which is known only once the plan has run: neither this function
    nor the library can check their length."""
    if after is None:
        after = offset_out is not None and size_out is not None
    a, keep = _compact_args(offset, size, live, arena_bytes, arena, ws, request_bytes, new_offset,
                            handles, h_out, n_invalid, offset_out, size_out, live_out, pinned_out,
                            tuning, pinned)
    plan = defrag_plan_t()
    post = defrag_stats_t() if after else None
    rc = lib.defrag_compact(ctypes.byref(a), _stream(stream), ctypes.byref(plan),
                            ctypes.byref(post) if after else None)
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_compact", plan.stats if rc == DEFRAG_EINVAL else None)
    return plan, post


def defrag_compact_static(offset, size, live, arena_bytes: int, arena: torch.Tensor,
                          request_bytes: int = 0, new_offset: Optional[torch.Tensor] = None,
                          handles: Optional[torch.Tensor] = None,
                          h_out: Optional[torch.Tensor] = None,
                          n_invalid: Optional[torch.Tensor] = None, offset_out=None,
                          size_out=None, live_out=None, pinned_out=None,
                          tuning: Optional[defrag_tuning] = None, stream=None, pinned=None,
                          after: Optional[bool] = None):
    """defrag_compact with the library's static scratch as its workspace:
    the library allocates nothing and creates no stream or event for it
    (every step runs on `stream`).  Returns (plan, post-move stats or None);
    DEFRAG_ETOOBIG when the table needs more than the scratch holds."""
    if after is None:
        after = offset_out is not None and size_out is not None
    a, keep = _compact_args(offset, size, live, arena_bytes, arena, None, request_bytes,
                            new_offset, handles, h_out, n_invalid, offset_out, size_out, live_out,
                            pinned_out, tuning, pinned)
    plan = defrag_plan_t()
    post = defrag_stats_t() if after else None
    rc = lib.defrag_compact_static(ctypes.byref(a), _stream(stream), ctypes.byref(plan),
                                   ctypes.byref(post) if after else None)
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_compact_static",
                          plan.stats if rc == DEFRAG_EINVAL else None)
    return plan, post


def defrag_monitor(stats: defrag_stats_t, warning_ratio: float = 0.85,
                   critical_ratio: float = 0.95, frag_threshold: float = 0.0,
                   next_request: int = 0, growth_bytes_per_s: float = 0.0) -> defrag_monitor_report:
    cfg = defrag_monitor_cfg(warning_ratio, critical_ratio, frag_threshold, next_request,
                             growth_bytes_per_s)
    out = defrag_monitor_report()
    rc = lib.defrag_monitor(ctypes.byref(stats), ctypes.byref(cfg), ctypes.byref(out))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_monitor")
    return out


def _kv_int(x: int, what: str, least: int = 0, most: int = 0xFFFFFFFF) -> int:
    """x where it fits its field, to which ctypes would cut it (heads, a length
    or a budget of 2^32 + n would be n); refused as the library refuses sizes."""
    if not least <= x <= most:
        raise DefragError(DEFRAG_EINVAL, f"{what} = {x}")
    return x


def defrag_kv_page_bytes(heads: int, dim: int) -> int:
    """Bytes of a cache page (64 tokens of every head), a multiple of 32."""
    nb = int(lib.defrag_kv_page_bytes(_kv_int(heads, "heads"), _kv_int(dim, "dim")))
    if nb == 0:
        raise DefragError(DEFRAG_EINVAL, "defrag_kv_page_bytes")
    return nb


def _kv_ptr(t, dtype: torch.dtype, n: int, dev: int, what: str) -> int:
    """The address of a contiguous tensor of dtype on GPU dev with at least n
    elements (one test on the way: a call of a few microseconds has a dozen)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or dev < 0 \
            or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous {dtype} tensor on the arena's GPU")
    if t.numel() < n:
        raise ValueError(f"{what}: {t.numel()} elements, {n} needed")
    return t.data_ptr()


def _kv_cache(arena, pages, lens, heads, dim, codes, n_invalid) -> defrag_kv_cache:
    """The defrag_kv_cache of a call and the checks of its tensors."""
    kind = KV_CODES.get(codes)
    if kind is None:
        raise ValueError(f"codes: {codes}, expected one of {list(KV_CODES)}")
    dev = arena.get_device() if isinstance(arena, torch.Tensor) else -1
    if dev >= 0 and dev != torch.cuda.current_device():
        raise ValueError(f"arena: on GPU {dev}, the current one is {torch.cuda.current_device()}")
    if not isinstance(pages, torch.Tensor) or pages.dim() != 2:
        raise ValueError("pages: [batch, pages] expected")
    batch, stride = pages.shape
    if not isinstance(lens, torch.Tensor) or lens.dtype is not torch.int32 or lens.dim() != 1 \
            or lens.shape[0] != batch:
        raise ValueError("lens: int32 [batch] expected, as many as pages has rows")
    if (heads | dim) >> 32:
        _kv_int(heads, "heads"), _kv_int(dim, "dim")
    return defrag_kv_cache(_kv_ptr(arena, torch.uint8, 0, dev, "arena"), arena.numel(),
                           _kv_ptr(pages, torch.int64, 0, dev, "pages"), stride,
                           _kv_ptr(lens, torch.int32, 0, dev, "lens"), batch, heads, dim, kind,
                           None if n_invalid is None else
                           _kv_ptr(n_invalid, torch.int64, 1, dev, "n_invalid"))


def _kv_rows(t, arena, what: str, dim: Optional[int] = None, heads: Optional[int] = None) -> None:
    """A [tokens, heads, dim] tensor of 16 bits whose last dimension is dense."""
    if not isinstance(t, torch.Tensor) or t.dtype not in KV_DTYPES:
        raise ValueError(f"{what}: expected a tensor of {list(KV_DTYPES)}")
    if t.dim() != 3 or (dim is not None and t.shape[2] != dim) or \
            (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{what}: shape {tuple(t.shape)}")
    if not t.is_cuda or t.get_device() != arena.get_device() or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{what}: expected a tensor on the arena's GPU with a dense last dimension")


def _kv_plane(t, arena, dtype, shape, what: str) -> int:
    """Checks a contiguous [batch, heads, places] tensor; its number of places."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.dim() != 3 \
            or t.shape[:2] != shape or not t.is_contiguous() or t.get_device() != arena.get_device():
        raise ValueError(f"{what}: expected a contiguous {dtype} [{shape[0]}, {shape[1]}, places] "
                         "on the arena's GPU")
    return t.shape[2]


def _kv_new(starts, max_new, tokens: int, batch: int, arena) -> int:
    """Checks starts and gives max_new its default."""
    if starts is None:
        if tokens != batch:
            raise ValueError(f"starts: {tokens} tokens of {batch} sequences need it")
        return min(1, tokens)
    _kv_ptr(starts, torch.int32, batch + 1, arena.get_device(), "starts")
    return tokens if max_new is None else _kv_int(min(int(max_new), tokens), "max_new")


def _kv_stream(stream, dev: int) -> int:
    """The stream's handle.  The current one is asked for as a handle:
    torch.cuda.current_stream() makes an object first, for 3 us."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _kv_new_empty(like: torch.Tensor, shape, stream) -> torch.Tensor:
    """Memory for one call, from the pool of the stream that it runs on."""
    if stream is None:
        return like.new_empty(shape)
    with torch.cuda.stream(stream):
        return like.new_empty(shape)


def _kv_scratch(need: int, ws, arena, stream, what: str):
    """(workspace tensor, address, bytes) of a call that needs `need` bytes."""
    if need == 0:
        raise DefragError(DEFRAG_EINVAL, what)
    if ws is not None:
        return ws, _kv_ptr(ws, torch.uint8, 0, arena.get_device(), "ws"), ws.numel()
    if need == 1:   # none
        return None, None, 0
    ws = _kv_new_empty(arena, (need,), stream)
    return ws, ws.data_ptr(), need


def _opt(t):
    return None if t is None else t.data_ptr()


def _kv_append_args(arena, pages, lens, k, v, codes, starts, max_new, weight, pos, first_pos, n_invalid):
    """The checked arguments of an append."""
    _kv_rows(k, arena, "k")
    tokens, heads, dim = k.shape
    _kv_rows(v, arena, "v", dim, heads)
    if v.shape[0] != tokens or v.dtype != k.dtype:
        raise ValueError("v: another shape or dtype than k")
    c = _kv_cache(arena, pages, lens, heads, dim, codes, n_invalid)
    batch = c.batch
    most = _kv_new(starts, max_new, tokens, batch, arena)
    cap = _kv_plane(weight, arena, torch.float32, (batch, heads), "weight")
    cap2 = _kv_plane(pos, arena, torch.int32, (batch, heads), "pos")
    if weight is not None and pos is not None and cap != cap2:
        raise ValueError("pos: another number of places than weight")
    if first_pos is not None:
        _kv_ptr(first_pos, torch.int32, batch, arena.get_device(), "first_pos")
    return defrag_kv_append_args(ctypes.pointer(c), k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1),
                                 v.stride(0), v.stride(1), KV_DTYPES[k.dtype], most, tokens,
                                 _opt(starts), _opt(weight), _opt(pos), _opt(first_pos), cap or cap2)


def defrag_kv_append(arena, pages, lens, k, v, codes, starts=None, max_new: Optional[int] = None,
                     weight=None, pos=None, first_pos=None, n_invalid=None, stream=None) -> None:
    """Quantise new tokens' keys and values [tokens, heads, dim] into the
    pages of the cache.  arena: uint8; pages: int64 [batch, pages] byte offsets
    in it; lens: int32 [batch], the lengths before the call (not changed);
    codes: torch.float8_e4m3fn or torch.int8; starts: int32 [batch + 1], the
    first new token of each sequence (None: one a sequence), at most max_new
    each.  weight (float32) and pos (int32), [batch, heads, places], get 0 and
    first_pos[b] + the token's number (default: its place)."""
    a = _kv_append_args(arena, pages, lens, k, v, codes, starts, max_new, weight, pos, first_pos, n_invalid)
    rc = lib.defrag_kv_append(a, _kv_stream(stream, arena.get_device()))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_kv_append")


def defrag_kv_append_rotary(arena, pages, lens, k, v, codes, freq, q=None, q_out=None, interleaved: bool = False,
                            starts=None, max_new: Optional[int] = None, token_pos=None, weight=None, pos=None,
                            first_pos=None, n_invalid=None, stream=None):
    """defrag_kv_append with keys that are rotated by their positions on the
    way.  freq: float64 [pairs], the radians a position that each pair turns
    by; pairs are (i, i + pairs), or with interleaved (2 i, 2 i + 1), of the
    first 2 * pairs dimensions.  token_pos: int32 [tokens], positions (default:
    first_pos[b] + the token's number), which pos gets.  q [tokens, query
    heads, dim], of k's type, is rotated likewise into q_out, which is returned
    (default: new memory; q itself: in place); tokens that belong to no
    sequence are left out."""
    a = _kv_append_args(arena, pages, lens, k, v, codes, starts, max_new, weight, pos, first_pos, n_invalid)
    dev, (tokens, _, dim) = arena.get_device(), k.shape
    if not isinstance(freq, torch.Tensor) or freq.dim() != 1:
        raise ValueError("freq: float64 [pairs] expected")
    if token_pos is not None:
        _kv_ptr(token_pos, torch.int32, tokens, dev, "token_pos")
    heads = 0
    if q is not None:
        _kv_rows(q, arena, "q", dim)
        if q.shape[0] != tokens or q.dtype != k.dtype:
            raise ValueError("q: other tokens or another dtype than k")
        heads = q.shape[1]
        if q_out is None:
            q_out = _kv_new_empty(q, q.shape, stream)
        else:
            _kv_rows(q_out, arena, "q_out", dim, heads)
            if q_out.shape[0] != tokens or q_out.dtype != q.dtype:
                raise ValueError("q_out: another shape or dtype than q")
    elif q_out is not None:
        raise ValueError("q_out: nothing to rotate without q")
    r = defrag_kv_rotary_args(ctypes.pointer(a), _kv_ptr(freq, torch.float64, 0, dev, "freq"),
                              _kv_int(2 * freq.shape[0], "rotated dimensions"), 1 if interleaved else 0,
                              _opt(token_pos), _opt(q), q.stride(0) if heads else 0, q.stride(1) if heads else 0,
                              _opt(q_out), q_out.stride(0) if heads else 0, q_out.stride(1) if heads else 0, heads, 0)
    rc = lib.defrag_kv_append_rotary(r, _kv_stream(stream, dev))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_kv_append_rotary")
    return q_out


def _kv_attend_args(arena, pages, lens, q, heads, codes, starts, max_new, max_len, scale, out, lse, weight, n_invalid,
                    stream):
    """(the checked arguments of an attention, its output)."""
    _kv_rows(q, arena, "q")
    tokens, q_heads, dim = q.shape
    if heads < 1 or q_heads % heads:
        raise ValueError(f"q: {q_heads} heads over {heads} key/value heads")
    c = _kv_cache(arena, pages, lens, heads, dim, codes, n_invalid)
    batch = c.batch
    most = _kv_new(starts, max_new, tokens, batch, arena)
    if max_len is None:
        max_len = pages.shape[1] * KV_PAGE_TOKENS
    dev = arena.get_device()
    if out is None:
        out = _kv_new_empty(q, q.shape, stream)
    elif not isinstance(out, torch.Tensor) or out.shape != q.shape:
        raise ValueError("out: another shape than q")
    else:
        _kv_ptr(out, q.dtype, 0, dev, "out")
    if lse is not None:
        _kv_ptr(lse, torch.float32, tokens * q_heads, dev, "lse")
    cap = _kv_plane(weight, arena, torch.float32, (batch, heads), "weight")
    if (max_len | q_heads) >> 32:
        _kv_int(max_len, "max_len"), _kv_int(q_heads, "query heads")
    return defrag_kv_attend_args(ctypes.pointer(c), q.data_ptr(), q.stride(0), q.stride(1),
                                 KV_DTYPES[q.dtype], q_heads // heads, tokens, _opt(starts), most,
                                 max_len, dim ** -0.5 if scale is None else scale, 0, out.data_ptr(),
                                 _opt(lse), _opt(weight), cap), out


def defrag_kv_attend(arena, pages, lens, q, heads: int, codes, starts=None,
                     max_new: Optional[int] = None, max_len: Optional[int] = None,
                     scale: Optional[float] = None, out=None, lse=None, weight=None,
                     n_invalid=None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of the newest tokens' queries [tokens, query heads, dim] over
    the cache; returns out, of q's type.  lens counts the new tokens too (call
    defrag_kv_append first).  `heads` key/value heads, each read by an equal
    share of the query heads.  max_len: no length exceeds it (default: what
    the page table holds); scale: default dim ** -0.5.  lse: float32 [tokens,
    query heads]; weight: float32 [batch, heads, places], increased by the
    weight each cached token receives.  ws: workspace, allocated if None."""
    a, out = _kv_attend_args(arena, pages, lens, q, heads, codes, starts, max_new, max_len, scale, out, lse, weight,
                             n_invalid, stream)
    need = lib.defrag_kv_attend_workspace_bytes(a)
    ws, at, size = _kv_scratch(need, ws, arena, stream, "defrag_kv_attend")
    rc = lib.defrag_kv_attend(a, at, size, _kv_stream(stream, arena.get_device()))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_kv_attend")
    return out


def defrag_kv_attend_terms(arena, pages, lens, q, heads: int, codes, mask=None, cap: Optional[float] = None,
                           slopes=None, pos=None, starts=None, max_new: Optional[int] = None,
                           max_len: Optional[int] = None, scale: Optional[float] = None, out=None, lse=None,
                           weight=None, n_invalid=None, ws: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """defrag_kv_attend with terms beside causal softmax.  mask: int64 [tokens,
    words], bit j % 64 of word j / 64 says that the token sees new token j of
    its sequence (it sees all older ones; max_new is then at most what the words
    hold, which is its default); cap: scores become cap * tanh(score
    / cap); slopes: float32 [query heads], times the cached token's position
    less the query's, is added to a score; pos: int32 [batch, heads, places],
    the positions (default: the places), a multiple of 64 of them and at least
    max_len."""
    words = 0
    if cap and not ctypes.c_float(cap).value:   # the field's 0 is none
        raise DefragError(DEFRAG_EINVAL, f"cap = {cap}")
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or mask.dim() != 2:
            raise ValueError("mask: int64 [tokens, words] expected")
        words = mask.shape[1]
        if max_new is None:
            max_new = 64 * words
    a, out = _kv_attend_args(arena, pages, lens, q, heads, codes, starts, max_new, max_len, scale, out, lse, weight,
                             n_invalid, stream)
    dev, (tokens, q_heads, _) = arena.get_device(), q.shape
    if mask is not None:
        if mask.shape[0] != tokens:
            raise ValueError(f"mask: {mask.shape[0]} rows of {tokens} tokens")
        _kv_ptr(mask, torch.int64, 0, dev, "mask")
    if slopes is not None:
        _kv_ptr(slopes, torch.float32, q_heads, dev, "slopes")
    c = a.cache.contents
    places = _kv_plane(pos, arena, torch.int32, (c.batch, c.heads), "pos")
    t = defrag_kv_terms(_opt(mask), words, 0.0 if cap is None else cap, 0, _opt(slopes), _opt(pos), places)
    need = lib.defrag_kv_attend_terms_workspace_bytes(a, t)
    ws, at, size = _kv_scratch(need, ws, arena, stream, "defrag_kv_attend_terms")
    rc = lib.defrag_kv_attend_terms(a, t, at, size, _kv_stream(stream, dev))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_kv_attend_terms")
    return out


def defrag_kv_accept(arena, pages, lens, path, kept, lens_out, heads: int, dim: int, codes, starts=None,
                     max_new: Optional[int] = None, weight=None, pos=None, n_invalid=None, stream=None) -> None:
    """Keep the accepted path of each sequence's drafted tokens, its last ones
    (lens counts them; starts: int32 [batch + 1], as in append, None: one
    each).  path: int32 [batch, most], ascending numbers of drafted tokens, of
    which kept (int32 [batch]) count; they move to the places behind the
    sequence's other tokens, with their weight (float32) and pos (int32),
    [batch, heads, places].  lens_out: int32 [batch], the new lengths, memory
    of its own."""
    c = _kv_cache(arena, pages, lens, heads, dim, codes, n_invalid)
    dev, batch = arena.get_device(), c.batch
    tokens = batch if starts is None else 1 << 29   # (none of them is read: starts may begin anywhere)
    most = _kv_new(starts, max_new, tokens, batch, arena)
    if not isinstance(path, torch.Tensor) or path.dim() != 2 or path.shape[0] != batch:
        raise ValueError("path: int32 [batch, most] expected")
    cap = _kv_plane(weight, arena, torch.float32, (batch, heads), "weight")
    cap2 = _kv_plane(pos, arena, torch.int32, (batch, heads), "pos")
    if weight is not None and pos is not None and cap != cap2:
        raise ValueError("pos: another number of places than weight")
    a = defrag_kv_accept_args(ctypes.pointer(c), tokens, _opt(starts), most, 0,
                              _kv_ptr(path, torch.int32, 0, dev, "path"), path.shape[1],
                              _kv_ptr(kept, torch.int32, batch, dev, "kept"), _opt(weight), _opt(pos), cap or cap2,
                              _kv_ptr(lens_out, torch.int32, batch, dev, "lens_out"))
    rc = lib.defrag_kv_accept(a, _kv_stream(stream, dev))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_kv_accept")


def defrag_kv_evict(arena, pages, lens, budget: int, weight, pos, weight_out, pos_out, lens_out,
                    dim: int, codes, sink: int = 0, recent: int = 0, next_pos=None,
                    max_len: Optional[int] = None, n_invalid=None,
                    ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """Keep `budget` (a multiple of 64) tokens of every (sequence, head): those
    whose position is below sink or at least next_pos - recent, then those of
    largest weight; they end in the first budget / 64 pages.  weight (float32)
    and pos (int32): [batch, heads, places]; weight_out, pos_out and lens_out
    (int32 [batch]) receive the result; weight_out may be weight and pos_out
    pos, lens_out has to be memory of its own.  next_pos: int32 [batch] (default:
    lens); max_len: no length exceeds it (default: what table and planes
    hold)."""
    if not isinstance(weight, torch.Tensor) or weight.dim() != 3:
        raise ValueError("weight: [batch, heads, places] expected")
    heads = weight.shape[1]
    c = _kv_cache(arena, pages, lens, heads, dim, codes, n_invalid)
    batch = c.batch
    cap = _kv_plane(weight, arena, torch.float32, (batch, heads), "weight")
    if _kv_plane(pos, arena, torch.int32, (batch, heads), "pos") != cap or pos is None:
        raise ValueError("pos: another shape than weight")
    cap_out = _kv_plane(weight_out, arena, torch.float32, (batch, heads), "weight_out")
    if _kv_plane(pos_out, arena, torch.int32, (batch, heads), "pos_out") != cap_out or pos_out is None:
        raise ValueError("pos_out: another shape than weight_out")
    dev = arena.get_device()
    if weight_out is None:
        raise ValueError("weight_out: needed, with pos_out and lens_out")
    if next_pos is None:
        next_pos = lens
    if max_len is None:
        max_len = min(pages.shape[1] * KV_PAGE_TOKENS, cap)
    if (budget | max_len | (sink + 0x80000000) | (recent + 0x80000000)) >> 32:
        _kv_int(budget, "budget"), _kv_int(max_len, "max_len")
        _kv_int(sink, "sink", -(1 << 31), 0x7FFFFFFF), _kv_int(recent, "recent", -(1 << 31), 0x7FFFFFFF)
    a = defrag_kv_evict_args(ctypes.pointer(c), budget, max_len, sink, recent,
                             _kv_ptr(next_pos, torch.int32, batch, dev, "next_pos"),
                             weight.data_ptr(), pos.data_ptr(), cap, weight_out.data_ptr(),
                             pos_out.data_ptr(), cap_out,
                             _kv_ptr(lens_out, torch.int32, batch, dev, "lens_out"))
    need = lib.defrag_kv_evict_workspace_bytes(a)
    ws, at, size = _kv_scratch(need, ws, arena, stream, "defrag_kv_evict")
    rc = lib.defrag_kv_evict(a, at, size, _kv_stream(stream, dev))
    if rc != DEFRAG_OK:
        raise DefragError(rc, "defrag_kv_evict")


def defrag_strerror(code: int) -> str:
    return strerror(code)
