"""ctypes view of liblp.so (the C ABI declared in include/lp.h).

Loading is explicit and loud: if the library has not been built, ``load()``
raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
import threading

from .build import LIB

c_i64, c_i32, c_u64, c_f32, c_vp = (ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64,
                                    ctypes.c_float, ctypes.c_void_p)

LP_F32, LP_F16, LP_BF16 = 0, 1, 2
LP_OK, LP_ERR_INVALID_ARGUMENT, LP_ERR_UNSUPPORTED_DTYPE, LP_ERR_CUDA, LP_ERR_TOO_LARGE = range(5)

EXPORTS = ("lp_apply_token_bitmask", "lp_apply_token_bitmask_rows", "lp_apply_packed_bitmask",
           "lp_upload_bitmask",
           "lp_sample",
           "lp_mask_and_sample", "lp_mask_and_sample_slots", "lp_sample_workspace_bytes",
           "lp_mask_and_sample_noalloc",
           "lp_beam_select", "lp_beam_select_workspace_bytes", "lp_reorder_states",
           "lp_cache_write", "lp_cache_read",
           "lp_cache_attend", "lp_cache_attend_workspace_bytes",
           "lp_cache_evict", "lp_cache_evict_workspace_bytes",
           "lp_verify_drafts", "lp_verify_drafts_workspace_bytes",
           "lp_philox4x32_10", "lp_status_string")


class SamplingParams(ctypes.Structure):
    """lp_sampling_params: each array is a device pointer to B values or NULL."""

    _fields_ = [("temperature", c_vp), ("temperature_scalar", c_f32),
                ("top_k", c_vp), ("top_k_scalar", c_i32),
                ("top_p", c_vp), ("top_p_scalar", c_f32),
                ("min_p", c_vp), ("min_p_scalar", c_f32),
                ("seed", c_u64), ("offset", c_u64)]


class State(ctypes.Structure):
    """lp_state: the bytes of a tensor's rows, strides in bytes."""

    _fields_ = [("data", c_vp), ("row_stride", c_i64), ("run_bytes", c_i64),
                ("token_bytes", c_i64), ("outer", c_i64 * 3), ("outer_stride", c_i64 * 3)]


class CachePart(ctypes.Structure):
    """lp_cache_part: codes and their scaling, strides in bytes."""

    _fields_ = [("codes", c_vp), ("params", c_vp), ("code_page_stride", c_i64),
                ("code_slot_stride", c_i64), ("code_head_stride", c_i64),
                ("param_page_stride", c_i64), ("param_slot_stride", c_i64),
                ("param_head_stride", c_i64)]


class Heads(ctypes.Structure):
    """lp_heads: [n, heads, dim], strides in elements."""

    _fields_ = [("data", c_vp), ("token_stride", c_i64), ("head_stride", c_i64)]


class Rows(ctypes.Structure):
    """lp_rows: [batch, rows, heads, dim], strides in elements."""

    _fields_ = [("data", c_vp), ("batch_stride", c_i64), ("row_stride", c_i64),
                ("head_stride", c_i64)]


class LPError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn}: {message} (status {status})")
        self.status = status


_lib = None
_lock = threading.Lock()


def declare(lib) -> None:
    """Set the argument and result types of the masking and sampling entry points."""
    lib.lp_apply_token_bitmask.restype = c_i32
    lib.lp_apply_token_bitmask.argtypes = [c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i64, c_i64,
                                           c_i64, c_i64, c_vp, c_i64, c_vp]
    lib.lp_apply_token_bitmask_rows.restype = c_i32
    lib.lp_apply_token_bitmask_rows.argtypes = [c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i64,
                                                c_i64, c_i64, c_i64, c_vp, c_vp, c_vp]
    lib.lp_upload_bitmask.restype = c_i32
    lib.lp_upload_bitmask.argtypes = [c_vp, c_i64, c_vp, c_i64, c_i64, c_i64, c_vp, c_vp, c_vp,
                                      c_vp]
    lib.lp_apply_packed_bitmask.restype = c_i32
    lib.lp_apply_packed_bitmask.argtypes = [c_vp, c_i64, c_vp, c_i32, c_i64, c_i64, c_i64, c_vp,
                                            c_i64, c_i64, c_i64, c_f32, c_i64, c_vp, c_i64, c_vp]
    lib.lp_sample.restype = c_i32
    lib.lp_sample.argtypes = [c_vp, c_i32, c_i64, c_i64, c_i64, ctypes.POINTER(SamplingParams),
                              c_vp, c_vp, c_i64, c_vp]
    lib.lp_mask_and_sample.restype = c_i32
    lib.lp_mask_and_sample.argtypes = [c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i64, c_i64,
                                       c_i64, c_i64, c_vp, c_i64, ctypes.POINTER(SamplingParams),
                                       c_vp, c_vp, c_i64, c_vp]
    lib.lp_mask_and_sample_slots.restype = c_i32
    lib.lp_mask_and_sample_slots.argtypes = [c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i64,
                                             c_i64, c_i64, c_i64, c_vp, c_i64,
                                             ctypes.POINTER(SamplingParams), c_i64, c_vp, c_vp,
                                             c_vp, c_i64, c_vp]
    lib.lp_mask_and_sample_noalloc.restype = c_i32
    lib.lp_mask_and_sample_noalloc.argtypes = [c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i64,
                                               c_i64, c_i64, c_i64, c_vp, c_i64,
                                               ctypes.POINTER(SamplingParams), c_vp, c_vp]
    lib.lp_sample_workspace_bytes.restype = c_i64
    lib.lp_sample_workspace_bytes.argtypes = [c_i32, c_i64, c_i64]
    lib.lp_philox4x32_10.restype = c_i32
    lib.lp_philox4x32_10.argtypes = [c_vp, c_vp, c_vp, c_i64, c_vp]
    lib.lp_status_string.restype = ctypes.c_char_p
    lib.lp_status_string.argtypes = [c_i32]


def declare_beam(lib) -> None:
    """The same for the beam-search entry points (csrc/beam.cu, reorder.cu, cache.cu)."""
    lib.lp_beam_select_workspace_bytes.restype = c_i64
    lib.lp_beam_select_workspace_bytes.argtypes = [c_i32, c_i64, c_i64]
    lib.lp_beam_select.restype = c_i32
    lib.lp_beam_select.argtypes = [c_vp, c_i32, c_i64, c_i64, c_i64, c_i64, c_vp, c_i64, c_i64,
                                   c_i64, c_i64, c_vp, c_vp, c_vp, c_i64, c_i64, c_vp, c_vp,
                                   c_vp, c_vp, c_i64, c_vp]
    lib.lp_reorder_states.restype = c_i32
    lib.lp_reorder_states.argtypes = [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp, c_vp, c_vp]
    for f in (lib.lp_cache_write, lib.lp_cache_read):
        f.restype = c_i32
        f.argtypes = [c_vp, c_vp, c_i64, c_i32, c_i32, c_i64, c_i64, c_i64, c_i64, c_i64, c_vp,
                      c_i64, c_vp]


def declare_attend(lib) -> None:
    """The same for csrc/attend.cu, evict.cu and verify.cu."""
    lib.lp_cache_attend_workspace_bytes.restype = c_i64
    lib.lp_cache_attend_workspace_bytes.argtypes = [c_i64] * 5
    lib.lp_cache_attend.restype = c_i32
    lib.lp_cache_attend.argtypes = [c_vp, c_i32, c_i64, c_i64, c_i64, c_i64, c_i64, c_vp, c_vp,
                                    c_i32, c_i64, c_i64, c_i64, c_vp, c_i64, c_i64, c_i64, c_vp,
                                    c_vp, c_f32, c_i64, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp]
    lib.lp_cache_evict_workspace_bytes.restype = c_i64
    lib.lp_cache_evict_workspace_bytes.argtypes = [c_i64] * 3
    lib.lp_cache_evict.restype = c_i32
    lib.lp_cache_evict.argtypes = [c_vp, c_i64, c_i32, c_i64, c_i64, c_i64, c_i64, c_i64, c_vp,
                                   c_i64, c_i64, c_i64, c_vp, c_i64, c_i64, c_i64, c_vp, c_i64,
                                   c_i64, c_i64, c_vp, c_vp, c_i64, c_vp]
    lib.lp_verify_drafts_workspace_bytes.restype = c_i64
    lib.lp_verify_drafts_workspace_bytes.argtypes = [c_i32, c_i64, c_i64]
    lib.lp_verify_drafts.restype = c_i32
    lib.lp_verify_drafts.argtypes = [c_vp, c_i32, c_i64, c_i64, c_i64, c_vp, c_i64, c_i64, c_i64,
                                     c_i64, c_vp, c_i64, c_vp, c_vp, c_i64, c_i64, c_vp, c_vp,
                                     c_f32, c_u64, c_u64, c_vp, c_vp, c_vp, c_vp, c_i64, c_vp]


def load(path: str | None = None):
    """Open liblp.so once per process; raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or LIB
            if not os.path.exists(p):
                raise RuntimeError(
                    f"{p} is not built: run `python -m grammar_constrained_logit_gb300.build` "
                    "(or __graft_entry__.build()) first; there is no fallback path")
            lib = ctypes.CDLL(p)
            declare(lib)
            declare_beam(lib)
            declare_attend(lib)
            _lib = lib
    return _lib


def check(fn: str, status: int) -> None:
    if status != LP_OK:
        msg = load().lp_status_string(status).decode()
        raise LPError(fn, status, msg)
