"""PyTorch-facing binding of liblp.so.

Argument marshalling only: every op passes device pointers, sizes, strides and
the current CUDA stream to the C entry point of the same name (include/lp.h),
which does all of the work in its own kernels.  PyTorch supplies device memory
and streams.  The names follow the pages: ``apply_token_bitmask_inplace``
(XGrammar "Bitmask Operations"), ``apply_packed_bitmask`` (Modular MAX), and
``sample`` (Kernel Hub "logits-processor"); ``lp_*`` aliases carry the C names.
"""
from __future__ import annotations

import ctypes
import functools
import threading
from typing import Sequence

import torch

from . import _lib
from ._lib import SamplingParams, check

_DT = {torch.float32: _lib.LP_F32, torch.float16: _lib.LP_F16, torch.bfloat16: _lib.LP_BF16}


def _dtype_code(t: torch.Tensor) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"logits must be float32, float16 or bfloat16, not {t.dtype}") from None


def _matrix(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        if t.dim() != 1:
            raise ValueError(f"{name} must be 1-D or 2-D, got {tuple(t.shape)}")
        t = t.unsqueeze(0)
    if t.stride(1) != 1 and t.size(1) > 1:
        raise ValueError(f"{name} rows must be contiguous (stride(1) == 1)")
    return t


def _matrix_host(t: torch.Tensor) -> torch.Tensor:
    if t.dim() != 2 or (t.size(1) > 1 and t.stride(1) != 1):
        raise ValueError("host bitmask must be 2-D with contiguous rows")
    return t


# The current stream's handle and the current device, without the objects and checks around
# them: a call of these operators is a few microseconds, and a Stream would be two of them.
# (A torch built for the CPU alone has neither; importing this module needs none.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _call(name: str, device, args: tuple) -> None:
    """The entry point ``name`` with ``device`` current: its kernels run there, and the default
    stream's handle, which is the same on every device, means that device's."""
    if _current_device() != device.index:
        with torch.cuda.device(device):
            return _call(name, device, args)
    st = getattr(_lib.load(), name)(*args)
    if st != _lib.LP_OK:
        check(name, st)


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(_raw_stream(t.device.index))


def _bitmask(bitmask: torch.Tensor, device) -> torch.Tensor:
    bm = _matrix(bitmask, "bitmask")
    if bm.dtype != torch.int32:
        raise TypeError("bitmask must be int32")
    if bm.device != device:
        raise ValueError("bitmask must be on the same device as logits")
    return bm


class _Indices:
    """Row list marshalled for the C ABI.  An empty list still needs a non-NULL
    pointer (NULL means "every row"), so it points at a one-element buffer."""

    def __init__(self, t: torch.Tensor):
        self.n = t.numel()
        self.t = t if self.n else torch.empty(1, dtype=torch.int32, device=t.device)

    def data_ptr(self):
        return self.t.data_ptr()

    def numel(self):
        return self.n


def _indices(indices, device):
    if indices is None:
        return None
    if isinstance(indices, torch.Tensor):
        idx = indices.to(device=device, dtype=torch.int32).contiguous().view(-1)
    else:
        idx = torch.tensor(list(indices), dtype=torch.int32, device=device)
    return _Indices(idx)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stride(t: torch.Tensor) -> int:
    return t.stride(0) if t.size(0) > 1 or t.size(1) <= 1 else max(t.stride(0), t.size(1))


def apply_token_bitmask_inplace(logits: torch.Tensor, bitmask: torch.Tensor, *,
                                vocab_size: int | None = None,
                                indices: Sequence[int] | torch.Tensor | None = None) -> None:
    """Set masked logits to -inf in place (bit 0 = masked, bit 1 = kept)."""
    lg = _matrix(logits, "logits")
    bm = _bitmask(bitmask, lg.device)
    idx = _indices(indices, lg.device)
    _call("lp_apply_token_bitmask", lg.device, (
        _ptr(lg), _dtype_code(lg), lg.size(0), lg.size(1), _stride(lg), _ptr(bm), bm.size(0),
        bm.size(1), _stride(bm), -1 if vocab_size is None else int(vocab_size), _ptr(idx),
        0 if idx is None else idx.numel(), _stream(lg)))


lp_apply_token_bitmask = apply_token_bitmask_inplace


def apply_token_bitmask_rows(logits: torch.Tensor, bitmask: torch.Tensor,
                             row_needs_mask: torch.Tensor | None = None, *,
                             vocab_size: int | None = None,
                             report: bool = False) -> torch.Tensor | None:
    """Set masked logits to -inf in place in the rows whose ``row_needs_mask``
    flag (uint8 or bool, one per row) is nonzero; every row when it is None.
    With ``report``, returns int32 [B]: 1 where the row keeps a token after the
    call, 0 where its mask admits none (an unsatisfiable row)."""
    lg = _matrix(logits, "logits")
    bm = _bitmask(bitmask, lg.device)
    B = lg.size(0)
    flags = None
    if row_needs_mask is not None:
        if row_needs_mask.device != lg.device:
            raise ValueError("row_needs_mask must be on the same device as logits")
        flags = row_needs_mask.to(torch.uint8).contiguous().view(-1)
        if flags.numel() != B:
            raise ValueError(f"row_needs_mask must have {B} entries")
    has = torch.empty(B, dtype=torch.int32, device=lg.device) if report else None
    _call("lp_apply_token_bitmask_rows", lg.device, (
        _ptr(lg), _dtype_code(lg), B, lg.size(1), _stride(lg), _ptr(bm), bm.size(0), bm.size(1),
        _stride(bm), -1 if vocab_size is None else int(vocab_size), _ptr(flags), _ptr(has),
        _stream(lg)))
    return has


lp_apply_token_bitmask_rows = apply_token_bitmask_rows


def upload_bitmask(device_bitmask: torch.Tensor, host_bitmask: torch.Tensor, *,
                   device_flags: torch.Tensor | None = None,
                   host_flags: torch.Tensor | None = None,
                   copy_stream: torch.cuda.Stream | None = None,
                   event: torch.cuda.Event | None = None) -> torch.cuda.Event:
    """Copy a host-filled bitmask (int32 [rows, words], best page-locked) and,
    optionally, its uint8 row flags into device buffers on ``copy_stream`` (the
    current stream when None), then record ``event`` (a new one when None) after
    the copies and return it.  A compute stream waits on the event before an
    apply reads the mask; the host must not touch the host buffers until the
    event has completed."""
    if host_bitmask.is_cuda or not device_bitmask.is_cuda:
        raise ValueError("host_bitmask must be on the CPU and device_bitmask on the GPU")
    hb, db = _matrix_host(host_bitmask), _matrix(device_bitmask, "device_bitmask")
    if hb.dtype != torch.int32 or db.dtype != torch.int32:
        raise TypeError("bitmasks must be int32")
    rows, words = hb.size(0), hb.size(1)
    if db.size(0) < rows or db.size(1) < words:
        raise ValueError("device_bitmask is smaller than host_bitmask")
    if (device_flags is None) != (host_flags is None):
        raise ValueError("pass both row-flag buffers or neither")
    if host_flags is not None and (host_flags.numel() < rows or device_flags.numel() < rows or
                                   host_flags.dtype != torch.uint8 or
                                   device_flags.dtype != torch.uint8):
        raise ValueError("row flags must be uint8 with at least one entry per row")
    stream = copy_stream if copy_stream is not None else torch.cuda.current_stream(db.device)
    ev = event if event is not None else torch.cuda.Event()
    # PyTorch creates an event's CUDA handle at its first record, so the event is
    # recorded here, on the copy stream right after the enqueued copies
    _call("lp_upload_bitmask", db.device, (
        _ptr(db), _stride(db), _ptr(hb), _stride(hb), rows, words, _ptr(device_flags),
        _ptr(host_flags), ctypes.c_void_p(stream.cuda_stream), None))
    ev.record(stream)
    return ev


lp_upload_bitmask = upload_bitmask


class BitmaskStager:
    """Double-buffered page-locked staging of the bitmask and its row flags.

    Each step: ``host()`` gives the host buffers to fill (after the upload that
    last used them has completed); ``upload()`` copies them to a device buffer
    on a copy stream and makes the current stream wait for that copy, returning
    the device buffers for the apply; ``consumed()`` marks, on the current
    stream, that the apply enqueued after ``upload`` is done with them, so that
    the copy two steps later may overwrite them."""

    def __init__(self, rows: int, words: int, device=None):
        dev = torch.device("cuda") if device is None else torch.device(device)
        self.rows, self.words = rows, words
        self.host_mask = [torch.zeros(rows, words, dtype=torch.int32).pin_memory()
                          for _ in range(2)]
        self.host_flags = [torch.zeros(rows, dtype=torch.uint8).pin_memory() for _ in range(2)]
        self.dev_mask = [torch.zeros(rows, words, dtype=torch.int32, device=dev) for _ in range(2)]
        self.dev_flags = [torch.zeros(rows, dtype=torch.uint8, device=dev) for _ in range(2)]
        self.copy_stream = torch.cuda.Stream(device=dev)
        self.uploaded = [None, None]
        self.released = [None, None]
        self.i = 0

    def host(self):
        """The host mask and flags of this step, free to fill."""
        if self.uploaded[self.i] is not None:
            self.uploaded[self.i].synchronize()
        return self.host_mask[self.i], self.host_flags[self.i]

    def upload(self):
        """Start this step's copy; the current stream waits for it.  Returns the
        device (mask, flags) the apply should read."""
        i = self.i
        if self.released[i] is not None:
            self.copy_stream.wait_event(self.released[i])
        ev = upload_bitmask(self.dev_mask[i], self.host_mask[i], device_flags=self.dev_flags[i],
                            host_flags=self.host_flags[i], copy_stream=self.copy_stream)
        self.uploaded[i] = ev
        torch.cuda.current_stream(self.dev_mask[i].device).wait_event(ev)
        return self.dev_mask[i], self.dev_flags[i]

    def consumed(self):
        """After enqueueing the apply: its device buffers may be reused later."""
        ev = torch.cuda.Event()
        ev.record(torch.cuda.current_stream(self.dev_mask[self.i].device))
        self.released[self.i] = ev
        self.i ^= 1


def apply_packed_bitmask(logits: torch.Tensor, bitmask: torch.Tensor,
                         fill_value: float = float("-inf"), *, out: torch.Tensor | None = None,
                         vocab_size: int | None = None,
                         indices: Sequence[int] | torch.Tensor | None = None) -> torch.Tensor:
    """Out-of-place apply: masked positions take ``fill_value``; returns ``out``."""
    lg = _matrix(logits, "logits")
    bm = _bitmask(bitmask, lg.device)
    if out is None:
        out = torch.empty_like(lg)
    o = _matrix(out, "out")
    if o.dtype != lg.dtype or o.shape != lg.shape:
        raise ValueError("out must match logits in dtype and shape")
    idx = _indices(indices, lg.device)
    _call("lp_apply_packed_bitmask", lg.device, (
        _ptr(o), _stride(o), _ptr(lg), _dtype_code(lg), lg.size(0), lg.size(1), _stride(lg),
        _ptr(bm), bm.size(0), bm.size(1), _stride(bm), float(fill_value),
        -1 if vocab_size is None else int(vocab_size), _ptr(idx), 0 if idx is None else idx.numel(),
        _stream(lg)))
    return out


lp_apply_packed_bitmask = apply_packed_bitmask


def _param(v, B, dtype, device, keep):
    """A per-row parameter: (device pointer or None, scalar)."""
    if isinstance(v, torch.Tensor) and v.numel() != 1:
        if v.numel() != B:
            raise ValueError(f"per-row parameter must have {B} values, got {v.numel()}")
        t = v.to(device=device, dtype=dtype).contiguous()
        keep.append(t)
        return ctypes.c_void_p(t.data_ptr()), 0
    s = v.item() if isinstance(v, torch.Tensor) else v
    return None, (int(s) if dtype == torch.int32 else float(s))


def _params(B, device, temperature, top_k, top_p, min_p, seed, offset, keep):
    p = SamplingParams()
    p.temperature, p.temperature_scalar = _param(temperature, B, torch.float32, device, keep)
    p.top_k, p.top_k_scalar = _param(top_k, B, torch.int32, device, keep)
    p.top_p, p.top_p_scalar = _param(top_p, B, torch.float32, device, keep)
    p.min_p, p.min_p_scalar = _param(min_p, B, torch.float32, device, keep)
    p.seed = int(seed) & (2**64 - 1)
    p.offset = int(offset) & (2**64 - 1)
    return p


def _ids_out(out, B, device):
    if out is None:
        return torch.empty(B, dtype=torch.int64, device=device)
    if out.dtype != torch.int64 or out.numel() != B or not out.is_contiguous():
        raise ValueError("out must be a contiguous int64 tensor of B elements")
    return out


class _Kept(threading.local):
    """Scratch kept between calls, a tensor for each (device, stream), apart for each thread:
    a call is several launches that hand on what they found, and two threads' launches on
    one stream can alternate."""

    def __init__(self):
        self.tensors: dict = {}


_sample_scratch, _beam_scratch = _Kept(), _Kept()


def _scratch(kept: _Kept, device, stream: int, need: int, make) -> torch.Tensor:
    """At least ``need`` bytes: the kept tensor, grown on demand.  A capture gets a new one,
    from the graph's memory: a kept one could be replaced while the graph lives, or be
    another graph's.  (Asking costs 0.3 us; a new tensor at every call took 3.)"""
    if torch.cuda.is_current_stream_capturing():
        return make(max(need, 8), dtype=torch.uint8, device=device)
    key = (device.index, stream)
    ws = kept.tensors.get(key)
    if ws is None or ws.numel() < need:
        ws = kept.tensors[key] = make(max(need, 8), dtype=torch.uint8, device=device)
    return ws


def sample_workspace_bytes(dtype: torch.dtype, batch_size: int, vocab_size: int) -> int:
    """Bytes of device scratch ``sample`` / ``mask_and_sample`` need."""
    n = _lib.load().lp_sample_workspace_bytes(_DT[dtype], batch_size, vocab_size)
    if n < 0:
        raise ValueError("invalid dtype or size")
    return int(n)


def _workspace(workspace, lg: torch.Tensor, B: int, vocab: int) -> torch.Tensor:
    """The caller's workspace (a uint8 CUDA tensor, zero-filled before its first
    use), or the thread's own for (device, stream); the library keeps its counters
    valid across calls.  A capture without one gets its own in the graph, zero-filled
    at each replay: pass one that was allocated before the capture to save that.
    Two threads, or graphs that replay side by side, must not share a workspace."""
    need = sample_workspace_bytes(lg.dtype, B, max(vocab, 0))
    if workspace is not None:
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or \
                workspace.device != lg.device:
            raise ValueError("workspace must be a contiguous uint8 tensor on the logits' device")
        return workspace
    device = lg.device
    return _scratch(_sample_scratch, device, _raw_stream(device.index), need, torch.zeros)


def sample(logits: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, seed: int = 0,
           offset: int = 0, *, vocab_size: int | None = None,
           out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Temperature, top-k ∩ top-p ∩ min-p, Gumbel-max draw keyed by
    (seed, row, offset); greedy for temperature <= 0 or top_k == 1.  Every
    parameter is a scalar or a length-B tensor.  Returns int64 ids [B]."""
    lg = _matrix(logits, "logits")
    B = lg.size(0)
    V = lg.size(1) if vocab_size is None else int(vocab_size)
    keep: list = []
    p = _params(B, lg.device, temperature, top_k, top_p, min_p, seed, offset, keep)
    ids = _ids_out(out, B, lg.device)
    ws = _workspace(workspace, lg, B, V)
    _call("lp_sample", lg.device, (
        _ptr(lg), _dtype_code(lg), B, V, _stride(lg), ctypes.byref(p), _ptr(ids), _ptr(ws),
        ws.numel(), _stream(lg)))
    return ids


lp_sample = sample


def mask_and_sample(logits: torch.Tensor, bitmask: torch.Tensor | None, temperature=1.0,
                    top_k=0, top_p=1.0, min_p=0.0, seed: int = 0, offset: int = 0, *,
                    indices: Sequence[int] | torch.Tensor | None = None,
                    vocab_size: int | None = None,
                    out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The bitmask applied on the fly (logits are not written), then ``sample``.
    Rows in ``indices`` (all rows when None) are masked; a masked row whose mask
    admits no token returns -1."""
    lg = _matrix(logits, "logits")
    B = lg.size(0)
    bm = None if bitmask is None else _bitmask(bitmask, lg.device)
    idx = _indices(indices, lg.device)
    keep: list = []
    p = _params(B, lg.device, temperature, top_k, top_p, min_p, seed, offset, keep)
    ids = _ids_out(out, B, lg.device)
    # the workspace is sized by the widest vocabulary the call can use
    ws = _workspace(workspace, lg, B, lg.size(1))
    _call("lp_mask_and_sample", lg.device, (
        _ptr(lg), _dtype_code(lg), B, lg.size(1), _stride(lg), _ptr(bm),
        0 if bm is None else bm.size(0), 0 if bm is None else bm.size(1),
        0 if bm is None else _stride(bm), -1 if vocab_size is None else int(vocab_size), _ptr(idx),
        0 if idx is None else idx.numel(), ctypes.byref(p), _ptr(ids), _ptr(ws), ws.numel(),
        _stream(lg)))
    return ids


lp_mask_and_sample = mask_and_sample


def mask_and_sample_slots(logits: torch.Tensor, bitmask: torch.Tensor | None,
                          rows_per_slot: int, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
                          seed: int = 0, offset: int = 0, *,
                          seeds: torch.Tensor | None = None,
                          indices: Sequence[int] | torch.Tensor | None = None,
                          vocab_size: int | None = None,
                          out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None) -> torch.Tensor:
    """``mask_and_sample`` on [slots, rows_per_slot, V] logits (or their
    [slots * rows_per_slot, V] view): every sampling parameter is a scalar or
    one value per slot, shared by the slot's rows; ``seeds`` (optional, one
    uint64 per row, as int64 bit patterns) replaces ``seed`` row by row.
    Returns int64 ids [slots * rows_per_slot]."""
    if logits.dim() == 3:
        if logits.size(1) != rows_per_slot:
            raise ValueError("logits [slots, rows_per_slot, V] must match rows_per_slot")
        logits = logits.reshape(-1, logits.size(2))
    lg = _matrix(logits, "logits")
    B = lg.size(0)
    R = int(rows_per_slot)
    if R < 1 or B % R:
        raise ValueError("rows_per_slot must be >= 1 and divide the number of rows")
    bm = None if bitmask is None else _bitmask(bitmask.reshape(-1, bitmask.size(-1)), lg.device)
    idx = _indices(indices, lg.device)
    keep: list = []
    p = _params(B // R, lg.device, temperature, top_k, top_p, min_p, seed, offset, keep)
    sd = None
    if seeds is not None:
        sd = seeds.to(device=lg.device, dtype=torch.int64).contiguous().view(-1)
        if sd.numel() != B:
            raise ValueError(f"seeds must have {B} entries")
    ids = _ids_out(out, B, lg.device)
    ws = _workspace(workspace, lg, B, lg.size(1))
    _call("lp_mask_and_sample_slots", lg.device, (
        _ptr(lg), _dtype_code(lg), B, lg.size(1), _stride(lg), _ptr(bm),
        0 if bm is None else bm.size(0), 0 if bm is None else bm.size(1),
        0 if bm is None else _stride(bm), -1 if vocab_size is None else int(vocab_size), _ptr(idx),
        0 if idx is None else idx.numel(), ctypes.byref(p), R, _ptr(sd), _ptr(ids), _ptr(ws),
        ws.numel(), _stream(lg)))
    return ids


lp_mask_and_sample_slots = mask_and_sample_slots


@functools.lru_cache(maxsize=256)
def beam_select_workspace_bytes(dtype: torch.dtype, rows: int, vocab_size: int) -> int:
    """Bytes of device scratch ``beam_select`` needs for ``rows`` = batch * beams."""
    n = _lib.load().lp_beam_select_workspace_bytes(_DT[dtype], rows, vocab_size)
    if n < 0:
        raise ValueError("invalid dtype or size")
    return int(n)


def _row_flags(flags, rows, device, name):
    if flags.device != device:
        raise ValueError(f"{name} must be on the same device as logits")
    if flags.numel() != rows:
        raise ValueError(f"{name} must have {rows} entries")
    if flags.dtype == torch.bool:
        flags = flags.view(torch.uint8)
    elif flags.dtype != torch.uint8:
        raise TypeError(f"{name} must be uint8 or bool")
    return flags.contiguous()


def beam_select(logits: torch.Tensor, scores: torch.Tensor, n_select: int | None = None, *,
                bitmask: torch.Tensor | None = None,
                row_needs_mask: torch.Tensor | None = None,
                finished: torch.Tensor | None = None, pad_id: int = 0,
                vocab_size: int | None = None, out: tuple | None = None,
                workspace: torch.Tensor | None = None):
    """One step of beam search: the ``n_select`` best continuations (the number of
    beams when None) of each batch entry over its beams and the vocabulary.

    ``logits`` [batch, beams, V] (or its [batch * beams, V] view), ``scores`` float32
    [batch, beams]: the beams' log-probabilities so far, -inf for a beam that does not
    exist (all but the first at the first step).  Log-probabilities are normalised over
    the tokens that ``bitmask`` keeps (in the rows that ``row_needs_mask`` flags; all
    when None).  A beam that ``finished`` (uint8 or bool) flags goes on as one candidate
    (``pad_id``, its score).

    Returns (scores float32, tokens int64, parents int32), each [batch, n_select],
    highest score first, ties to the lowest (beam, token); empty places are
    (-inf, -1, -1).  ``out`` takes the three tensors to write instead.  ``workspace``
    (uint8, ``beam_select_workspace_bytes``, any content) is scratch to use instead of
    what is kept for the thread and stream, or in a capture a part of the graph's memory;
    two threads, or graphs that replay side by side, must not share one."""
    shape = scores.shape
    if len(shape) != 2:
        raise ValueError(f"scores must be [batch, beams], got {tuple(shape)}")
    if scores.dtype != torch.float32:
        raise TypeError("scores must be float32")
    batch, beams = shape
    if logits.dim() == 3:
        if logits.shape[:2] != shape:
            raise ValueError("logits [batch, beams, V] must match scores [batch, beams]")
        logits = logits.flatten(0, 1)
    lg = _matrix(logits, "logits")
    dtype = lg.dtype
    rows, cols = lg.shape
    if rows != batch * beams:
        raise ValueError(f"logits must have {batch * beams} rows, got {rows}")
    device = lg.device
    if scores.device != device:
        raise ValueError("scores must be on the same device as logits")
    dt = _DT[dtype] if dtype in _DT else _dtype_code(lg)
    n = beams if n_select is None else int(n_select)
    bm = flags = ended = None
    if bitmask is not None:
        bm = _bitmask(bitmask.flatten(0, -2) if bitmask.dim() > 2 else bitmask, device)
        if row_needs_mask is not None:
            flags = _row_flags(row_needs_mask, rows, device, "row_needs_mask")
    elif row_needs_mask is not None:
        raise ValueError("row_needs_mask needs a bitmask")
    if finished is not None:
        ended = _row_flags(finished, rows, device, "finished")
    sc = scores if scores.is_contiguous() else scores.contiguous()
    if out is None:
        if n < 0:
            raise ValueError("n_select must not be negative")
        out = (torch.empty((batch, n), dtype=torch.float32, device=device),
               torch.empty((batch, n), dtype=torch.int64, device=device),
               torch.empty((batch, n), dtype=torch.int32, device=device))
    else:
        for t, d in zip(out, (torch.float32, torch.int64, torch.int32), strict=True):
            if t.dtype != d or t.shape != (batch, n) or not t.is_contiguous() or \
                    t.device != device:
                raise ValueError("out must be contiguous float32, int64 and int32 tensors "
                                 "[batch, n_select] on the logits' device")
    stream = _raw_stream(device.index)
    ws = workspace
    if ws is None:
        ws = _scratch(_beam_scratch, device, stream,
                      beam_select_workspace_bytes(dtype, rows, cols), torch.empty)
    elif ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.device != device:
        raise ValueError("workspace must be a contiguous uint8 tensor on the logits' device")
    _call("lp_beam_select", device, (
        lg.data_ptr(), dt, batch, beams, cols,
        lg.stride(0) if rows > 1 else max(lg.stride(0), cols),
        None if bm is None else bm.data_ptr(), 0 if bm is None else bm.size(0),
        0 if bm is None else bm.size(1), 0 if bm is None else _stride(bm),
        -1 if vocab_size is None else int(vocab_size), None if flags is None else flags.data_ptr(),
        sc.data_ptr(), None if ended is None else ended.data_ptr(), int(pad_id), n,
        out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), ws.data_ptr(), ws.numel(), stream))
    return out


lp_beam_select = beam_select


def _expanded(t: torch.Tensor) -> bool:
    """Whether elements of ``t`` share their memory by a stride of zero."""
    return any(n > 1 and st == 0 for n, st in zip(t.shape, t.stride()))


def _state(t: torch.Tensor, row_dim: int, token_dim: int | None) -> _lib.State:
    """A tensor's rows as lp_state: the longest contiguous run, up to the tokens' axis
    when one is given, and the axes around it."""
    if not t.is_cuda:
        raise ValueError("states must be CUDA tensors")
    d = t.dim()
    if not -d <= row_dim < d or (token_dim is not None and not -d <= token_dim < d):
        raise ValueError(f"axis out of range for a state of shape {tuple(t.shape)}")
    row_dim %= d
    if token_dim is not None:
        token_dim %= d
        if token_dim == row_dim:
            raise ValueError("the tokens' axis must not be the rows'")
    if _expanded(t):
        raise ValueError("a state must not be expanded: its rows would overlap")
    size = t.element_size()
    axes = sorted(((st * size, n, i) for i, (n, st) in enumerate(zip(t.shape, t.stride()))
                   if i != row_dim and (n != 1 or i == token_dim)),
                  key=lambda a: (a[0], a[1] == 1))
    run, token, outer, around, closed = size, 0, [], None, False
    for st, n, i in axes:
        if i == token_dim:
            closed = True
            if not outer and (st == run or n == 1):
                token, run = run, run * n
            else:
                around = (st, n)  # tokens apart from each other: an axis around the runs
        elif not outer and not closed and st == run:
            run *= n
        elif outer and outer[-1][0] * outer[-1][1] == st:
            outer[-1] = (outer[-1][0], outer[-1][1] * n)
        else:
            outer.append((st, n))
    if around is not None:
        token = -1
        outer.append(around)
    if len(outer) > 3:
        raise ValueError("a state's other axes must fold to three at most")
    s = _lib.State()
    s.data, s.row_stride, s.run_bytes = t.data_ptr(), t.stride(row_dim) * size, run
    s.token_bytes = token
    if t.numel() == 0:
        s.run_bytes = s.token_bytes = 0
    for d in range(3):
        st, n = outer[-1 - d] if d < len(outer) else (0, 1)
        s.outer[d], s.outer_stride[d] = n, st
    return s


class StateReorder:
    """The states that follow the beams of a search: made once for the tensors that a
    model keeps, then ``reorder`` after each selection moves all of them in place.

    ``states``: tensors whose first axis is the ``batch * beams`` rows, or tuples
    (tensor, rows' axis) or (tensor, rows' axis, tokens' axis).  Views are fine (a cache
    laid out heads first, a slice) as long as rows do not overlap; what is contiguous
    moves in long runs.  The tensors are held, their memory is read and written at each
    call."""

    def __init__(self, states, batch: int, beams: int):
        self.batch, self.beams = int(batch), int(beams)
        if self.batch < 0 or self.beams < 1:
            raise ValueError("batch must not be negative and beams at least 1")
        self.states = []
        for s in states:
            t, rows, tokens = ((s, 0, None) if isinstance(s, torch.Tensor) else
                               (*s, None) if len(s) == 2 else s)
            self.states.append((t, rows, tokens))
        self._c = (_lib.State * max(1, len(self.states)))()
        self.device = None
        for i, (t, rows, tokens) in enumerate(self.states):
            self._c[i] = _state(t, rows, tokens)
            if t.size(rows) != self.batch * self.beams:
                raise ValueError(f"state {i} must have {self.batch * self.beams} rows, "
                                 f"got {t.size(rows)}")
            if self.device is None:
                self.device = t.device
            elif t.device != self.device:
                raise ValueError("states must be on one device")

    def _check(self, t, name, shape, n):
        if t.dtype != torch.int32:
            raise TypeError(f"{name} must be int32")
        if t.device != self.device:
            raise ValueError(f"{name} must be on the states' device")
        if t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {shape}")
        return t.data_ptr()

    def reorder(self, parents: torch.Tensor, start: torch.Tensor | None = None,
                stop: torch.Tensor | None = None) -> None:
        """Row b * beams + k of every state becomes what row b * beams + parents[b, k]
        was.  ``parents`` int32 [batch, beams], as ``beam_select`` returns them; one
        outside [0, beams) leaves its row.  ``start`` / ``stop`` int32 [batch]: of the
        states that have a tokens' axis only tokens [start[b], stop[b]) move (a prompt
        that all beams share need not)."""
        if not self.states:
            return
        b, k = self.batch, self.beams
        p = self._check(parents, "parents", "[batch, beams]", b * k)
        lo = None if start is None else self._check(start, "start", "[batch]", b)
        hi = None if stop is None else self._check(stop, "stop", "[batch]", b)
        _call("lp_reorder_states", self.device, (
            self._c, len(self.states), b, k, p, lo, hi, _raw_stream(self.device.index)))


def reorder_states(states, parents: torch.Tensor, start: torch.Tensor | None = None,
                   stop: torch.Tensor | None = None) -> None:
    """``StateReorder(states, *parents.shape).reorder(parents, start, stop)``, for a
    single call."""
    if parents.dim() != 2:
        raise ValueError("parents must be [batch, beams]")
    StateReorder(states, *parents.shape).reorder(parents, start, stop)


lp_reorder_states = reorder_states


class QuantCache:
    """Keys and values (or any number of parts up to 8) held in 8 or 4 bits.

    ``codes`` uint8 [parts, slots, heads, dim * bits / 8] and ``params`` [parts, slots,
    heads, groups] float32 (8 bits) or [parts, slots, heads, groups, 2] bfloat16 (4
    bits); or with the slots on pages, [parts, pages, page_size, heads, ...].  Any
    strides, as long as a head's codes and its params are contiguous: heads-first
    storage is a permuted view.  ``QuantCache.allocate`` makes both.  A group is dim /
    groups elements.  The tensors are held; both are states that ``StateReorder`` can
    move."""

    def __init__(self, codes: torch.Tensor, params: torch.Tensor, *, dim: int, bits: int = 8):
        if bits not in (4, 8):
            raise ValueError("bits must be 8 or 4")
        if codes.dtype != torch.uint8:
            raise TypeError("codes must be uint8")
        if params.dtype != (torch.float32 if bits == 8 else torch.bfloat16):
            raise TypeError("params must be float32 for 8 bits, bfloat16 for 4")
        if not codes.is_cuda or params.device != codes.device:
            raise ValueError("codes and params must be CUDA tensors on one device")
        d = codes.dim()
        if d not in (4, 5) or params.dim() != d + (bits == 4):
            raise ValueError("codes must be [parts, slots, heads, bytes] or [parts, pages, "
                             "page_size, heads, bytes], params alike")
        if codes.shape[:-1] != params.shape[:d - 1] or (bits == 4 and params.size(-1) != 2):
            raise ValueError("codes and params must agree in parts, slots and heads")
        groups = params.size(d - 1)
        dim = int(dim)
        if dim < 1 or groups < 1 or dim % groups or (bits == 4 and dim // groups % 2) or \
                codes.size(-1) * 8 != dim * bits:
            raise ValueError(f"dim {dim} does not fit {codes.size(-1)} bytes of {bits}-bit codes "
                             f"in {groups} groups")
        want = (1,) if bits == 8 else (2, 1)
        if (codes.size(-1) > 1 and codes.stride(-1) != 1) or any(
                n > 1 and a != b
                for n, a, b in zip(params.shape[d - 1:], params.stride()[d - 1:], want)):
            raise ValueError("a head's codes and params must be contiguous")
        if _expanded(codes) or _expanded(params):
            raise ValueError("codes and params must not be expanded: slots would overlap")
        if codes.size(0) > 8:
            raise ValueError("a cache has 8 parts at most")
        self.codes, self.params, self.dim, self.bits = codes, params, dim, bits
        self.parts, self.heads, self.group = codes.size(0), codes.size(d - 2), dim // groups
        self.page_size = codes.size(d - 3)
        self.slots = self.page_size * (codes.size(1) if d == 5 else 1)
        self.device = codes.device
        self._sizes = (self.slots, max(1, self.page_size), self.heads, dim, self.group)
        self._parts = (_lib.CachePart * max(1, self.parts))()
        self._heads_type = _lib.Heads * max(1, self.parts)
        e = params.element_size()
        for i in range(self.parts):
            p = self._parts[i]
            p.codes, p.params = codes[i].data_ptr(), params[i].data_ptr()
            p.code_page_stride = codes.stride(1) if d == 5 else 0
            p.code_slot_stride, p.code_head_stride = codes.stride(d - 3), codes.stride(d - 2)
            p.param_page_stride = params.stride(1) * e if d == 5 else 0
            p.param_slot_stride = params.stride(d - 3) * e
            p.param_head_stride = params.stride(d - 2) * e

    @classmethod
    def allocate(cls, slots: int, heads: int, dim: int, *, bits: int = 8,
                 group: int | None = None, parts: int = 2, device=None) -> "QuantCache":
        """A cache of ``slots`` slots, its memory zero.  ``group``: dim when None in 8
        bits; in 4 bits 32 where that divides dim, else dim."""
        if group is None:
            group = 32 if bits == 4 and dim % 32 == 0 else dim
        if bits not in (4, 8) or dim < 1 or group < 1 or dim % group or dim * bits % 8:
            raise ValueError("bits must be 8 or 4, and group divide dim")
        dev = torch.device("cuda") if device is None else torch.device(device)
        codes = torch.zeros(parts, slots, heads, dim * bits // 8, dtype=torch.uint8, device=dev)
        shape = (parts, slots, heads, dim // group)
        params = (torch.zeros(shape, device=dev) if bits == 8 else
                  torch.zeros(*shape, 2, dtype=torch.bfloat16, device=dev))
        return cls(codes, params, dim=dim, bits=bits)


def _cache_call(name, cache: QuantCache, xs, slots: torch.Tensor):
    if slots.dtype != torch.int64:
        raise TypeError("slots must be int64")
    device, parts = cache.device, cache.parts
    if slots.dim() != 1 or not slots.is_contiguous() or slots.device != device:
        raise ValueError("slots must be contiguous, 1-D and on the cache's device")
    n = slots.numel()
    if len(xs) != parts:
        raise ValueError(f"expected {parts} tensors, one for each part, got {len(xs)}")
    dtype = xs[0].dtype if xs else torch.float32
    dt = _DT.get(dtype)
    if dt is None:
        raise TypeError(f"tensors must be float32, float16 or bfloat16, not {dtype}")
    shape = (n, cache.heads, cache.dim)
    heads = []
    for x in xs:
        if x.dtype != dtype:
            raise TypeError("the parts' tensors must be of one type")
        if x.device != device:
            raise ValueError("tensors must be on the cache's device")
        if x.shape != shape:
            raise ValueError(f"tensors must be {list(shape)}, got {list(x.shape)}")
        token, head, inner = x.stride()
        if inner != 1 and cache.dim > 1:
            raise ValueError("a head's elements must be contiguous")
        heads.append((x.data_ptr(), token, head))
    _call(name, device, (
        cache._parts, cache._heads_type(*heads), parts, cache.bits, dt, *cache._sizes,
        slots.data_ptr(), n, _raw_stream(device.index)))


def cache_write(cache: QuantCache, x, slots: torch.Tensor) -> None:
    """Quantise ``x`` (one [n, heads, dim] tensor for each part of the cache: keys and
    values; or the tensor itself for a cache of one part) into the cache: token i goes
    to slot ``slots[i]`` (int64), or nowhere when that is outside the cache."""
    _cache_call("lp_cache_write", cache, (x,) if isinstance(x, torch.Tensor) else x, slots)


lp_cache_write = cache_write


def cache_read(cache: QuantCache, slots: torch.Tensor, *, dtype: torch.dtype = torch.bfloat16,
               out=None) -> tuple:
    """The values that slots ``slots`` (int64 [n]) hold, one [n, heads, dim] tensor of
    ``dtype`` for each part; zeros for a slot outside the cache.  ``out`` takes the
    tensors to write instead (their type then counts, dim contiguous)."""
    if out is None:
        if slots.dim() != 1:
            raise ValueError("slots must be contiguous, 1-D and on the cache's device")
        shape = (slots.numel(), cache.heads, cache.dim)
        out = tuple([torch.empty(shape, dtype=dtype, device=cache.device)
                     for _ in range(cache.parts)])
    else:
        out = (out,) if isinstance(out, torch.Tensor) else tuple(out)
        if any(_expanded(t) for t in out):
            raise ValueError("out must not be expanded: tokens would overlap")
    _cache_call("lp_cache_read", cache, out, slots)
    return out


lp_cache_read = cache_read


def philox4x32_10(counters: torch.Tensor, keys: torch.Tensor) -> torch.Tensor:
    """Device Philox4x32-10 on n blocks: counters [n, 4], keys [n, 2] (int32 bit
    patterns on the GPU) -> [n, 4] words (int32 bit patterns)."""
    c = counters.to(torch.int32).contiguous()
    k = keys.to(torch.int32).contiguous()
    if c.dim() != 2 or c.size(1) != 4 or k.shape != (c.size(0), 2) or not c.is_cuda:
        raise ValueError("counters must be [n, 4] and keys [n, 2], on the GPU")
    out = torch.empty_like(c)
    _call("lp_philox4x32_10", c.device, (
        _ptr(c), _ptr(k), _ptr(out), c.size(0), _stream(c)))
    return out


lp_philox4x32_10 = philox4x32_10


def get_bitmask_shape(batch_size: int, vocab_size: int) -> tuple[int, int]:
    """(batch_size, ceil(vocab_size / 32)), the packed int32 bitmask shape."""
    return batch_size, (vocab_size + 31) // 32


bitmask_dtype = torch.int32
