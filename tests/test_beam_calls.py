"""Calls of the operators whose checks and launches are followed on the host: nothing here
reaches a GPU."""
import ctypes
import os
import subprocess
import sys
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from grammar_constrained_logit_gb300 import _lib, ops  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class OnGpu:
    """A CPU tensor that says it lies on a CUDA device."""

    def __init__(self, t, index=0):
        self.t, self.is_cuda, self.device = t, True, torch.device("cuda", index)

    def __getattr__(self, name):
        return getattr(self.t, name)

    def __getitem__(self, i):
        return OnGpu(self.t[i], self.device.index)


class Recorder:
    """Stands for the library: notes its calls and the device that is current in them."""

    def __init__(self, current):
        self.current, self.calls = current, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.current[0]))
            return _lib.LP_OK

        return call


@pytest.fixture
def recorded(monkeypatch):
    """A recorder in the library's place, with device 0 current."""
    current = [0]

    class Device:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            self.was, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.was

    r = Recorder(current)
    monkeypatch.setattr(_lib, "load", lambda: r)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(ops, "_current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(ops, "_raw_stream", lambda index: 0)
    return r


def test_import_without_cuda_in_torch():
    """A torch built for the CPU alone has no stream handles; importing needs none."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
            "    del torch._C._cuda_getCurrentRawStream\n"
            "from grammar_constrained_logit_gb300 import ops\n"
            "assert ops.get_bitmask_shape(2, 33) == (2, 2)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("index", [0, 1])
def test_launches_are_on_the_tensors_device(recorded, monkeypatch, index):
    """The default stream's handle is the same on every device: what a call launches on is
    the current one, so that has to be the tensors'."""
    def gpu(*shape, dtype=torch.float32):
        return OnGpu(torch.zeros(*shape, dtype=dtype), index)

    monkeypatch.setattr(ops, "sample_workspace_bytes", lambda *a: 8)
    monkeypatch.setattr(ops, "beam_select_workspace_bytes", lambda *a: 8)
    x, bm = gpu(8, 64), gpu(8, 2, dtype=torch.int32)
    ids, ws = gpu(8, dtype=torch.int64), gpu(8, dtype=torch.uint8)
    slots = gpu(3, dtype=torch.int64)
    kv = [gpu(3, 2, 8) for _ in range(2)]
    scores = gpu(2, 4)
    scores.contiguous = lambda: scores
    best = (gpu(2, 5), gpu(2, 5, dtype=torch.int64), gpu(2, 5, dtype=torch.int32))
    cache = ops.QuantCache(gpu(2, 6, 2, 8, dtype=torch.uint8), gpu(2, 6, 2, 1), dim=8)
    ops.apply_token_bitmask_inplace(x, bm)
    ops.apply_token_bitmask_rows(x, bm)
    ops.apply_packed_bitmask(x, bm, out=gpu(8, 64))
    ops.sample(x, out=ids, workspace=ws)
    ops.mask_and_sample(x, bm, out=ids, workspace=ws)
    bm.reshape = lambda *a: bm
    ops.mask_and_sample_slots(x, bm, 2, out=ids, workspace=ws)
    ops.beam_select(x, scores, 5, out=best, workspace=ws)
    ops.StateReorder([(gpu(8, 10), 0)], 2, 4).reorder(gpu(2, 4, dtype=torch.int32))
    ops.cache_write(cache, kv, slots)
    ops.cache_read(cache, slots, out=kv)
    ops.upload_bitmask(bm, torch.zeros(8, 2, dtype=torch.int32),
                       copy_stream=SimpleNamespace(cuda_stream=0),
                       event=SimpleNamespace(record=lambda s: None))
    assert len(recorded.calls) == 11
    assert {device for _, device in recorded.calls} == {index}
    assert recorded.current == [0]


def test_what_is_written_must_not_be_expanded(recorded):
    codes, params = torch.zeros(2, 6, 2, 8, dtype=torch.uint8), torch.zeros(2, 6, 2, 1)
    for c, p in ((codes[:, :1].expand(2, 6, 2, 8), params),
                 (codes, params[:, :, :1].expand(2, 6, 2, 1)),
                 (codes[:1].expand(2, 6, 2, 8), params)):
        with pytest.raises(ValueError, match="expanded"):
            ops.QuantCache(OnGpu(c), OnGpu(p), dim=8)
    one = torch.zeros(1, 1, 1, 8, dtype=torch.uint8).as_strided((1, 1, 1, 8), (0, 0, 0, 1))
    ops.QuantCache(OnGpu(one), OnGpu(torch.zeros(1, 1, 1, 1)), dim=8)  # nothing overlaps

    cache = ops.QuantCache(OnGpu(codes), OnGpu(params), dim=8)
    slots = OnGpu(torch.arange(3))
    full = OnGpu(torch.zeros(3, 2, 8))
    for wide in (torch.zeros(1, 2, 8).expand(3, 2, 8), torch.zeros(3, 1, 8).expand(3, 2, 8)):
        with pytest.raises(ValueError, match="expanded"):
            ops.cache_read(cache, slots, out=(full, OnGpu(wide)))
        assert not recorded.calls
    ops.cache_write(cache, (full, OnGpu(torch.zeros(1, 2, 8).expand(3, 2, 8))), slots)  # reads
    ops.cache_read(cache, slots, out=(full, OnGpu(torch.zeros(3, 2, 8))))
    assert [name for name, _ in recorded.calls] == ["lp_cache_write", "lp_cache_read"]


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("bits, dt, group", [(8, 0, (1 << 29) + 1), (4, 2, 1 << 30),
                                             (8, 1, (1 << 31) - 1)])
def test_groups_whose_bytes_pass_31_bits_are_refused(write, bits, dt, group):
    """A thread's place within a group is a 32-bit number of bytes."""
    from grammar_constrained_logit_gb300 import build

    build.build()
    p, h = _lib.CachePart(), _lib.Heads()
    p.codes = p.params = h.data = 0x10000  # never dereferenced: the calls are refused
    lib = _lib.load()
    st = (lib.lp_cache_write if write else lib.lp_cache_read)(
        ctypes.byref(p), ctypes.byref(h), 1, bits, dt, 4, 4, 1, group, group, 0x10000, 1, None)
    assert st == _lib.LP_ERR_TOO_LARGE
