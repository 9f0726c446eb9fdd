"""Calls of the operators around their kernels: what a launch needs, what a failed one leaves
behind, whose scratch it uses."""
import ctypes
import math
import os
import subprocess
import sys
import threading

import pytest

torch = pytest.importorskip("torch")

from grammar_constrained_logit_gb300 import _lib, ops  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.load()


EVERY_COUNT = """
import sys
import torch
from grammar_constrained_logit_gb300 import ops
for beams in map(int, sys.argv[1:]):
    t = torch.arange(2 * beams * 40, device="cuda", dtype=torch.int32).view(2 * beams, 40)
    p = torch.stack([(torch.arange(beams) * 7 + 1) % beams, torch.arange(beams) // 2])
    want = t.view(2, beams, 40).cpu().gather(1, p[..., None].expand(2, beams, 40))
    ops.reorder_states([t], p.int().cuda())
    assert torch.equal(t.view(2, beams, 40).cpu(), want), beams
"""


@pytest.mark.parametrize("counts", [[12], range(1, 257)])
def test_every_number_of_beams(counts):
    """In a process of its own, fewest beams first: how much shared memory a launch may
    take is set for the whole process by the first call that asks for more."""
    r = subprocess.run([sys.executable, "-c", EVERY_COUNT, *map(str, counts)], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


class _FailingStream:
    """A stream on which every launch fails on the host: its capture was made invalid."""

    def __enter__(self):
        with open("/proc/self/maps") as f:
            path = next(p for p in (line.split()[-1] for line in f) if "libcudart.so" in p)
        self.rt, self.h = ctypes.CDLL(path), ctypes.c_void_p()
        assert self.rt.cudaStreamCreateWithFlags(ctypes.byref(self.h), 1) == 0  # non-blocking
        assert self.rt.cudaStreamBeginCapture(self.h, 2) == 0  # relaxed
        assert self.rt.cudaStreamSynchronize(self.h) != 0  # not while capturing
        self.rt.cudaGetLastError()
        return torch.cuda.ExternalStream(self.h.value)

    def __exit__(self, *_):
        graph = ctypes.c_void_p()
        assert self.rt.cudaStreamEndCapture(self.h, ctypes.byref(graph)) != 0
        assert self.rt.cudaStreamDestroy(self.h) == 0
        self.rt.cudaGetLastError()


@pytest.mark.parametrize("failing", ["select", "reorder", "write", "read"])
def test_a_failed_launch_is_reported_once(failing):
    t = torch.randn(8, 900, device="cuda")
    scores = torch.zeros(2, 4, device="cuda")
    n = 5
    out = tuple(torch.empty(2, n, dtype=d, device="cuda")
                for d in (torch.float32, torch.int64, torch.int32))
    ws = torch.empty(ops.beam_select_workspace_bytes(t.dtype, 8, 900), dtype=torch.uint8,
                     device="cuda")
    rows = torch.arange(8, device="cuda").float().view(8, 1).repeat(1, 64)
    mover = ops.StateReorder([rows], 2, 4)
    parents = torch.tensor([[1, 2, 3, 0], [0, 0, 2, 2]], dtype=torch.int32, device="cuda")
    cache = ops.QuantCache.allocate(6, 2, 64)
    x = [torch.randn(6, 2, 64, device="cuda") for _ in range(2)]
    back = [torch.zeros_like(v) for v in x]
    slots = torch.arange(6, device="cuda")
    calls = {"select": lambda: ops.beam_select(t, scores, n, out=out, workspace=ws),
             "reorder": lambda: mover.reorder(parents),
             "write": lambda: ops.cache_write(cache, x, slots),
             "read": lambda: ops.cache_read(cache, slots, out=back)}
    for call in calls.values():  # whatever a first call sets up is set up
        call()
    torch.cuda.synchronize()
    before = rows.clone()
    with _FailingStream() as s, torch.cuda.stream(s):
        with pytest.raises(_lib.LPError) as e:
            calls[failing]()
    assert e.value.status == _lib.LP_ERR_CUDA
    torch.cuda.synchronize()
    assert torch.equal(rows, before)
    for name in ("reorder", "write", "read", "select"):  # none of them hears of it again
        calls[name]()
    torch.cuda.synchronize()
    at = [(parents[b, k] + 4 * b).item() for b in range(2) for k in range(4)]
    assert torch.equal(rows, before[at])
    assert all(float((a - b).abs().max()) < 0.5 for a, b in zip(back, x))


class _Watched:
    """The library, which notes the scratch that a call of one entry point is given."""

    def __init__(self, lib, name, instead=None):
        self._lib, self._name, self._instead, self.seen = lib, name, instead, []

    def __getattr__(self, name):
        fn = getattr(self._lib, name)
        if name != self._name:
            return fn

        def call(*args):
            self.seen.append(getattr(args[-3], "value", args[-3]))
            return self._instead() if self._instead else fn(*args)

        return call


def _search_step(seed, batch=2, beams=4, V=5000):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(batch * beams, V, device="cuda", generator=g) * 2
    return x, -torch.rand(batch, beams, device="cuda", generator=g) * 5


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def _two_threads(work):
    failed = []

    def run(i):
        try:
            work(i)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failed:
        raise failed[0]


def test_two_threads_on_one_stream_have_their_own_scratch(monkeypatch):
    """A selection is two launches that hand on partial sums: with both threads between
    the call and its return, neither's scratch may be the other's."""
    steps = [_search_step(i) for i in range(2)]
    torch.cuda.synchronize()
    inside = threading.Barrier(2)
    lib = _Watched(_lib.load(), "lp_beam_select", lambda: inside.wait(30) and 0)
    monkeypatch.setattr(_lib, "load", lambda: lib)
    _two_threads(lambda i: ops.beam_select(*steps[i]))
    assert len(lib.seen) == 2 and lib.seen[0] != lib.seen[1]


def test_two_threads_on_one_stream_select_as_one():
    steps = [_search_step(i, 2 + i, 4, 20000 + 999 * i) for i in range(2)]
    want = [ops.beam_select(*s) for s in steps]
    torch.cuda.synchronize()

    def work(i):
        got = [ops.beam_select(*steps[i]) for _ in range(300)]
        torch.cuda.synchronize()
        assert all(_same(g, want[i]) for g in got)

    _two_threads(work)


def test_captured_without_a_workspace(monkeypatch):
    """A graph's scratch is its own: neither that of the calls before it on its stream, nor
    freed by a larger one after it, nor another graph's."""
    small, large = _search_step(1), _search_step(2, 16, 8, 60000)
    want = ops.beam_select(*small)
    torch.cuda.synchronize()
    lib = _Watched(_lib.load(), "lp_beam_select")
    monkeypatch.setattr(_lib, "load", lambda: lib)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.beam_select(*small)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(ops.beam_select(*small))
        graphs.append(g)
    with torch.cuda.stream(side):
        ops.beam_select(*large)
    torch.cuda.synchronize()
    before, one, two, after = lib.seen
    assert len({before, one, two}) == 3 and after not in (one, two)
    # what the large call made the allocator give up is someone else's now
    torch.cuda.empty_cache()
    others = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(_same(o, want) for o in outs)
    assert all(bool((o == 7).all()) for o in others)


@pytest.mark.parametrize("failing", ["sample", "upload", "rows", "apply"])
def test_a_failed_masking_or_sampling_call_is_reported_once(failing):
    x, bm = torch.randn(4, 900, device="cuda"), torch.full((4, 29), -1, dtype=torch.int32,
                                                           device="cuda")
    ws = torch.zeros(ops.sample_workspace_bytes(x.dtype, 4, 900), dtype=torch.uint8, device="cuda")
    ids = torch.empty(4, dtype=torch.int64, device="cuda")
    host = torch.zeros(4, 29, dtype=torch.int32).pin_memory()
    mask = torch.zeros_like(bm)
    has = torch.empty(4, dtype=torch.int32, device="cuda")
    lib = _lib.load()

    def rows():  # the entry point itself: the binding would allocate
        st = lib.lp_apply_token_bitmask_rows(
            x.data_ptr(), _lib.LP_F32, 4, 900, 900, bm.data_ptr(), 4, 29, 29, -1, None,
            has.data_ptr(), torch.cuda.current_stream().cuda_stream)
        _lib.check("lp_apply_token_bitmask_rows", st)

    def upload():
        st = lib.lp_upload_bitmask(mask.data_ptr(), 29, host.data_ptr(), 29, 4, 29, None, None,
                                   torch.cuda.current_stream().cuda_stream, None)
        _lib.check("lp_upload_bitmask", st)

    calls = {"sample": lambda: ops.sample(x, temperature=0.0, out=ids, workspace=ws),
             "upload": upload, "rows": rows,
             "apply": lambda: ops.apply_token_bitmask_inplace(x, bm)}
    for call in calls.values():
        call()
    torch.cuda.synchronize()
    with _FailingStream() as s, torch.cuda.stream(s):
        with pytest.raises(_lib.LPError) as e:
            calls[failing]()
    assert e.value.status == _lib.LP_ERR_CUDA
    for name in ("apply", "rows", "sample", "upload"):
        calls[name]()
    torch.cuda.synchronize()
    assert torch.equal(ids, x.argmax(1)) and torch.equal(mask.cpu(), host)


def test_sampler_two_threads_on_one_stream_have_their_own_scratch(monkeypatch):
    x = torch.randn(4, 3000, device="cuda")
    torch.cuda.synchronize()
    inside = threading.Barrier(2)
    lib = _Watched(_lib.load(), "lp_sample", lambda: inside.wait(30) and 0)
    monkeypatch.setattr(_lib, "load", lambda: lib)

    def work(i):
        for _ in range(2):
            ops.sample(x)

    _two_threads(work)
    one, two, three, four = lib.seen  # the calls went in pairs, one of each thread
    assert one != two and {one, two} == {three, four}  # kept between calls


def test_sampler_two_threads_on_one_stream_draw_as_one():
    xs = [torch.randn(64, 20000 + 1000 * i, device="cuda") for i in range(2)]
    want = [[ops.sample(x, 0.8, 40, 0.9, seed=j) for j in range(100)] for x in xs]
    torch.cuda.synchronize()

    def work(i):
        got = [ops.sample(xs[i], 0.8, 40, 0.9, seed=j) for j in range(100)]
        torch.cuda.synchronize()
        assert _same(got, want[i])

    _two_threads(work)


@pytest.mark.parametrize("entry", ["lp_sample", "lp_mask_and_sample", "lp_mask_and_sample_slots"])
def test_sampler_captured_without_a_workspace(monkeypatch, entry):
    def call(x):
        if entry == "lp_sample":
            return ops.sample(x, 0.8, 40, 0.9, seed=5)
        if entry == "lp_mask_and_sample":
            return ops.mask_and_sample(x, None, 0.8, 40, 0.9, seed=5)
        return ops.mask_and_sample_slots(x, None, 2, 0.8, 40, 0.9, seed=5)

    small, large = (torch.randn(r, v, device="cuda") for r, v in ((8, 5000), (512, 90000)))
    want = call(small)
    torch.cuda.synchronize()
    lib = _Watched(_lib.load(), entry)
    monkeypatch.setattr(_lib, "load", lambda: lib)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(small)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(call(small))
        graphs.append(g)
    with torch.cuda.stream(side):
        call(large)
    torch.cuda.synchronize()
    before, one, two, after = lib.seen
    assert len({before, one, two}) == 3 and after not in (one, two)
    torch.cuda.empty_cache()
    others = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert all(bool((o == 7).all()) for o in others)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kept", [0, 9])
def test_more_chunks_at_the_bound_than_a_clusters_lists_hold(dtype, kept):
    """More than 16 to find in few requests: eight blocks go through the chunks side by
    side, each with a list of 2048.  Every chunk's maximum is the row's, and there are more
    than 8 x 2048: the first tokens of the first beam of the best score come out.  Scores are
    near -14: a rounding to 32 bits, and 4e-6 for the logarithm of the row's sum."""
    beams, V, n = 64, 300001 if dtype == torch.bfloat16 else 150001, 40
    assert beams * -(-V // (2048 // dtype.itemsize)) > 8 * 2048
    t = torch.ones(2 * beams, V, dtype=dtype, device="cuda")
    t[:, :kept] = 0.5
    scores = torch.full((2, beams), -1.5, device="cuda")
    scores[:, 0] = -2.0
    scores[1, 1] = float("-inf")
    s, k, p = ops.beam_select(t, scores, n)
    for b in range(2):
        assert p[b].tolist() == [1 + b] * n and k[b].tolist() == list(range(kept, kept + n))
        z = math.log((V - kept) + kept * math.exp(-0.5))
        assert s[b].unique().numel() == 1 and abs(float(s[b, 0]) + 1.5 + z) <= 4e-6 + 2.0 ** -24 * 16


def test_tokens_of_more_than_4_gb():
    """A token of 2^32 bytes and more: the range up to the last token, or to one far beyond
    it, ends at the row's end."""
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    t = torch.empty(2, 1, (1 << 32) + 16, dtype=torch.uint8, device="cuda")
    p = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    for i, stop in enumerate((None, 1, 2, (1 << 31) - 1)):
        t[0].fill_(10 + i)
        t[1].fill_(20 + i)
        end = None if stop is None else torch.tensor([stop], dtype=torch.int32, device="cuda")
        ops.reorder_states([(t, 0, 1)], p, stop=end)
        for row, value in ((0, 20 + i), (1, 10 + i)):
            assert int(t[row].amin()) == value == int(t[row].amax()), (stop, row)
