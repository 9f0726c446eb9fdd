"""The operators together: the example's loop of attention, verification and eviction on the
package's operators against the same loop on their plain definitions; their calls in graphs,
on other streams, by two threads, and where a launch fails."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from attend_oracle import attended, evicted, held, slots_of, verified  # noqa: E402
from grammar_constrained_logit_gb300 import _lib, ops  # noqa: E402
from test_gpu_beam_calls import _FailingStream, _two_threads  # noqa: E402
from test_gpu_verify import gumbel  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(ROOT, "examples", "speculative_decoding.py")
    spec = importlib.util.spec_from_file_location("speculative_decoding", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Plain:
    """The same cache, written by the package; what is new by its definition."""

    QuantCache, cache_write = ops.QuantCache, staticmethod(ops.cache_write)

    @staticmethod
    def cache_attend(cache, q, blocks, lengths, *, block_size, weights):
        out, _, w, _ = attended(held(cache), q.double().cpu().numpy(), blocks.cpu().numpy(),
                                lengths.tolist(), block_size)
        weights += torch.from_numpy(w).to(weights)
        return torch.from_numpy(out).to(q)

    @staticmethod
    def verify_drafts(logits, drafts, uniforms, *, draft_probs, bitmask, row_needs_mask,
                      temperature, seed, offset, vocab_size):
        x = logits.double().cpu().numpy()
        slots, rows, V = x.shape
        words = np.ascontiguousarray(bitmask.cpu().numpy()).view(np.uint8)
        allowed = np.unpackbits(words, axis=1, bitorder="little")[:, :V] != 0
        allowed |= (row_needs_mask.cpu().numpy() == 0)[:, None]
        got = [verified(x[s], allowed.reshape(slots, rows, V)[s], drafts[s].tolist(),
                        draft_probs[s].cpu().numpy(), uniforms[s].tolist(), temperature,
                        lambda n, s=s: gumbel(seed, s * rows + n, offset, V))
               for s in range(slots)]
        return (torch.from_numpy(np.stack([t for t, _, _ in got])).cuda(),
                torch.tensor([n for _, n, _ in got], dtype=torch.int32, device="cuda"))

    @staticmethod
    def cache_evict(cache, weights, blocks, lengths, keep, *, first, recent, block_size):
        new = []
        for b, n in enumerate(lengths.tolist()):
            new.append(min(n, keep))
            at = torch.from_numpy(slots_of(blocks.cpu().numpy(), b, n, block_size, cache.slots))
            for h in range(cache.heads if n > keep else 0):
                kept = torch.from_numpy(evicted(n, weights[b, h].cpu().numpy(), keep, first,
                                                recent))
                for t in (cache.codes, cache.params):
                    t[:, at[:keep].cuda(), h] = t[:, at[kept].cuda(), h].clone()
                w = weights[b, h, kept.cuda()].clone()
                weights[b, h, :n] = 0.0
                weights[b, h, :keep] = w
        return torch.tensor(new, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("batch, drafts, budget", [(1, 1, 12), (3, 3, 16), (2, 5, 40)])
def test_loop_as_on_the_plain_definitions(example, bits, batch, drafts, budget):
    model = example.Decoder(seed=batch, dim=64)
    g = torch.Generator().manual_seed(drafts)
    prompts = torch.randint(4, model.vocab, (batch, 9), generator=g).cuda()
    got = example.generate(model, prompts, 12, drafts, bits, budget)
    assert got == example.generate(model, prompts, 12, drafts, bits, budget, ops=Plain)


def test_loop_keeps_to_the_grammar(example):
    model = example.Decoder(seed=9)
    prompts = torch.randint(4, model.vocab, (4, 7)).cuda()
    said, accepted = example.generate(model, prompts, 20, 4, 4, 14, seed=3)
    grammar = example.Grammar(model.vocab)
    assert any(accepted)
    for row in said:
        state = grammar.START
        for t in row:
            assert int(grammar.rows[state][t // 32]) >> (t % 32) & 1
            state = grammar.advance(state, t)


def _attend_case(seed, n=700, rows=2, heads=4, shared=4, chunk=False):
    """A call's arguments: (cache, q, blocks, lengths), and weights."""
    g = torch.Generator("cuda").manual_seed(seed)
    if chunk:
        rows, heads, shared = 70, 40, 2
    cache = ops.QuantCache.allocate(n, heads, 128, bits=8)
    x = [torch.randn(n, heads, 128, device="cuda", generator=g) for _ in range(2)]
    ops.cache_write(cache, x, torch.arange(n, device="cuda"))
    q = torch.randn(1, rows, heads * shared, 128, device="cuda", generator=g).to(torch.bfloat16)
    return (cache, q, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
            torch.tensor([n], dtype=torch.int32, device="cuda"))


def _verify_case(seed, V=9000):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(4, 3, V, device="cuda", generator=g) * 3
    q = torch.softmax(torch.randn(4, 2, V, device="cuda", generator=g) * 3, -1)
    return x, q.argmax(-1), torch.rand(4, 2, device="cuda", generator=g), q


CALLS = {
    "attend": lambda seed, k=1: (lambda a: lambda: (ops.cache_attend(*a, block_size=a[0].slots),))(
        _attend_case(seed, 700 * k)),
    "chunk": lambda seed, k=1: (lambda a: lambda: (ops.cache_attend(*a, block_size=a[0].slots),))(
        _attend_case(seed, 300 * k, chunk=True)),
    "verify": lambda seed, k=1: (lambda a: lambda: ops.verify_drafts(
        *a[:3], draft_probs=a[3], seed=7))(_verify_case(seed, 9000 * k)),
}


def _evict_call(seed, n=900, keep=300):
    cache, _, blocks, lengths = _attend_case(seed, n)
    w = torch.rand(1, 4, n, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
    codes, params, was = cache.codes.clone(), cache.params.clone(), w.clone()

    def call():
        cache.codes.copy_(codes)
        cache.params.copy_(params)
        w.copy_(was)
        left = ops.cache_evict(cache, w, blocks, lengths, keep, recent=20, block_size=n)
        return left, w.clone(), cache.codes.clone(), cache.params.clone()

    return call


CALLS["evict"] = lambda seed, k=1: _evict_call(seed, 900 * k)


@pytest.mark.parametrize("name", list(CALLS))
def test_captured_and_replayed(name):
    """Two graphs without a workspace replay side by side, with other calls between, and give
    what the eager call gives; a larger eager call after the capture changes nothing."""
    calls = [CALLS[name](s) for s in (1, 2)]
    want = [tuple(t.clone() for t in c()) for c in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for c in calls:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(c())
        graphs.append(g)
    with torch.cuda.stream(side):
        CALLS[name](3, 5)()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


@pytest.mark.parametrize("name", list(CALLS))
def test_two_threads_on_one_stream(name):
    calls = [CALLS[name](s, 1 + s) for s in (1, 2)]
    want = [tuple(t.clone() for t in c()) for c in calls]
    torch.cuda.synchronize()

    def work(i):
        for _ in range(50):
            got = calls[i]()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))

    _two_threads(work)


@pytest.mark.parametrize("name", list(CALLS))
def test_on_another_stream_one_after_another(name):
    """Calls of different sizes follow one another on a side stream, sharing its scratch."""
    calls = [CALLS[name](1, 3), CALLS[name](2, 1), CALLS[name](3, 2)]
    want = [tuple(t.clone() for t in c()) for c in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [c() for _ in range(20) for c in calls]
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(o, want[i % 3]))


@pytest.mark.parametrize("failing", ["attend", "chunk", "verify", "evict"])
def test_a_failed_launch_is_reported_once(failing):
    a, c, v = _attend_case(1), _attend_case(2, 300, chunk=True), _verify_case(3)
    outs = [torch.empty_like(x[1]) for x in (a, c)]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    vout = (torch.empty(4, 3, dtype=torch.int64, device="cuda"),
            torch.empty(4, dtype=torch.int32, device="cuda"))
    w = torch.rand(1, 4, 700, device="cuda")
    left = torch.empty(1, dtype=torch.int32, device="cuda")
    calls = {
        "attend": lambda: ops.cache_attend(*a, block_size=700, out=outs[0], workspace=ws),
        "chunk": lambda: ops.cache_attend(*c, block_size=300, out=outs[1], workspace=ws),
        "verify": lambda: ops.verify_drafts(*v[:3], draft_probs=v[3], out=vout, workspace=ws),
        "evict": lambda: ops.cache_evict(a[0], w, a[2], a[3], 700, block_size=700, out=left,
                                         workspace=ws)}
    for call in calls.values():
        call()
    torch.cuda.synchronize()
    want = [t.clone() for t in (*outs, *vout, left)]
    with _FailingStream() as s, torch.cuda.stream(s):
        with pytest.raises(_lib.LPError) as e:
            calls[failing]()
    assert e.value.status == _lib.LP_ERR_CUDA
    for call in calls.values():  # none of them hears of it again
        call()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, (*outs, *vout, left)))


def test_workspaces_of_any_content():
    for name, make in CALLS.items():
        want = make(1)()
        kept = {"attend": ops._attend_scratch, "chunk": ops._attend_scratch,
                "verify": ops._verify_scratch, "evict": ops._evict_scratch}[name]
        for byte in (0, 0xff, 0x7f):
            for ws in kept.tensors.values():
                ws.fill_(byte)
            assert all(torch.equal(x, y) for x, y in zip(make(1)(), want)), (name, byte)
