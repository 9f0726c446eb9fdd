"""Beam selection on the GPU against its plain 64-bit definition."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from beam_oracle import check_beam  # noqa: E402
from grammar_constrained_logit_gb300 import ops  # noqa: E402
from grammar_constrained_logit_gb300 import synthetic as syn  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from grammar_constrained_logit_gb300 import _lib

    _lib.load()


def placed(x, dtype, shift=0, pad=0, poison=float("nan")):
    """x [rows, V] as a device matrix that starts `shift` elements into its buffer, with
    `pad` poisoned columns behind each row."""
    R, V = x.shape
    t = torch.full((R * (V + pad) + shift + 8,), poison, dtype=TYPES[dtype], device="cuda")
    t = t[shift:shift + R * (V + pad)].view(R, V + pad)
    t[:, :V] = torch.from_numpy(x.astype(np.float32)).cuda().to(TYPES[dtype])
    return t


def run(t, scores, n, V, **kw):
    out = ops.beam_select(t, torch.from_numpy(scores).cuda(), n, vocab_size=V, **kw)
    return [o.cpu().numpy() for o in out]


def seen(t, V):
    return t[:, :V].double().cpu().numpy()


def dense(R, V, density, rng):
    allowed = rng.random((R, V)) < density
    bm = syn.pack_bits(allowed)
    syn.garbage_tail(bm, V, rng)
    return allowed, bm


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("batch, beams, V, n, shift, pad", [
    (1, 1, 1, 1, 0, 0), (1, 1, 1, 4, 3, 0), (2, 3, 7, 6, 1, 0), (3, 2, 31, 4, 0, 1),
    (1, 4, 32, 8, 0, 0), (2, 4, 33, 8, 5, 0), (2, 5, 511, 10, 0, 0), (2, 2, 513, 4, 2, 7),
    (1, 4, 1023, 8, 0, 0), (1, 4, 1024, 8, 0, 0), (3, 4, 1025, 8, 7, 0), (2, 3, 4099, 7, 4, 3),
    (5, 1, 2049, 2, 0, 0), (1, 16, 3001, 32, 0, 0), (1, 64, 1500, 128, 1, 0),
    (1, 256, 65, 256, 0, 0), (2, 8, 20011, 16, 0, 0), (1, 3, 70001, 256, 6, 0)])
def test_shapes(dtype, batch, beams, V, n, shift, pad):
    rng = np.random.default_rng(V * 7 + n)
    R = batch * beams
    t = placed(rng.standard_normal((R, V)) * 2.5, dtype, shift, pad)
    scores = -rng.random((batch, beams), dtype=np.float32) * 10
    check_beam(run(t, scores, n, V), seen(t, V), scores, n)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V, shift", [(1003, 0), (1003, 3), (4096, 0), (9001, 1)])
@pytest.mark.parametrize("density", [0.0, 0.002, 0.1, 0.9])
def test_masks(dtype, V, shift, density):
    rng = np.random.default_rng(int(density * 1000) + V)
    batch, beams, n = 4, 5, 10
    R = batch * beams
    t = placed(rng.standard_normal((R, V)) * 3, dtype, shift, 5, float("inf"))
    allowed, bm = dense(R, V, density, rng)
    allowed[1], bm[1] = False, 0  # a row that keeps nothing
    syn.garbage_tail(bm, V, rng)
    scores = -rng.random((batch, beams), dtype=np.float32) * 10
    scores[2, 1:] = -np.inf
    scores[3, 0] = np.nan
    needs = (rng.random(R) < 0.8).astype(np.uint8)
    needs[1] = 1
    finished = (rng.random((batch, beams)) < 0.3).astype(np.uint8)
    finished[0] = 0
    for f, m in ((None, None), (needs, None), (None, finished), (needs, finished)):
        eff = allowed if f is None else allowed | (f == 0)[:, None]
        got = run(t, scores, n, V, bitmask=torch.from_numpy(bm).cuda(), pad_id=2,
                  row_needs_mask=None if f is None else torch.from_numpy(f).cuda(),
                  finished=None if m is None else torch.from_numpy(m.astype(bool)).cuda())
        check_beam(got, seen(t, V), scores, n, allowed=eff, finished=m, pad=2)


def test_bitmask_narrower_or_wider_than_logits():
    rng = np.random.default_rng(3)
    t = placed(rng.standard_normal((4, 200)), "bf16")
    allowed, bm = dense(4, 96, 0.5, rng)
    scores = -rng.random((2, 2), dtype=np.float32)
    got = ops.beam_select(t, torch.from_numpy(scores).cuda(), 4,
                          bitmask=torch.from_numpy(bm).cuda())
    check_beam([o.cpu().numpy() for o in got], seen(t, 96), scores, 4, allowed=allowed)
    wide = np.full((6, 20), -1, dtype=np.int32)
    got = ops.beam_select(t.view(2, 2, 200), torch.from_numpy(scores).cuda(), 4,
                          bitmask=torch.from_numpy(wide).cuda())
    check_beam([o.cpu().numpy() for o in got], seen(t, 200), scores, 4)


def test_nothing_to_choose():
    """No live beam, no kept token, no vocabulary: empty places and no more."""
    t = torch.zeros(6, 40, device="cuda")
    dead = np.full((2, 3), -np.inf, dtype=np.float32)
    s, k, p = run(t, dead, 3, 40)
    assert np.isneginf(s).all() and (k == -1).all() and (p == -1).all()
    live = np.zeros((2, 3), dtype=np.float32)
    s, k, p = run(torch.full_like(t, float("-inf")), live, 3, 40)
    assert np.isneginf(s).all() and (k == -1).all() and (p == -1).all()
    fin = torch.tensor([[0, 1, 0], [0, 0, 0]], dtype=torch.uint8, device="cuda")
    s, k, p = run(t, live, 3, 0, finished=fin, pad_id=5)
    assert s[0, 0] == 0 and k[0, 0] == 5 and p[0, 0] == 1
    assert (k[0, 1:] == -1).all() and (k[1] == -1).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_lowest_and_infinite_logits(dtype):
    rng = np.random.default_rng(9)
    V = 2500
    x = rng.standard_normal((8, V))
    low = float(torch.finfo(TYPES[dtype]).min)
    x[0] = low                              # the type's lowest value is a logit
    x[1, 5:] = low
    x[2, [7, 1800]] = np.inf                # two tokens share the mass
    x[3, ::2] = np.nan                      # NaN are no candidates
    x[4] = np.nan
    x[5] = -np.inf
    x[6, 3] = np.nan
    x[6, 1024:] = -np.inf
    x[7] = float(torch.finfo(TYPES[dtype]).max)
    t = placed(x, dtype, 1)
    scores = -rng.random((4, 2), dtype=np.float32)
    for n in (2, 5):
        check_beam(run(t, scores, n, V), seen(t, V), scores, n)
    # the same values in masked places leave no trace
    allowed = np.isfinite(x) & (np.abs(x) < 100)
    allowed[0, 3] = True
    got = run(t, scores, 5, V, bitmask=torch.from_numpy(syn.pack_bits(allowed)).cuda())
    check_beam(got, seen(t, V), scores, 5, allowed=allowed)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "capped", "steps", "two"])
def test_many_equal_or_ordered(dtype, kind):
    """Rows on which a threshold admits far more than n candidates, or comes in the worst
    order."""
    V, batch, beams, n = 9003, 2, 4, 8
    j = np.arange(V, dtype=np.float64)
    rng = np.random.default_rng(2)
    x = {"equal": np.zeros(V), "rising": j / 1000, "falling": -j / 1000,
         "capped": np.minimum(rng.standard_normal(V) * 3, 2.0),
         "steps": np.floor(j / 700), "two": (j % 2)}[kind]
    t = placed(np.tile(x, (batch * beams, 1)), dtype)
    # beams of one batch entry equal (ties go by beam, then token), of the other not
    scores = np.array([[-1.0] * 4, [-4.0, -3.0, -2.0, -1.0]], dtype=np.float32)
    s, k, p = run(t, scores, n, V)
    check_beam((s, k, p), seen(t, V), scores, n)
    top = np.flatnonzero(seen(t, V)[0] == seen(t, V)[0].max())
    want = [(b, v) for b in range(beams) for v in top][:n]
    if len(want) == n:
        assert list(zip(p[0], k[0])) == want and len(set(s[0])) == 1


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1001, 5003])
def test_equal_rows_score_equally_at_any_alignment(dtype, V):
    rng = np.random.default_rng(4)
    x = np.tile(rng.standard_normal(V) * 2, (8, 1))  # odd V: each row is aligned differently
    t = placed(x, dtype, 3)
    s, k, p = run(t, np.full((1, 8), -2.5, dtype=np.float32), 16, V)
    order = np.argsort(-seen(t, V)[0], kind="stable")
    assert list(zip(p[0], k[0])) == [(b, order[i]) for i in range(2) for b in range(8)] or \
        seen(t, V)[0][order[0]] == seen(t, V)[0][order[1]]
    assert len(set(s[0, :8])) == 1 and len(set(s[0, 8:])) == 1


def test_infinite_scores():
    rng = np.random.default_rng(5)
    t = placed(rng.standard_normal((4, 3000)), "f32")
    scores = np.array([[0.0, np.inf, -1.0, -np.inf]], dtype=np.float32)
    s, k, p = run(t, scores, 6, 3000)
    assert np.isposinf(s).all() and (p == 1).all() and k[0].tolist() == list(range(6))
    scores = np.array([[3e38, -3e38, 1e-30, 0.0]], dtype=np.float32)
    check_beam(run(t, scores, 6, 3000), seen(t, 3000), scores, 6)


def test_large_offsets():
    """Logits far from zero: the difference is taken before anything is scaled."""
    rng = np.random.default_rng(6)
    x = rng.standard_normal((4, 3000)) * 2
    x[1] += 3e4
    x[2] -= 5e4
    t = placed(x, "f32")
    scores = -rng.random((1, 4), dtype=np.float32)
    check_beam(run(t, scores, 8, 3000), seen(t, 3000), scores, 8)


def test_any_workspace_content_stream_and_graph():
    rng = np.random.default_rng(7)
    V, n = 5000, 8
    t = placed(rng.standard_normal((8, V)) * 2, "bf16")
    scores = -rng.random((2, 4), dtype=np.float32) * 5
    want = run(t, scores, n, V)
    sc = torch.from_numpy(scores).cuda()
    need = ops.beam_select_workspace_bytes(t.dtype, 8, V)
    for fill in (0, 0x7f, 0xff):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got = ops.beam_select(t, sc, n, workspace=ws)
        for g, w in zip(got, want):
            assert np.array_equal(g.cpu().numpy(), w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ops.beam_select(t, sc, n)
    side.synchronize()
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = tuple(torch.empty(2, n, dtype=d, device="cuda")
                for d in (torch.float32, torch.int64, torch.int32))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.beam_select(t, sc, n, workspace=ws, out=out)
    t2 = torch.randn(8, V, device="cuda").to(torch.bfloat16)
    t.copy_(t2)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    fresh = ops.beam_select(t, sc, n)
    for a, b in zip(out, fresh):
        assert torch.equal(a, b)


def test_logits_are_not_written_and_bad_arguments():
    t = torch.randn(8, 100, device="cuda")
    keep = t.clone()
    sc = torch.zeros(2, 4, device="cuda")
    ops.beam_select(t, sc)
    assert torch.equal(t, keep)
    with pytest.raises(ValueError):
        ops.beam_select(t[:6], sc)
    with pytest.raises(ValueError):
        ops.beam_select(t, sc.cpu())
    with pytest.raises(ValueError):
        ops.beam_select(t.t(), torch.zeros(25, 4, device="cuda"))
    with pytest.raises(TypeError):
        ops.beam_select(t.double(), sc)
    with pytest.raises(ValueError):
        ops.beam_select(t, sc, row_needs_mask=torch.ones(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        ops.beam_select(t, sc, finished=torch.zeros(8, device="cuda"))
    with pytest.raises(ValueError):
        ops.beam_select(t, sc, 3, out=(sc, sc, sc))
    with pytest.raises(Exception, match="too large"):
        ops.beam_select(t, sc, 257)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("n", [3, 40, 200])
@pytest.mark.parametrize("batch, beams, V, kept", [(2, 64, 40001, 0), (1, 256, 16000, 5),
                                                   (2, 5, 1100003, 17)])
def test_more_chunks_at_the_bound_than_a_list_holds(dtype, n, batch, beams, V, kept):
    """Every chunk's maximum is the row's: the first tokens of the first beam come out.
    `kept`: the rows' first tokens are lower, so the winners begin behind them."""
    t = torch.ones(batch * beams, V, dtype=TYPES[dtype], device="cuda")
    t[:, :kept] = 0.5
    t[:, 3 * V // 4:] = 1.0
    scores = np.full((batch, beams), -1.5, dtype=np.float32)
    scores[:, 0] = -2.0
    scores[-1, 1] = -np.inf
    s, k, p = run(t, scores, n, V)
    for b in range(batch):
        first = 1 if b < batch - 1 else 2
        assert (p[b] == first).all() and k[b].tolist() == list(range(kept, kept + n))
        assert len(set(s[b])) == 1


@pytest.mark.parametrize("n", [4, 40])
def test_more_chunks_than_shared_memory_holds(n):
    """64 beams of 600001 tokens: the chunks' maxima are read from memory."""
    beams, V = 64, 600001
    g = torch.Generator("cuda").manual_seed(3)
    t = torch.rand(beams, V, device="cuda", generator=g).to(torch.bfloat16)
    at = torch.randperm(beams * V, device="cuda", generator=g)[:60]
    t.view(-1)[at] = (2.0 + torch.arange(60, device="cuda") / 8).to(torch.bfloat16)
    scores = torch.zeros(1, beams, device="cuda")
    s, k, p = ops.beam_select(t, scores, n)
    lp = t.double().log_softmax(-1).view(-1)
    best = lp.topk(n)
    assert torch.equal(p[0].long() * V + k[0], best.indices)
    assert bool(((s[0].double() - best.values).abs() <= 4e-6 + 2.0 ** -24 * best.values.abs()).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("beams, V, n", [(3, 2001, 6), (1, 1025, 1), (7, 300, 14)])
def test_more_requests_than_multiprocessors(dtype, beams, V, n):
    rng = np.random.default_rng(V)
    batch = 170
    t = placed(rng.standard_normal((batch * beams, V)) * 2.5, dtype, 1, 2)
    scores = -rng.random((batch, beams), dtype=np.float32) * 10
    check_beam(run(t, scores, n, V), seen(t, V), scores, n)


def test_a_single_token_scores_as_its_beam():
    """One kept token has probability 1: its score is the beam's, to the last bit, and ties
    with finished beams fall by beam."""
    V = 2100
    t = torch.randn(6, V, device="cuda").half()
    allowed = np.zeros((6, V), dtype=bool)
    allowed[np.arange(6), [5, 0, 2099, 1024, 77, 3]] = True
    scores = np.array([[-0.3, -0.3, -0.3, -1e-6, -0.3, -7.7]], dtype=np.float32)
    fin = torch.tensor([[0, 1, 0, 0, 1, 0]], dtype=torch.uint8, device="cuda")
    s, k, p = run(t, scores, 8, V, bitmask=torch.from_numpy(syn.pack_bits(allowed)).cuda(),
                  finished=fin, pad_id=9)
    assert p[0].tolist() == [3, 0, 1, 2, 4, 5, -1, -1]
    assert k[0].tolist() == [1024, 5, 9, 2099, 9, 3, -1, -1]
    assert np.array_equal(s[0, :6], scores[0, [3, 0, 1, 2, 4, 5]])
