"""Eviction from the cache by accumulated attention weight: byte for byte as defined."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from attend_oracle import evicted, slots_of  # noqa: E402
from grammar_constrained_logit_gb300 import ops  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from grammar_constrained_logit_gb300 import _lib

    _lib.load()


def random_cache(rng, total, heads, dim, bits, group, parts=2, page=None, heads_first=False):
    """Bytes that nothing wrote: an eviction moves them as they are."""
    shape = (parts, heads, total) if heads_first else (parts, total, heads)
    codes = torch.from_numpy(rng.integers(0, 256, (*shape, dim * bits // 8), dtype=np.uint8))
    words = rng.integers(-2 ** 31, 2 ** 31, (*shape, dim // group)).astype(np.int32)
    params = torch.from_numpy(words).view(torch.float32) if bits == 8 else \
        torch.from_numpy(words).view(torch.bfloat16).view(*shape, dim // group, 2)
    codes, params = codes.cuda(), params.cuda()
    if heads_first:
        codes, params = codes.transpose(1, 2), params.transpose(1, 2)
    if page:
        codes, params = (t.unflatten(1, (total // page, page)) for t in (codes, params))
    return ops.QuantCache(codes, params, dim=dim, bits=bits)


def raw(cache):
    codes, params = cache.codes, cache.params
    if codes.dim() == 5:
        codes, params = codes.flatten(1, 2), params.flatten(1, 2)
    return (codes.contiguous().cpu().numpy().copy(),
            params.contiguous().cpu().view(torch.uint8).numpy().copy())


def check(cache, weights, blocks, lengths, size, keep, first=0, recent=0):
    codes, params = raw(cache)
    want_w = weights.copy()
    most = blocks.shape[1] * size
    new = []
    for b in range(len(lengths)):
        n = min(max(int(lengths[b]), 0), most)
        new.append(min(n, keep))
        if n <= keep:
            continue
        at = slots_of(blocks, b, n, size, codes.shape[1])
        for h in range(cache.heads):
            kept = evicted(n, weights[b, h], keep, first, recent)
            assert kept.size == keep
            move = [(int(at[s]), int(at[j])) for j, s in enumerate(kept)
                    if s != j and at[s] >= 0 and at[j] >= 0]
            if move:
                src, dst = (np.array(x) for x in zip(*move))
                codes[:, dst, h] = codes[:, src, h]
                params[:, dst, h] = params[:, src, h]
            want_w[b, h, :keep] = weights[b, h, kept]
            want_w[b, h, keep:n] = 0.0
    w = torch.from_numpy(weights.copy()).cuda()
    got = ops.cache_evict(cache, w, torch.from_numpy(blocks).cuda(),
                          torch.tensor(lengths, dtype=torch.int32, device="cuda"), keep,
                          first=first, recent=recent, block_size=size)
    assert got.dtype == torch.int32 and got.tolist() == new
    assert np.array_equal(w.cpu().numpy().view(np.uint32), want_w.view(np.uint32))
    c, p = raw(cache)
    assert np.array_equal(c, codes) and np.array_equal(p, params)


def table(rng, lengths, size, total):
    need = [-(-max(n, 0) // size) for n in lengths]
    order = rng.permutation(total // size)
    blocks = np.full((len(lengths), max(need) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        blocks[b, :n] = order[at:at + n]
        at += n
    return blocks


def some_weights(rng, batch, heads, width, kind):
    w = np.exp(rng.standard_normal((batch, heads, width)) * 2).astype(np.float32)
    if kind == "ties":
        w = np.round(w)
    elif kind == "equal":
        w[:] = 0.5
    elif kind == "zero":
        w *= rng.random(w.shape) < 0.1
        w = np.where(rng.random(w.shape) < 0.5, w, -w).astype(np.float32)  # -0 among them
    elif kind == "odd":
        odd = np.array([np.nan, np.inf, -np.inf, -1.0, 0.0, -0.0, 1e-45, 3e38], np.float32)
        w = odd[rng.integers(0, 8, w.shape)]
    return w


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "zero", "odd"])
@pytest.mark.parametrize("bits, heads, dim, group, page", [
    (8, 8, 128, 128, 16), (4, 8, 128, 32, 16), (4, 5, 80, 16, None), (8, 3, 72, 24, None),
    (8, 1, 7, 7, None), (4, 2, 6, 2, 16), (8, 2, 576, 64, None)])
def test_shapes(kind, bits, heads, dim, group, page):
    rng = np.random.default_rng(dim + bits)
    size = 16 if page else 9
    lengths = [200, 64, 65, 0, 63, 1, 130]
    total = (sum(-(-n // size) for n in lengths) + 2) * size
    cache = random_cache(rng, total, heads, dim, bits, group, page=page)
    blocks = table(rng, lengths, size, total)
    w = some_weights(rng, len(lengths), heads, blocks.shape[1] * size, kind)
    check(cache, w, blocks, lengths, size, 64, first=4, recent=10)


@pytest.mark.parametrize("keep, first, recent", [
    (0, 0, 0), (1, 0, 0), (1, 1, 0), (1, 0, 1), (50, 50, 0), (50, 0, 50), (50, 20, 30),
    (99, 0, 0), (100, 10, 10), (101, 0, 0), (10 ** 9, 5, 5)])
def test_what_stays(keep, first, recent):
    rng = np.random.default_rng(keep % 1000 + first)
    lengths = [100, 300, 99, 2]
    cache = random_cache(rng, 40 * 16, 3, 64, 8, 64)
    blocks = table(rng, lengths, 16, 40 * 16)
    w = some_weights(rng, 4, 3, blocks.shape[1] * 16, "spread")
    check(cache, w, blocks, lengths, 16, keep, first, recent)


@pytest.mark.parametrize("bits, dim, group", [(8, 128, 128), (4, 80, 16), (8, 33, 11)])
@pytest.mark.parametrize("n, keep", [(5000, 1200), (5000, 4999), (20001, 3), (9000, 8191)])
def test_long(bits, dim, group, n, keep):
    rng = np.random.default_rng(n + keep)
    lengths = [n, 70]
    total = (-(-n // 16) + 8) * 16
    cache = random_cache(rng, total, 2, dim, bits, group, page=16)
    blocks = table(rng, lengths, 16, total)
    w = some_weights(rng, 2, 2, blocks.shape[1] * 16, "spread")
    check(cache, w, blocks, lengths, 16, keep, first=min(2, keep), recent=min(1, keep - 2))


def test_layouts():
    """Heads first, one part, eight parts, a whole sequence a block."""
    rng = np.random.default_rng(3)
    for parts, heads_first in ((2, True), (1, False), (8, False)):
        cache = random_cache(rng, 300, 2, 32, 8, 32, parts=parts, heads_first=heads_first)
        blocks = np.array([[1], [0], [2]], np.int32)
        w = some_weights(rng, 3, 2, 100, "spread")
        check(cache, w, blocks, [100, 90, 10], 100, 40, 2, 3)


@pytest.mark.parametrize("shift", [0, 4, 1])
def test_pages_among_others(shift):
    """A page holds several layers' slots; codes start at any byte."""
    rng = np.random.default_rng(6)
    heads, pages, page, dim = 3, 14, 16, 64
    n = 2 * pages * 3 * page * heads * dim
    every = torch.from_numpy(rng.integers(0, 256, n + 16, dtype=np.uint8)).cuda()
    was = every.clone()
    codes = every[shift:shift + n].view(2, pages, 3, page, heads, dim)[:, :, 1]
    params = torch.rand(2, pages, 3, page, heads, 1, device="cuda")[:, :, 1]
    cache = ops.QuantCache(codes, params, dim=dim, bits=8)
    blocks = table(rng, [100, 90], page, pages * page)
    w = some_weights(rng, 2, heads, blocks.shape[1] * page, "spread")
    check(cache, w, blocks, [100, 90], page, 40, 2, 5)
    for layer in (0, 2):  # the others' bytes stay
        a, b = (t[shift:shift + n].view(2, pages, 3, page, heads, dim)[:, :, layer]
                for t in (every, was))
        assert torch.equal(a, b)


def test_slots_outside_and_long_lengths():
    rng = np.random.default_rng(4)
    cache = random_cache(rng, 320, 2, 64, 4, 32)
    blocks = table(rng, [160, 100], 16, 320)
    blocks[0, 3], blocks[0, 6], blocks[1, 0] = -1, 2 ** 31 - 1, 20
    w = some_weights(rng, 2, 2, blocks.shape[1] * 16, "spread")
    check(cache, w, blocks, [10 ** 9, -5], 16, 60, 4, 8)
    check(cache, w, blocks, [170, 100], 16, 30, 0, 0)


def test_weights_with_gaps():
    """Weights that are a slice of something larger: what is around them stays."""
    rng = np.random.default_rng(5)
    cache = random_cache(rng, 160, 2, 64, 8, 64)
    room = torch.full((2, 4, 200), 9.0, device="cuda")
    w = room[:, 1:3, 7:7 + 96]
    w.copy_(torch.from_numpy(some_weights(rng, 2, 2, 96, "spread")))
    was = w.cpu().numpy().copy()
    blocks = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5)
    lens = torch.tensor([80, 50], dtype=torch.int32, device="cuda")
    out = torch.empty(2, dtype=torch.int32, device="cuda")
    assert ops.cache_evict(cache, w, blocks, lens, 30, block_size=16, out=out) is out
    for b, n in enumerate((80, 50)):
        for h in range(2):
            kept = evicted(n, was[b, h], 30, 0, 0)
            assert np.array_equal(w[b, h, :30].cpu().numpy(), was[b, h, kept])
            assert (w[b, h, 30:n] == 0).all()
            assert np.array_equal(w[b, h, n:].cpu().numpy(), was[b, h, n:])
    w.fill_(9.0)
    assert (room == 9.0).all()


@pytest.mark.parametrize("kind, keep", [("spread", 1000), ("ties", 300000), ("equal", 7)])
def test_longer_than_shared_memory(kind, keep):
    """More weights than a cluster's shared memory holds: one block reads them a digit a time."""
    rng = np.random.default_rng(keep)
    n, size = 330001, 512
    total = -(-n // size) * size + 3 * size
    cache = random_cache(rng, total, 1, 16, 8, 16)
    blocks = table(rng, [n, 900], size, total)
    w = some_weights(rng, 2, 1, blocks.shape[1] * size, kind)
    check(cache, w, blocks, [n, 900], size, keep, first=3, recent=4)


@pytest.mark.parametrize("bits, heads, dim, group", [
    (8, 2, 4096, 4096), (8, 3, 301, 301), (8, 2, 256, 1), (4, 1, 8192, 32)])
def test_wide_heads(bits, heads, dim, group):
    """More pieces to a token than a block has threads for."""
    rng = np.random.default_rng(dim)
    lengths = [90, 300, 12, 0]
    total = 40 * 16
    cache = random_cache(rng, total, heads, dim, bits, group, page=16)
    blocks = table(rng, lengths, 16, total)
    w = some_weights(rng, len(lengths), heads, blocks.shape[1] * 16, "ties")
    check(cache, w, blocks, lengths, 16, 50, first=2, recent=6)
