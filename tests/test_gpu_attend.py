"""Attention over the quantised cache against its definition in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from attend_oracle import attended, held, reach  # noqa: E402
from grammar_constrained_logit_gb300 import ops  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from grammar_constrained_logit_gb300 import _lib

    _lib.load()


def filled(total, heads, dim, bits, group, *, page=None, heads_first=False, seed=0, spread=1.0):
    """A cache whose every slot was written: keys and values of different means."""
    g = torch.Generator("cuda").manual_seed(seed)
    groups = dim // group
    tail = () if bits == 8 else (2,)
    ptype = torch.float32 if bits == 8 else torch.bfloat16
    if heads_first:
        codes = torch.zeros(2, heads, total, dim * bits // 8, dtype=torch.uint8, device="cuda")
        params = torch.zeros(2, heads, total, groups, *tail, dtype=ptype, device="cuda")
        codes, params = codes.transpose(1, 2), params.transpose(1, 2)
    else:
        codes = torch.zeros(2, total, heads, dim * bits // 8, dtype=torch.uint8, device="cuda")
        params = torch.zeros(2, total, heads, groups, *tail, dtype=ptype, device="cuda")
    if page:
        codes, params = (t.unflatten(1, (total // page, page)) for t in (codes, params))
    cache = ops.QuantCache(codes, params, dim=dim, bits=bits)
    x = [torch.randn(total, heads, dim, device="cuda", generator=g) * s + m
         for s, m in ((spread, 0.2), (spread * 2, -0.5))]
    ops.cache_write(cache, x, torch.arange(total, device="cuda"))
    return cache


def table(rng, lengths, size, total):
    """Blocks anywhere in the cache, and more columns than any sequence needs."""
    need = [-(-max(n, 0) // size) for n in lengths]
    order = rng.permutation(total // size)
    blocks = np.full((len(lengths), max(need) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        blocks[b, :n] = order[at:at + n]
        at += n
    assert at <= total // size
    return blocks


def check(cache, q, blocks, lengths, size, dtype, *, weights=False, **kw):
    qd = torch.from_numpy(q).cuda().to(TYPES[dtype])
    width = blocks.shape[1] * size
    w = torch.full((q.shape[0], cache.heads, width), 0.25, device="cuda") if weights else None
    n_rows = kw.pop("n_rows", None)
    nr = None if n_rows is None else torch.tensor(n_rows, dtype=torch.int32, device="cuda")
    got = ops.cache_attend(cache, qd, torch.from_numpy(blocks).cuda(),
                           torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                           block_size=size, n_rows=nr, weights=w, **kw)
    want, off, ww, woff = attended(held(cache), qd.double().cpu().numpy(), blocks, lengths, size,
                                   n_rows=n_rows, dtype=dtype, reach=reach(cache), **kw)
    d = np.abs(got.double().cpu().numpy() - want)
    assert got.dtype == qd.dtype and got.shape == qd.shape
    assert (d <= off).all(), (d.max(), (d / np.maximum(off, 1e-300)).max())
    if weights:
        # on top of 0.25: one rounding of the sum
        d = np.abs(w.double().cpu().numpy() - (0.25 + ww))
        assert (d <= woff + 2.0 ** -24 * (0.25 + ww) + 2.0 ** -26 * (ww > 0)).all(), d.max()
        assert (w.cpu().numpy()[ww == 0] == 0.25).all()
    return got


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("batch, rows, heads, shared, dim, group, size", [
    (3, 1, 8, 4, 128, 128, 16), (2, 1, 2, 1, 128, 32, 16), (3, 5, 5, 3, 80, 16, 16),
    (2, 4, 1, 8, 64, 64, 16), (3, 2, 3, 7, 96, 32, 7), (2, 3, 4, 2, 192, 192, 32),
    (2, 1, 2, 5, 256, 32, 16), (2, 8, 2, 8, 128, 64, 16), (1, 40, 2, 3, 64, 16, 16),
    (2, 2, 3, 2, 72, 24, 5), (2, 1, 1, 1, 34, 34, 3), (1, 2, 2, 2, 6, 2, 16),
    (2, 1, 16, 1, 64, 32, 1), (1, 1, 1, 1, 1024, 1024, 16), (2, 3, 11, 1, 128, 128, 64)])
def test_shapes(dtype, bits, batch, rows, heads, shared, dim, group, size):
    rng = np.random.default_rng(dim * rows + heads)
    lengths = [int(n) for n in rng.integers(rows, 150, batch)]
    lengths[0] = 257
    total = (sum(-(-n // size) for n in lengths) + 2) * size
    cache = filled(total, heads, dim, bits, group, page=size if size in (16, 32) else None)
    q = rng.standard_normal((batch, rows, heads * shared, dim)).astype(np.float32)
    check(cache, q, table(rng, lengths, size, total), lengths, size, dtype, weights=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bits, dim, group", [(8, 128, 128), (4, 128, 32), (8, 72, 72)])
@pytest.mark.parametrize("window", [None, 1, 7, 40, 10 ** 12])
def test_rows_and_window(dtype, bits, dim, group, window):
    """Lengths of 0 and 1 and below the rows', fewer rows than there is room for, lengths
    past the table."""
    rng = np.random.default_rng(3)
    lengths = [0, 1, 3, 100, 64, 5, 33, 10 ** 6, -4]
    n_rows = [4, 4, 4, 2, 0, 9, 1, 3, 4]
    size = 16
    total = 40 * size
    blocks = table(rng, [0, 1, 3, 100, 64, 5, 33, 128, 0], size, total)
    cache = filled(total, 2, dim, bits, group)
    q = rng.standard_normal((9, 4, 6, dim)).astype(np.float32)
    kw = {} if window is None else {"window": window}
    check(cache, q, blocks, lengths, size, dtype, weights=True, n_rows=n_rows, **kw)


@pytest.mark.parametrize("bits, dim, group", [(8, 128, 128), (4, 128, 32), (8, 34, 34)])
def test_slots_outside_the_cache(bits, dim, group):
    """A block id of -1, or past the end, inside a sequence: its tokens take no part."""
    rng = np.random.default_rng(4)
    size, total = 16, 20 * 16
    lengths = [100, 90, 40]
    blocks = table(rng, lengths, size, total)
    blocks[0, 2], blocks[1, 0], blocks[1, 5] = -1, 2 ** 31 - 1, 20
    blocks[2] = -7
    cache = filled(total, 2, dim, bits, group)
    q = rng.standard_normal((3, 2, 4, dim)).astype(np.float32)
    got = check(cache, q, blocks, lengths, size, "f32", weights=True)
    assert (got[2] == 0).all()


@pytest.mark.parametrize("dim", [128, 80, 40])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_where_nobody_looks(dim, dtype):
    """NaN codes in hidden tokens, behind the end and outside the window, do not count; a row
    that sees one has it."""
    rng = np.random.default_rng(5)
    size, total, n = 16, 96, 60
    cache = filled(total, 1, dim, 8, dim)
    blocks = np.arange(6, dtype=np.int32)[None]
    lengths = [n]
    bad = torch.full((1, 1, dim), float("nan"), device="cuda")
    for t in (n, n + 1, 70, 95, 0, 10):  # behind the end; before every row's window
        ops.cache_write(cache, (bad, bad), torch.tensor([t], device="cuda"))
    q = rng.standard_normal((1, 3, 2, dim)).astype(np.float32)
    kv = np.nan_to_num(held(cache))
    qd = torch.from_numpy(q).cuda().to(TYPES[dtype])
    args = (torch.from_numpy(blocks).cuda(), torch.tensor(lengths, dtype=torch.int32,
                                                          device="cuda"))
    kw = dict(block_size=size, window=40)
    got = ops.cache_attend(cache, qd, *args, **kw).double().cpu().numpy()
    want, off, _, _ = attended(kv, qd.double().cpu().numpy(), blocks, lengths, size, window=40,
                               dtype=dtype)
    assert (np.abs(got - want) <= off).all()
    # the last row alone sees the last token
    x = torch.full((1, 1, dim), 0.5, device="cuda")
    value = x.clone()
    value[..., dim // 2] = float("nan")
    ops.cache_write(cache, (x, value), torch.tensor([n - 1], device="cuda"))
    kv = held(cache)
    kv[:, [0, 10]] = 0.0
    got = ops.cache_attend(cache, qd, *args, **kw).double().cpu().numpy()
    want, off, _, _ = attended(kv, qd.double().cpu().numpy(), blocks, lengths, size, window=40,
                               dtype=dtype)
    assert np.isnan(got[0, 2, :, dim // 2]).all() and np.isnan(want[0, 2, :, dim // 2]).all()
    ok = np.isfinite(want)
    assert (np.isfinite(got) == ok).all() and ok[0, :2].all()
    assert (np.abs(got - want)[ok] <= off[ok]).all()
    # NaN as a key: rows that see it have no finite output
    ops.cache_write(cache, (bad, x), torch.tensor([n - 1], device="cuda"))
    got = ops.cache_attend(cache, qd, *args, **kw)
    assert got[0, 2].isnan().all() and got[0, :2].isfinite().all()


@pytest.mark.parametrize("bits, dim, group", [(8, 128, 128), (8, 128, 32), (4, 128, 32),
                                              (4, 80, 16), (8, 36, 36)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scales_far_apart(bits, dim, group, dtype):
    """Values of very different sizes: tokens of large values and little weight, tokens of
    small values and most of it, zeros."""
    rng = np.random.default_rng(6)
    size, total = 16, 256
    cache = filled(total, 2, dim, bits, group)
    g = torch.Generator("cuda").manual_seed(9)
    x = torch.randn(total, 2, dim, device="cuda", generator=g)
    mag = torch.exp(torch.randn(total, 1, 1, device="cuda", generator=g) * 6)
    mag[::5] = 0.0
    ops.cache_write(cache, (x * 2, x.flip(0) * mag), torch.arange(total, device="cuda"))
    blocks = np.arange(16, dtype=np.int32)[None]
    q = rng.standard_normal((1, 3, 4, dim)).astype(np.float32) * 2
    check(cache, q, blocks, [250], size, dtype, weights=True)
    # all of them large, and all of them tiny
    for s in (1e20, 1e-20):
        ops.cache_write(cache, (x, x * s), torch.arange(total, device="cuda"))
        if dtype == "f32" or s < 1e10:
            check(cache, q, blocks, [250], size, "f32")
    # queries far from 1, whose scores are not
    ops.cache_write(cache, (x * 1e-15, x), torch.arange(total, device="cuda"))
    check(cache, q * np.float32(1e15), blocks, [250], size, dtype if dtype == "bf16" else "f32")


@pytest.mark.parametrize("bits, group", [(8, 128), (4, 32)])
def test_peaked(bits, group):
    """Scores of hundreds: one token has all of the weight."""
    rng = np.random.default_rng(7)
    cache = filled(512, 2, 128, bits, group, spread=3.0)
    q = rng.standard_normal((1, 1, 8, 128)).astype(np.float32) * 20
    check(cache, q, np.arange(32, dtype=np.int32)[None], [500], 16, "bf16", weights=True)


@pytest.mark.parametrize("bits, group", [(8, 128), (4, 32)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides(bits, group, dtype):
    """Queries out of a fused projection, an output with gaps, heads-first storage."""
    rng = np.random.default_rng(8)
    heads, dim, size = 4, 128, 16
    cache = filled(320, heads, dim, bits, group, heads_first=True)
    lengths = [77, 130]
    blocks = table(rng, lengths, size, 320)
    fused = torch.from_numpy(rng.standard_normal((2, 3, 3 * 8 * dim)).astype(np.float32))
    fused = fused.cuda().to(TYPES[dtype])
    q = fused[..., :8 * dim].view(2, 3, 8, dim)
    room = torch.full((2, 3, 10, dim + 16), 7.0, device="cuda", dtype=TYPES[dtype])
    out = room[:, :, 1:9, 8:8 + dim]
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    got = ops.cache_attend(cache, q, torch.from_numpy(blocks).cuda(), lens, block_size=size,
                           out=out)
    assert got is out
    want, off, _, _ = attended(held(cache), q.double().cpu().numpy(), blocks, lengths, size,
                               dtype=dtype, reach=reach(cache))
    assert (np.abs(out.double().cpu().numpy() - want) <= off).all()
    out.fill_(7.0)
    assert (room == 7.0).all()
    # a token a sequence without the rows' axis, and queries at odd addresses
    odd = torch.empty(2 * 8 * dim + 1, device="cuda", dtype=TYPES[dtype])[1:].view(2, 8, dim)
    odd.copy_(q[:, 2])
    one = ops.cache_attend(cache, odd, torch.from_numpy(blocks).cuda(), lens, block_size=size)
    assert one.shape == (2, 8, dim)
    assert (np.abs(one.double().cpu().numpy() - want[:, 2]) <= off[:, 2]).all()


@pytest.mark.parametrize("rows", [2, 70])
@pytest.mark.parametrize("bits, dim, group", [(8, 128, 128), (4, 128, 32), (4, 80, 16),
                                              (8, 96, 32)])
def test_pages_among_others(bits, dim, group, rows):
    """A page holds several layers' slots, and codes and params start where they like: a
    layer's pages are apart, its addresses of any alignment."""
    rng = np.random.default_rng(30)
    heads, pages, page, layers = 4, 14, 16, 3
    tail, ptype = ((), torch.float32) if bits == 8 else ((2,), torch.bfloat16)
    for shift in (0, 8, 1):  # bytes; params stay on their words
        n = 2 * pages * layers * page * heads * (dim * bits // 8)
        codes = torch.zeros(n + 16, dtype=torch.uint8, device="cuda")[shift:shift + n]
        codes = codes.view(2, pages, layers, page, heads, -1)[:, :, 1]
        params = torch.zeros(2, pages, layers, page, heads, dim // group, *tail, dtype=ptype,
                             device="cuda")[:, :, 1]
        cache = ops.QuantCache(codes, params, dim=dim, bits=bits)
        x = [torch.randn(cache.slots, heads, dim, device="cuda") for _ in range(2)]
        ops.cache_write(cache, x, torch.arange(cache.slots, device="cuda"))
        lengths = [100, 75]
        q = rng.standard_normal((2, rows, heads * 3, dim)).astype(np.float32)
        check(cache, q, table(rng, lengths, page, cache.slots), lengths, page, "bf16",
              weights=True)


@pytest.mark.parametrize("bits, group, dtype", [(8, 128, "bf16"), (4, 32, "f16")])
def test_long_and_ragged(bits, group, dtype):
    rng = np.random.default_rng(10)
    lengths = [9000, 17, 1200, 0, 4097]
    total = (sum(-(-n // 16) for n in lengths) + 1) * 16
    cache = filled(total, 2, 128, bits, group, page=16)
    q = rng.standard_normal((5, 2, 8, 128)).astype(np.float32)
    check(cache, q, table(rng, lengths, 16, total), lengths, 16, dtype, weights=True)


def test_many_sequences():
    """More sequences than a warp has lanes, most of them empty."""
    rng = np.random.default_rng(11)
    lengths = [int(n) if n < 90 else 0 for n in rng.integers(0, 200, 150)]
    total = (sum(-(-n // 16) for n in lengths) + 1) * 16
    cache = filled(total, 2, 64, 8, 64, page=16)
    q = rng.standard_normal((150, 1, 4, 64)).astype(np.float32)
    check(cache, q, table(rng, lengths, 16, total), lengths, 16, "bf16", weights=True)


@pytest.mark.parametrize("bits, group", [(8, 128), (4, 32)])
@pytest.mark.parametrize("rows", [130, 300])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_prompt_chunk(bits, group, rows, dtype):
    rng = np.random.default_rng(12)
    lengths = [rows + 200, rows, 90]
    total = (sum(-(-n // 16) for n in lengths) + 1) * 16
    cache = filled(total, 1, 128, bits, group, page=16)
    q = rng.standard_normal((3, rows, 2, 128)).astype(np.float32)
    check(cache, q, table(rng, lengths, 16, total), lengths, 16, dtype, weights=True,
          n_rows=[rows, rows - 7, rows])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("window", [None, 100])
def test_many_rows(dtype, dim, window):
    """As many queries to a head as the tensor-memory kernels take: odd numbers of them, rows
    that see nothing or are not there, lengths below a tile and at its end."""
    rng = np.random.default_rng(20)
    rows, heads, shared = 97, 8, 3
    lengths = [97, 600, 128, 256, 5, 0, 301]
    n_rows = [97, 97, 60, 97, 97, 97, 0]
    total = (sum(-(-n // 16) for n in lengths) + 1) * 16
    cache = filled(total, heads, dim, 8, dim, page=16)
    blocks = table(rng, lengths, 16, total)
    blocks[1, 20] = -1  # 16 tokens that are not there
    q = rng.standard_normal((7, rows, heads * shared, dim)).astype(np.float32)
    kw = {} if window is None else {"window": window}
    check(cache, q, blocks, lengths, 16, dtype, weights=True, n_rows=n_rows, **kw)


@pytest.mark.parametrize("batch", [5, 9])
def test_many_rows_peaked_and_far(batch):
    """Scores of hundreds, and values of sizes far apart: what a row's weights are taken against
    moves often.  With few queries in all, and with as many as the tensor-memory kernels take."""
    rng = np.random.default_rng(21)
    cache = filled(1024, 8, 128, 8, 128, spread=3.0)
    g = torch.Generator("cuda").manual_seed(9)
    x = torch.randn(1024, 8, 128, device="cuda", generator=g)
    mag = torch.exp(torch.randn(1024, 1, 1, device="cuda", generator=g) * 4)
    mag[::5] = 0.0
    ops.cache_write(cache, (x * 2, x.flip(0) * mag), torch.arange(1024, device="cuda"))
    blocks = np.arange(64, dtype=np.int32)[None].repeat(batch, 0)
    lengths = [1000, 900, 777, 512, 300, 41, 128, 129, 1024][:batch]
    for scale in (None, 2.0, -1.0, 0.0):
        q = rng.standard_normal((batch, 40, 32, 128)).astype(np.float32)
        check(cache, q, blocks, lengths, 16, "bf16", scale=scale, weights=True)


@pytest.mark.parametrize("batch", [5, 6])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_many_rows_nan(dtype, batch):
    """NaN values where some rows do not look, and where all of them do."""
    rng = np.random.default_rng(22)
    cache = filled(512, 8, 128, 8, 128)
    blocks = np.arange(32, dtype=np.int32)[None].repeat(batch, 0)
    q = rng.standard_normal((batch, 130, 16, 128)).astype(np.float32)
    bad = torch.full((1, 8, 128), 0.5, device="cuda")
    bad[..., 7] = float("nan")
    fine = torch.full((1, 8, 128), 0.5, device="cuda")
    lengths = [400] * batch
    qd = torch.from_numpy(q).cuda().to(TYPES[dtype])
    args = (torch.from_numpy(blocks).cuda(),
            torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    # token 390 is hidden from rows below 120; tokens behind the end are nobody's
    for t in (390, 400, 511):
        ops.cache_write(cache, (fine, bad), torch.tensor([t], device="cuda"))
    got = ops.cache_attend(cache, qd, *args, block_size=16).double().cpu().numpy()
    assert np.isnan(got[:, 120:, :, 7]).all()
    got[:, 120:, :, 7] = 0.0
    assert np.isfinite(got).all()
    want, off, _, _ = attended(np.nan_to_num(held(cache)), qd[:1].double().cpu().numpy(),
                               blocks[:1], lengths[:1], 16, dtype=dtype)
    want[:, 120:, :, 7] = 0.0
    assert (np.abs(got[:1] - want) <= off).all()
    # seen by all
    ops.cache_write(cache, (fine, bad), torch.tensor([3], device="cuda"))
    got = ops.cache_attend(cache, qd, *args, block_size=16)
    assert got[..., 7].isnan().all() and got[..., :7].isfinite().all()


def test_block_larger_than_a_page_and_smaller():
    rng = np.random.default_rng(13)
    cache = filled(512, 2, 64, 8, 64, page=32)
    q = rng.standard_normal((2, 1, 4, 64)).astype(np.float32)
    for size in (1, 8, 32, 64, 256, 24):
        lengths = [100, 50]
        check(cache, q, table(rng, lengths, size, 512 // size * size), lengths, size, "f32")


def test_bits_are_the_same_every_time():
    rng = np.random.default_rng(14)
    lengths = [3000, 40, 700]
    total = (sum(-(-n // 16) for n in lengths) + 1) * 16
    cache = filled(total, 4, 128, 4, 32, page=16)
    q = torch.from_numpy(rng.standard_normal((3, 2, 16, 128)).astype(np.float32)).cuda()
    blocks = torch.from_numpy(table(rng, lengths, 16, total)).cuda()
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    runs = []
    for _ in range(5):
        w = torch.zeros(3, 4, blocks.size(1) * 16, device="cuda")
        runs.append((ops.cache_attend(cache, q, blocks, lens, block_size=16, weights=w), w))
    assert all(torch.equal(a, runs[0][0]) and torch.equal(b, runs[0][1]) for a, b in runs)


def test_offsets_past_32_bits():
    """Slots whose codes lie more than 4 GB from the first."""
    heads, dim, size = 8, 128, 16
    slots = (5 << 30) // (2 * heads * dim) // size * size + 4096
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("little memory")
    codes = torch.empty(2, slots, heads, dim, dtype=torch.uint8, device="cuda")
    params = torch.empty(2, slots, heads, 1, device="cuda")
    # one tensor of interleaved parts: a part's slots are 2 * heads * dim apart
    codes = codes.view(slots, 2, heads, dim).transpose(0, 1)
    cache = ops.QuantCache(codes, params, dim=dim, bits=8)
    g = torch.Generator("cuda").manual_seed(1)
    n = 200
    x = [torch.randn(n, heads, dim, device="cuda", generator=g) for _ in range(2)]
    base = slots - 256
    ops.cache_write(cache, x, torch.arange(base, base + n, device="cuda"))
    small = ops.QuantCache.allocate(256, heads, dim)
    ops.cache_write(small, x, torch.arange(n, device="cuda"))
    q = torch.randn(1, 2, 16, dim, device="cuda", generator=g).to(torch.bfloat16)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    ids = torch.arange(16, dtype=torch.int32, device="cuda")[None]
    a = ops.cache_attend(cache, q, ids + base // size, lens, block_size=size)
    b = ops.cache_attend(small, q, ids, lens, block_size=size)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bits, dim, group", [(8, 40, 40), (4, 112, 16), (8, 160, 10), (4, 300, 30),
                                              (8, 1024, 128), (4, 514, 514), (8, 1, 1)])
def test_widths_without_tensor_cores(bits, dim, group, dtype):
    """Queries of several rows in a block's four, more tokens than its warps take at once."""
    rng = np.random.default_rng(dim)
    rows, heads, shared = 3, 2, 3
    lengths, n_rows = [400, 0, 1, 33, 290], [3, 3, 3, 2, 0]
    total = (sum(-(-n // 16) for n in lengths) + 1) * 16
    cache = filled(total, heads, dim, bits, group, page=16)
    blocks = table(rng, lengths, 16, total)
    blocks[0, 4] = -1
    q = rng.standard_normal((5, rows, heads * shared, dim)).astype(np.float32)
    for window in (None, 37):
        kw = {} if window is None else {"window": window}
        check(cache, q, blocks, lengths, 16, dtype, weights=True, n_rows=n_rows, **kw)


@pytest.mark.parametrize("dim", [128, 72])
def test_empty_cache(dim):
    cache = ops.QuantCache.allocate(0, 2, dim)
    q = torch.randn(2, 3, 4, dim, device="cuda")
    blocks = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    lengths = torch.tensor([20, 0], dtype=torch.int32, device="cuda")
    weights = torch.ones(2, 2, 32, device="cuda")
    out = ops.cache_attend(cache, q, blocks, lengths, block_size=16, weights=weights)
    assert (out == 0).all() and (weights == 1).all()
