"""Attention over the quantised cache where it is called in earnest at an edge: tables that share
their memory, tokens that hold no numbers, values of every size."""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from grammar_constrained_logit_gb300 import ops  # noqa: E402
from test_gpu_attend import check, filled  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from grammar_constrained_logit_gb300 import _lib

    _lib.load()


@pytest.mark.parametrize("rows", [1, 60])
@pytest.mark.parametrize("bits, dim, group", [(8, 128, 128), (4, 128, 32), (8, 72, 72)])
def test_one_table_for_all(bits, dim, group, rows):
    """Several answers to one prompt share its blocks, by a table that is expanded."""
    cache = filled(512, 8, dim, bits, group, page=16)
    row = torch.from_numpy(np.random.default_rng(1).permutation(32).astype(np.int32)).cuda()
    g = torch.Generator("cuda").manual_seed(2)
    q = torch.randn(6, rows, 16, dim, device="cuda", generator=g).to(torch.bfloat16)
    lengths = torch.tensor([500, 60, 333, 512, 16, 17], dtype=torch.int32, device="cuda")
    for table in (row[None].expand(6, 32), row.as_strided((6, 20), (2, 1))):
        apart = table.clone(memory_format=torch.contiguous_format)
        got, want = (ops.cache_attend(cache, q, t, lengths) for t in (table, apart))
        assert torch.equal(got, want)
    # a graph has its own copy of the table
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
    table = row[None].expand(6, 32)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        ops.cache_attend(cache, q, table, lengths, out=out)
    torch.cuda.current_stream().wait_stream(stream)
    with torch.cuda.graph(graph):
        ops.cache_attend(cache, q, table, lengths, out=out)
    row.copy_(row.flip(0))
    out.zero_()
    graph.replay()
    assert torch.equal(out, ops.cache_attend(cache, q, table.contiguous(), lengths))


def spoil(cache, t, bad, part=1):
    """Puts what is no number into a token's params, in each of its groups in turn."""
    params = cache.params.flatten(1, 2) if cache.codes.dim() == 5 else cache.params
    for i in range(params.size(3)):
        if cache.bits == 8:
            params[part, t, :, i] = bad
        else:
            params[part, t, :, i, i % 2] = bad


SPOILT = [float("nan"), float("inf"), -float("inf")]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bits, dim, group, rows, shared", [
    (8, 128, 128, 3, 2), (8, 128, 32, 3, 2), (8, 64, 64, 5, 4), (8, 72, 72, 3, 2),
    (4, 128, 32, 3, 2), (4, 128, 128, 2, 8), (4, 80, 16, 6, 3), (4, 192, 64, 3, 2),
    (4, 112, 16, 3, 2), (8, 128, 128, 130, 2), (8, 64, 64, 130, 2)])
def test_params_that_are_no_numbers(bits, dim, group, rows, shared, dtype):
    """Scales and lows of tokens that a row does not see, before its window and behind it, do
    not count, whatever they are, keys' as values'; rows that see them have no number."""
    n, window, batch = 400, 150, 6
    g = torch.Generator("cuda").manual_seed(dim)
    q = torch.randn(batch, rows, 8 * shared, dim, device="cuda", generator=g).to(dtype)
    blocks = torch.arange(32, dtype=torch.int32, device="cuda").expand(batch, 32).contiguous()
    lengths = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    cache = filled(512, 8, dim, bits, group, page=16)
    want = ops.cache_attend(cache, q, blocks, lengths, window=window)
    weights = torch.zeros(batch, 8, 512, device="cuda")
    ops.cache_attend(cache, q, blocks, lengths, window=window, weights=weights)
    last = n - rows  # what the first row sees last
    for bad in SPOILT:
        cache = filled(512, 8, dim, bits, group, page=16)
        # nobody sees these, though they share a tile with tokens that somebody sees
        for t in (last - window, last - window - 1, n, n + 1):
            for part in range(2):
                spoil(cache, t, bad, part)
        again = torch.zeros_like(weights)
        got = ops.cache_attend(cache, q, blocks, lengths, window=window, weights=again)
        assert torch.equal(got, want) and torch.equal(again, weights)
        # the last row alone sees the last token
        spoil(cache, n - 1, bad)
        got = ops.cache_attend(cache, q, blocks, lengths, window=window)
        assert torch.equal(got[:, :-1], want[:, :-1]) and not got[:, -1].isfinite().any()
        # the first row alone sees what its window begins with
        spoil(cache, last - window + 1, bad)
        got = ops.cache_attend(cache, q, blocks, lengths, window=window)
        assert torch.equal(got[:, 1:-1], want[:, 1:-1])
        assert not got[:, 0].isfinite().any() and not got[:, -1].isfinite().any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits, dim, group", [(8, 128, 32), (4, 128, 32), (4, 80, 16), (8, 72, 24)])
def test_a_group_that_is_no_number(bits, dim, group, dtype):
    """A value's group that is no number leaves the head's other elements as they are, whether
    all rows see the token or some."""
    g = torch.Generator("cuda").manual_seed(dim)
    q = torch.randn(2, 4, 4, dim, device="cuda", generator=g).to(dtype)
    blocks = torch.arange(20, dtype=torch.int32, device="cuda").expand(2, 20).contiguous()
    lengths = torch.full((2,), 300, dtype=torch.int32, device="cuda")
    # (token, the first row that sees it)
    for (t, first), bad in itertools.product(((40, 0), (299, 3)), SPOILT):
        cache = filled(320, 2, dim, bits, group)
        for bits_of_it in range(1 if bits == 8 else 2):
            was = cache.params[1, t].clone()
            zeroed = cache.params[1, t, :, 1].clone()
            cache.params[1, t, :, 1] = 0.0
            want = ops.cache_attend(cache, q, blocks, lengths, block_size=16)
            cache.params[1, t, :, 1] = zeroed
            (cache.params[1, t, :, 1] if bits == 8 else
             cache.params[1, t, :, 1, bits_of_it]).fill_(bad)
            got = ops.cache_attend(cache, q, blocks, lengths, block_size=16)
            cache.params[1, t] = was
            mine = slice(group, 2 * group)
            assert not got[:, first:, :, mine].isfinite().any()
            got[..., mine] = want[..., mine] = 0.0
            assert (got.double() - want.double()).abs().max() < 2.0 ** -7 * want.abs().max()
            # (the token's largest scale may have been that group's: weights are rounded anew)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bits, dim, group, batch, rows", [
    (8, 128, 128, 1, 3), (8, 128, 32, 1, 3), (4, 128, 32, 1, 3), (4, 80, 16, 1, 3),
    (8, 36, 36, 1, 3), (8, 128, 128, 6, 40), (8, 64, 64, 6, 40)])
def test_values_of_every_size(bits, dim, group, batch, rows, dtype):
    """Values that are all large, and all so small that their scales are below 2^-60: each type's
    own rounding, by the kernels of few queries and of many."""
    rng = np.random.default_rng(40)
    cache = filled(256, 8, dim, bits, group)
    g = torch.Generator("cuda").manual_seed(41)
    x = torch.randn(256, 8, dim, device="cuda", generator=g)
    blocks = np.arange(16, dtype=np.int32)[None].repeat(batch, 0)
    q = rng.standard_normal((batch, rows, 32, dim)).astype(np.float32) * 2
    # (fp16 has neither, and a step of 2^-24 where it is smallest)
    for size in (1e3, 1e-2) if dtype == "f16" else (1e20, 1e-20, 1e30):
        ops.cache_write(cache, (x, x.flip(0) * size), torch.arange(256, device="cuda"))
        check(cache, q, blocks, [250] * batch, 16, dtype, weights=True)
