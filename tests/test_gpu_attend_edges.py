"""Attention over the quantised cache where it is called in earnest at an edge: tables that share
their memory, tokens that hold no numbers, values of every size."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from grammar_constrained_logit_gb300 import ops  # noqa: E402
from test_gpu_attend import filled  # noqa: E402

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
