"""What attention over the cache and eviction hand to the library, followed on the host: nothing
here reaches a GPU."""
import pytest

torch = pytest.importorskip("torch")

from grammar_constrained_logit_gb300 import ops  # noqa: E402
from test_attend_args import INT, _cache, _gpu  # noqa: E402
from test_beam_calls import OnGpu  # noqa: E402

# where a call has its block table, and the blocks' stride, count and size behind it
ATTEND, EVICT = 13, 12


@pytest.fixture
def handed(monkeypatch):
    """The arguments of the calls that would be made, and block tables as they are then."""
    calls = []
    monkeypatch.setattr(ops, "_call", lambda name, device, args: calls.append(args))
    monkeypatch.setattr(ops, "_raw_stream", lambda index: 0)
    return calls


def attend(blocks, batch=3, **kw):
    ops.cache_attend(_cache(), _gpu(batch, 1, 4, 64), blocks, _gpu(batch, dtype=INT),
                     out=_gpu(batch, 1, 4, 64), block_size=16,
                     workspace=_gpu(4096, dtype=torch.uint8), **kw)


def evict(blocks, batch=3):
    ops.cache_evict(_cache(), _gpu(batch, 2, 64), blocks, _gpu(batch, dtype=INT), 16,
                    block_size=16, out=_gpu(batch, dtype=INT),
                    workspace=_gpu(4096, dtype=torch.uint8))


def tables():
    row = torch.arange(8, dtype=INT)
    return {"expanded": row[None, :4].expand(3, 4), "overlapping": row.as_strided((3, 4), (2, 1)),
            "one block": row[:1].view(1, 1).expand(3, 1)}


@pytest.mark.parametrize("kind", ["expanded", "overlapping", "one block"])
def test_rows_that_share_memory(handed, monkeypatch, kind):
    """Attention reads a copy whose rows are apart; eviction refuses."""
    table = tables()[kind]
    copies = []
    contiguous = torch.Tensor.contiguous
    monkeypatch.setattr(torch.Tensor, "contiguous",
                        lambda t: copies.append(contiguous(t)) or copies[-1])
    attend(OnGpu(table))
    (args,) = handed
    (copy,) = copies
    n = table.size(1)
    assert args[ATTEND:ATTEND + 4] == (copy.data_ptr(), n, n, 16)
    assert copy.is_contiguous() and torch.equal(copy, table)
    with pytest.raises(ValueError, match="overlap"):
        evict(OnGpu(table))
    assert len(handed) == 1


@pytest.mark.parametrize("shape, stride", [((3, 4), (4, 1)), ((3, 4), (7, 1)), ((3, 1), (1, 5)),
                                           ((1, 4), (0, 1)), ((1, 4), (2, 1)), ((3, 0), (1, 1))])
def test_rows_apart(handed, shape, stride):
    """Others go to the library as they are, rows by their stride."""
    table = torch.zeros(40, dtype=INT).as_strided(shape, stride)
    for call, at in ((attend, ATTEND), (evict, EVICT)):
        call(OnGpu(table), batch=shape[0])
        want = max(stride[0], shape[1]) if shape[0] == 1 else stride[0]
        assert handed.pop()[at:at + 4] == (table.data_ptr(), want, shape[1], 16)
