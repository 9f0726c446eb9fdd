"""The states' reorder on the GPU against its plain definition, bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from beam_oracle import reordered  # noqa: E402
from grammar_constrained_logit_gb300 import ops  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from grammar_constrained_logit_gb300 import _lib

    _lib.load()


def parents_of(rng, batch, beams, wild=True):
    p = rng.integers(0, beams, (batch, beams)).astype(np.int32)
    p[0] = (np.arange(beams) + 1) % beams  # one cycle through all rows
    if batch > 1:
        p[1] = np.arange(beams)            # nothing moves
    if batch > 2 and wild:
        p[2, ::2] = [-1, beams, 1 << 30, -(1 << 31)][beams % 4]
    if batch > 3:
        p[3] = beams - 1                   # all from the last
    return p


def check(t, rows, tokens, parents, start=None, stop=None):
    """Reorders t (a view of a larger buffer) and compares the whole buffer."""
    cpu = t.cpu().numpy() if t.dtype != torch.bfloat16 else t.view(torch.int16).cpu().numpy()
    dev = [None if x is None else torch.from_numpy(np.asarray(x, np.int32)).cuda()
           for x in (parents, start, stop)]
    ops.reorder_states([(t, rows, tokens)], *dev)
    got = t.cpu().numpy() if t.dtype != torch.bfloat16 else t.view(torch.int16).cpu().numpy()
    if tokens is None:
        want = np.moveaxis(cpu, rows, 0)
        want = np.moveaxis(reordered(want[:, None], parents)[:, 0], 0, rows)
    else:
        want = np.moveaxis(cpu, (rows, tokens), (0, 1))
        want = np.moveaxis(reordered(want, parents, start, stop), (0, 1), (rows, tokens))
    assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype", [torch.uint8, torch.bfloat16, torch.float32, torch.int64])
@pytest.mark.parametrize("batch, beams, width", [
    (1, 1, 5), (1, 2, 1), (5, 3, 7), (4, 4, 16), (5, 5, 1001), (4, 8, 4096), (5, 10, 33000),
    (4, 16, 257), (3, 17, 640), (2, 31, 100), (4, 32, 31), (4, 33, 63), (2, 64, 5000),
    (2, 255, 77), (1, 256, 1024)])
def test_flat_rows(dtype, batch, beams, width):
    rng = np.random.default_rng(beams * 1000 + width)
    t = torch.randint(-100 if dtype != torch.uint8 else 0, 100, (batch * beams, width),
                      device="cuda").to(dtype)
    check(t, 0, None, parents_of(rng, batch, beams))


@pytest.mark.parametrize("offset", [0, 1, 2, 4, 8, 24])
@pytest.mark.parametrize("width", [64, 65, 66, 68, 72])
def test_alignment(offset, width):
    rng = np.random.default_rng(offset + width)
    buf = torch.randint(0, 256, (offset + 12 * width + 40,), dtype=torch.uint8, device="cuda")
    keep = buf.cpu().numpy()
    t = buf[offset:offset + 12 * width].view(12, width)
    check(t, 0, None, parents_of(rng, 4, 3))
    after = buf.cpu().numpy()
    assert np.array_equal(after[:offset], keep[:offset])
    assert np.array_equal(after[offset + 12 * width:], keep[offset + 12 * width:])


@pytest.mark.parametrize("layout", ["tokens", "heads", "sliced", "interleaved", "last", "strided"])
@pytest.mark.parametrize("T, H, D", [(1, 1, 1), (7, 3, 5), (33, 2, 8), (129, 2, 64), (600, 4, 32)])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.bfloat16])
def test_layouts_and_ranges(layout, T, H, D, dtype):
    rng = np.random.default_rng(T + D)
    batch, beams = 5, 3
    R = batch * beams

    def rand(*shape):
        return torch.randint(0, 200, shape, device="cuda").to(dtype)

    t, rows, tokens = {
        "tokens": lambda: (rand(2, R, T, H, D), 1, 2),
        "heads": lambda: (rand(2, R, H, T, D), 1, 3),
        "sliced": lambda: (rand(2, R, H, T + 9, D)[:, :, :, 3:3 + T], 1, 3),
        "interleaved": lambda: (rand(R, T, 2, H, D)[:, :, 1], 0, 1),
        "last": lambda: (rand(R, D, T), 0, 2),
        "strided": lambda: (rand(T, R, H, 2 * D)[..., :D], 1, 0)}[layout]()
    base = t._base if t._base is not None else t
    before = base.clone()
    parents = parents_of(rng, batch, beams)
    start = np.array([0, 0, T // 3, T // 2, -5])
    stop = np.array([T, T, T // 2 + 1, T // 2, T + 50])
    for lo, hi in ((None, None), (start, None), (None, stop), (start, stop), (stop, start)):
        check(t, rows, tokens, parents, lo, hi)
    # what is not the view's is untouched
    mark = torch.zeros_like(base, dtype=torch.bool)
    mark.as_strided(t.shape, t.stride(), t.storage_offset()).fill_(True)
    assert torch.equal(base[~mark], before[~mark])


def test_extreme_ranges():
    t = torch.randint(0, 200, (4, 40, 3), dtype=torch.uint8, device="cuda")
    big = (1 << 31) - 1
    check(t, 0, 1, np.array([[1, 0], [1, 0]]), [-big, big], [big, -big])
    check(t, 0, 1, np.array([[1, 0], [1, 0]]), [39, 40], [40, 41])


def test_many_states_in_one_call():
    """More states than one launch takes, of several types, one of them empty."""
    rng = np.random.default_rng(1)
    batch, beams = 3, 4
    p = parents_of(rng, batch, beams)
    states, want = [], []
    for i in range(150):
        t = torch.randn(batch * beams, 1 + i % 7, 1 + i % 3, device="cuda")
        t = t.to([torch.float32, torch.bfloat16, torch.float16][i % 3])
        if i == 70:
            t = t[:, :0]
        states.append((t, 0, 1))
        want.append(torch.from_numpy(reordered(t.float().cpu().numpy(), p, None, [2, 9, 1])))
    ops.StateReorder(states, batch, beams).reorder(
        torch.from_numpy(p).cuda(), stop=torch.tensor([2, 9, 1], dtype=torch.int32, device="cuda"))
    for (t, _, _), w in zip(states, want):
        assert torch.equal(t.float().cpu(), w)


def test_offsets_beyond_32_bits():
    """Rows that lie more than 4 GB apart."""
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    buf = torch.empty(3 * (1 << 32) + 4096, dtype=torch.uint8, device="cuda")
    t = buf[:3 * (1 << 32)].view(3, 1 << 32)[:, -5000:]
    t.copy_(torch.randint(0, 256, t.shape, dtype=torch.uint8, device="cuda"))
    check(t, 0, None, np.array([[2, 0, 1]], dtype=np.int32))


def test_stream_and_graph():
    t = torch.arange(8, device="cuda").repeat_interleave(1000).view(8, 1000).float()
    p = torch.tensor([[1, 2, 3, 0], [0, 0, 1, 1]], dtype=torch.int32, device="cuda")
    m = ops.StateReorder([t], 2, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.reorder(p)
    side.synchronize()
    assert t[:, 0].tolist() == [1, 2, 3, 0, 4, 4, 5, 5] and bool((t == t[:, :1]).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.reorder(p)
    g.replay()
    torch.cuda.synchronize()
    assert t[:, 999].tolist() == [2, 3, 0, 1, 4, 4, 4, 4]


def test_bad_arguments():
    t = torch.zeros(8, 10, device="cuda")
    m = ops.StateReorder([t], 2, 4)
    p = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        m.reorder(p.long())
    with pytest.raises(ValueError):
        m.reorder(p.cpu())
    with pytest.raises(ValueError):
        m.reorder(p[:, :3])
    with pytest.raises(ValueError):
        m.reorder(p, start=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ops.StateReorder([t], 2, 5)
    with pytest.raises(ValueError):
        ops.StateReorder([t.expand(2, 8, 10)], 1, 2)
    with pytest.raises(ValueError):
        ops.StateReorder([(t, 0, 0)], 2, 4)
