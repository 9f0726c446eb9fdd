"""The quantised cache on the GPU: codes, scaling and values bit for bit as defined."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from beam_oracle import e4m3_values, held_values, quantised  # noqa: E402
from grammar_constrained_logit_gb300 import ops  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from grammar_constrained_logit_gb300 import _lib

    _lib.load()


def held(cache, part, slots):
    """(code values [n, heads, groups, group], scale, low) that the cache's slots hold."""
    n = len(slots)
    codes, params = cache.codes[part], cache.params[part]
    if codes.dim() == 4:
        codes, params = codes.flatten(0, 1), params.flatten(0, 1)
    c = codes.cpu().numpy()[slots]
    p = params.float().cpu().numpy()[slots]
    if cache.bits == 8:
        code, scale, low = e4m3_values()[c], p, np.zeros_like(p)
    else:
        code = np.stack((c & 15, c >> 4), -1).astype(np.float64)
        scale, low = p[..., 0], p[..., 1]
    return code.reshape(n, cache.heads, -1, cache.group), scale, low


def rounded(v, dtype):
    return torch.from_numpy(v).to(TYPES[dtype])


def same(a, b):
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


def check(cache, xs, slots, dtype, out_dtype=None):
    """Writes, compares what is held, reads back, and compares that."""
    out_dtype = out_dtype or dtype
    before = cache.codes.clone(), cache.params.clone()
    dev = torch.from_numpy(slots).cuda()
    ops.cache_write(cache, xs, dev)
    ok = (slots >= 0) & (slots < cache.slots)
    back = ops.cache_read(cache, dev, dtype=TYPES[out_dtype])
    for part, x in enumerate(xs):
        code, scale, low = quantised(x.float().cpu().numpy()[ok], cache.bits, cache.group)
        c, s, m = held(cache, part, slots[ok])
        assert np.array_equal(c, code, equal_nan=True)
        assert np.array_equal(s, scale) and np.array_equal(m, low)
        want = np.zeros(x.shape, np.float32)
        want[ok] = held_values(code, scale, low, cache.bits)
        assert same(back[part].cpu(), rounded(want, out_dtype))
    # slots that nobody wrote keep their bytes
    rest = torch.ones(cache.slots, dtype=torch.bool)
    rest[slots[ok]] = False
    for now, was in zip((cache.codes, cache.params), before):
        if now.dim() - (cache.bits == 4 and now.dtype != torch.uint8) == 5:
            now, was = now.flatten(1, 2), was.flatten(1, 2)
        assert torch.equal(now[:, rest.cuda()], was[:, rest.cuda()])
    return back


def some_slots(rng, n, total, out=True):
    slots = rng.permutation(total)[:n].astype(np.int64)
    if out and n > 3:
        slots[1], slots[2], slots[n - 1] = -1, total, -(1 << 62)
    return slots


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("n, heads, dim, group", [
    (1, 1, 2, 2), (1, 8, 128, 128), (3, 1, 64, 64), (5, 3, 6, 6), (4, 2, 80, 16), (7, 5, 80, 40),
    (9, 2, 96, 32), (33, 8, 128, 32), (65, 1, 576, 64), (17, 2, 72, 72), (130, 4, 64, 8),
    (6, 2, 256, 256), (5, 1, 512, 512), (11, 3, 34, 34), (300, 8, 128, 128), (19, 2, 48, 24),
    (4, 1, 1030, 1030), (21, 16, 192, 16)])
def test_shapes(dtype, bits, n, heads, dim, group):
    rng = np.random.default_rng(n * dim + group)
    total = n + 9
    cache = ops.QuantCache.allocate(total, heads, dim, bits=bits, group=group)
    xs = [(torch.randn(n, heads, dim, device="cuda") * (1 + 3 * i) + i).to(TYPES[dtype])
          for i in range(2)]
    check(cache, xs, some_slots(rng, n, total), dtype)


def test_odd_group_in_8_bits():
    rng = np.random.default_rng(1)
    for dim, group in ((1, 1), (7, 7), (33, 11), (15, 5)):
        cache = ops.QuantCache.allocate(20, 3, dim, bits=8, group=group, parts=1)
        x = torch.randn(10, 3, dim, device="cuda").to(torch.bfloat16)
        check(cache, [x], some_slots(rng, 10, 20), "bf16")


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype, out_dtype", [("f32", "bf16"), ("bf16", "f32"), ("f16", "f32"),
                                              ("f32", "f16")])
def test_read_as_another_type(bits, dtype, out_dtype):
    rng = np.random.default_rng(2)
    cache = ops.QuantCache.allocate(50, 4, 64, bits=bits, group=32)
    xs = [(torch.randn(40, 4, 64, device="cuda") * 30).to(TYPES[dtype]) for _ in range(2)]
    check(cache, xs, some_slots(rng, 40, 50), dtype, out_dtype)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [16, 24, 128])
def test_values_at_the_edges(bits, dtype, group):
    """Groups of zeros, of one value, of the type's least and largest, infinities and NaN
    among finite ones and alone, ties between codes."""
    dim = group * 8
    rng = np.random.default_rng(3)
    info = torch.finfo(TYPES[dtype])
    x = torch.randn(6, 1, 8, group, dtype=torch.float64)
    x[0, 0, 0] = 0.0
    x[0, 0, 1] = 3.25
    x[0, 0, 2] = -7.0
    x[0, 0, 3, 0], x[0, 0, 3, 1] = info.max, info.min
    x[0, 0, 4] = info.tiny
    x[0, 0, 5] = torch.linspace(-1.0, 14.0, group)
    x[0, 0, 6, 3], x[0, 0, 6, 5] = float("inf"), float("-inf")
    x[0, 0, 7, 2] = float("nan")
    x[1, 0, 0] = float("inf")
    x[1, 0, 1] = float("nan")
    x[1, 0, 2] = float("-inf")
    x[1, 0, 3] = float("nan")
    x[1, 0, 3, 4] = 2.0
    x[1, 0, 4] = info.smallest_normal / 4
    x[1, 0, 5] = torch.arange(group) * 0.5 - 1.0       # half-way between codes
    x[1, 0, 5, -1] = 14.0
    x[1, 0, 6] = torch.arange(group) * 16.0 + 8.0
    x[1, 0, 6, -1] = 448.0                             # scale 1: ties of e4m3
    x[1, 0, 7, :3] = torch.tensor([1000.0, 1000.01, 999.99])
    x[2] *= 1e-6
    x[3] *= 1e4 if dtype != "f16" else 1e3
    x[4, 0, :, 0] = 50.0                               # one outlier
    x = x.to(TYPES[dtype]).view(6, 1, dim).cuda()
    cache = ops.QuantCache.allocate(9, 1, dim, bits=bits, group=group, parts=1)
    check(cache, [x], some_slots(rng, 6, 9, out=False), dtype)


@pytest.mark.parametrize("bits", [8, 4])
def test_error_of_the_values(bits):
    """Against the inputs themselves.  8 bits: half an e4m3 step, 2^-4 |x|, or of the
    least steps s 2^-10; and the 32-bit roundings.  4 bits: half a step s; what the
    rounding of the pair to bf16 takes from the ends, 15 * 2^-8 s and 2^-8 |lo|."""
    x = torch.randn(64, 4, 128, device="cuda", dtype=torch.float32) * 3 + 1
    cache = ops.QuantCache.allocate(64, 4, 128, bits=bits, group=32, parts=1)
    slots = torch.arange(64, device="cuda")
    ops.cache_write(cache, x, slots)
    v = ops.cache_read(cache, slots, dtype=torch.float32)[0].double()
    x = x.double()
    p = cache.params[0].double()
    if bits == 8:
        s = p.repeat_interleave(32, -1)
        most = x.abs() * (2.0 ** -4 + 2.0 ** -21) + s * 2.0 ** -10
    else:
        s = p[..., 0].repeat_interleave(32, -1)
        lo = x.view(64, 4, 4, 32).amin(-1).abs().repeat_interleave(32, -1)
        most = s * (0.5 + 15 * 2.0 ** -8 * 1.01) + (2.0 ** -8 + 2.0 ** -22) * lo + x.abs() * 2.0 ** -22
    assert bool(((v - x).abs() <= most).all())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("shift", [0, 1, 2, 3])
def test_strided_inputs_and_outputs(bits, shift):
    rng = np.random.default_rng(4)
    n, H, D = 21, 3, 64
    qkv = torch.randn(n, 5 * H * D + shift, device="cuda").to(torch.bfloat16)
    k = qkv[:, shift:shift + H * D].view(n, H, D) if shift == 0 else \
        qkv.as_strided((n, H, D), (5 * H * D + shift, D, 1), shift)
    v = torch.randn(H, n, D + shift, device="cuda").to(torch.bfloat16)[..., :D].transpose(0, 1)
    cache = ops.QuantCache.allocate(30, H, D, bits=bits, group=32)
    slots = some_slots(rng, n, 30)
    back = check(cache, [k, v], slots, "bf16")
    wide = torch.full((2, H, n, D + 3 + shift), 9.0, device="cuda", dtype=torch.bfloat16)
    outs = [wide[i, :, :, shift:shift + D].transpose(0, 1) for i in range(2)]
    got = ops.cache_read(cache, torch.from_numpy(slots).cuda(), out=outs)
    for a, b in zip(got, back):
        assert torch.equal(a, b)
    assert bool((wide[..., :shift] == 9).all()) and bool((wide[..., shift + D:] == 9).all())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("pages, page, H, D, group", [(5, 16, 2, 64, 32), (3, 7, 3, 80, 80),
                                                      (4, 1, 1, 128, 16), (1, 33, 4, 40, 20)])
def test_pages_and_heads_first_storage(bits, pages, page, H, D, group):
    """Slots on pages, in storage laid out [pages, heads, page_size, ...]."""
    rng = np.random.default_rng(5)
    codes = torch.randint(0, 256, (2, pages, H, page, D * bits // 8), dtype=torch.uint8,
                          device="cuda")
    params = (torch.randn(2, pages, H, page, D // group, device="cuda") if bits == 8 else
              torch.randn(2, pages, H, page, D // group, 2, device="cuda").to(torch.bfloat16))
    cache = ops.QuantCache(codes.transpose(2, 3), params.transpose(2, 3), dim=D, bits=bits)
    assert cache.slots == pages * page and cache.group == group
    n = pages * page - 1
    xs = [torch.randn(n, H, D, device="cuda").to(torch.float16) for _ in range(2)]
    check(cache, xs, some_slots(rng, n, pages * page), "f16")


def test_slots_beyond_32_bits():
    """Codes more than 4 GB into the cache."""
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    n = (5 << 30) // 256 + 3
    cache = ops.QuantCache.allocate(n, 1, 256, bits=8, parts=1)
    x = torch.randn(4, 1, 256, device="cuda")
    slots = torch.tensor([n - 1, 0, (4 << 30) // 256, 5], device="cuda")
    ops.cache_write(cache, x, slots)
    code, scale, low = quantised(x.cpu().numpy(), 8, 256)
    back = ops.cache_read(cache, slots, dtype=torch.float32)[0].cpu().numpy()
    assert np.array_equal(back, held_values(code, scale, low, 8))
    assert int((cache.params != 0).sum()) == 4


def test_empty_stream_and_graph():
    cache = ops.QuantCache.allocate(8, 2, 64, bits=4)
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    x = torch.randn(0, 2, 64, device="cuda")
    ops.cache_write(cache, [x, x], none)
    assert ops.cache_read(cache, none)[0].shape == (0, 2, 64)
    empty = ops.QuantCache.allocate(0, 2, 64)
    s = torch.tensor([0, 3], device="cuda")
    y = torch.randn(2, 2, 64, device="cuda")
    ops.cache_write(empty, [y, y], s)
    assert not ops.cache_read(empty, s)[1].any()
    xs = [torch.randn(2, 2, 64, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.cache_write(cache, xs, s)
        got = ops.cache_read(cache, s, dtype=torch.float32)
    side.synchronize()
    out = [torch.empty_like(t) for t in xs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.cache_write(cache, xs, s)
        ops.cache_read(cache, s, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], got[0]) and torch.equal(out[1], got[1])
    xs[0].mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    code, scale, low = quantised(xs[0].cpu().numpy(), 4, 32)
    assert np.array_equal(out[0].cpu().numpy(), held_values(code, scale, low, 4))


def test_codes_and_params_follow_their_beams():
    """The cache's tensors as states of a reorder, its slots those of the beams' rows."""
    batch, beams, T, H, D = 2, 3, 10, 2, 64
    cache = ops.QuantCache.allocate(batch * beams * T, H, D, bits=4)
    slots = torch.arange(batch * beams * T, device="cuda")
    xs = [torch.randn(batch * beams * T, H, D, device="cuda") for _ in range(2)]
    ops.cache_write(cache, xs, slots)
    was = [t.view(batch * beams, T, H, D) for t in ops.cache_read(cache, slots)]
    rows = [(t.unflatten(1, (batch * beams, T)), 1, 2) for t in (cache.codes, cache.params)]
    p = torch.tensor([[2, 0, 0], [1, 1, 2]], dtype=torch.int32, device="cuda")
    ops.reorder_states(rows, p, stop=torch.tensor([10, 4], dtype=torch.int32, device="cuda"))
    now = [t.view(batch * beams, T, H, D) for t in ops.cache_read(cache, slots)]
    for a, b in zip(now, was):
        assert torch.equal(a[:3], b[[2, 0, 0]])
        assert torch.equal(a[3:, :4], b[[4, 4, 5], :4]) and torch.equal(a[3:, 4:], b[3:, 4:])


def test_bad_arguments():
    cache = ops.QuantCache.allocate(8, 2, 64)
    x = torch.zeros(3, 2, 64, device="cuda")
    s = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in ((x, x[:2]), (x,), (x, x[..., :32]), (x, x.cpu())):
        with pytest.raises(ValueError):
            ops.cache_write(cache, bad, s)
    for bad in ((x, x.half()), (x.double(), x.double())):
        with pytest.raises(TypeError):
            ops.cache_write(cache, bad, s)
    with pytest.raises(TypeError):
        ops.cache_write(cache, (x, x), s.int())
    with pytest.raises(ValueError):
        ops.cache_read(cache, s.cpu())
    with pytest.raises(ValueError):
        ops.cache_write(cache, (x, x.transpose(1, 2).contiguous().transpose(1, 2)), s)
    with pytest.raises(TypeError):
        ops.cache_read(cache, s, dtype=torch.float64)
    with pytest.raises(ValueError):
        ops.QuantCache(cache.codes, cache.params, dim=96)
    with pytest.raises(ValueError):
        ops.QuantCache(cache.codes[:, :4], cache.params, dim=64)
