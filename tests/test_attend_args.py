"""Arguments of attention over the cache, eviction and verification that are refused on the
host: nothing here reaches a GPU.  Also pins of the plain definitions that the GPU tests
compare with."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from attend_oracle import attended, evicted, row_probs, verified  # noqa: E402
from grammar_constrained_logit_gb300 import _lib, build, ops  # noqa: E402
from test_beam_calls import OnGpu, recorded  # noqa: E402, F401

FAKE = 0x10000  # never dereferenced: every call below is refused or has nothing to do


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _parts(n=2, **kw):
    a = dict(codes=FAKE, params=FAKE, code_page_stride=0, code_slot_stride=1024,
             code_head_stride=128, param_page_stride=0, param_slot_stride=32, param_head_stride=4)
    a.update(kw)
    return (_lib.CachePart * n)(*[_lib.CachePart(**a) for _ in range(n)])


def _attend(lib, **kw):
    a = dict(parts=_parts(), bits=8, n_slots=64, page=16, heads=8, dim=128, group=128,
             q=_at(FAKE), out=_at(2 * FAKE), dt=2, batch=2, rows=1, q_heads=32, blocks=FAKE, blocks_stride=4,
             max_blocks=4, block=16, lengths=FAKE, n_rows=None, scale=0.1, window=0,
             weights=None, wb=0, wh=0, ws=FAKE, ws_bytes=1 << 40, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.lp_cache_attend(*a.values())


def _at(p):
    return ctypes.byref(_lib.Rows(p, 4096, 4096, 128))


@pytest.mark.parametrize("kw, want", [
    (dict(dt=3), 2), (dict(dt=-1), 2),
    (dict(bits=5), 1), (dict(n_slots=-1), 1), (dict(page=0), 1), (dict(heads=-1), 1),
    (dict(dim=-1), 1), (dict(group=0), 1), (dict(group=48), 1), (dict(bits=4, dim=9, group=9), 1),
    (dict(batch=-1), 1), (dict(rows=-1), 1), (dict(q_heads=-8), 1), (dict(q_heads=12), 1),
    (dict(heads=0), 1), (dict(max_blocks=-1), 1), (dict(block=0), 1), (dict(blocks_stride=3), 1),
    (dict(window=-1), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(parts=None), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(q=_at(None)), 1),
    (dict(out=_at(None)), 1), (dict(out=_at(FAKE)), 1), (dict(q=_at(FAKE + 1)), 1), (dict(out=_at(FAKE + 1)), 1),
    (dict(dt=0, q=_at(FAKE + 2)), 1), (dict(blocks=None), 1), (dict(lengths=None), 1),
    (dict(blocks=FAKE + 2), 1), (dict(lengths=FAKE + 1), 1), (dict(n_rows=FAKE + 2), 1),
    (dict(weights=FAKE + 2), 1), (dict(ws=None), 1), (dict(ws=FAKE + 8), 1), (dict(ws_bytes=0), 1),
    (dict(parts=_parts(codes=None)), 1), (dict(parts=_parts(params=None)), 1),
    (dict(parts=_parts(params=FAKE + 2)), 1), (dict(parts=_parts(param_slot_stride=6)), 1),
    (dict(dim=1025, group=1025), 4), (dict(max_blocks=1 << 20, block=1 << 11,
                                           blocks_stride=1 << 20), 4),
    (dict(rows=1 << 20), 4), (dict(batch=1 << 31), 4), (dict(batch=1 << 27), 4),
    (dict(batch=0), 0), (dict(rows=0), 0), (dict(q_heads=0), 0), (dict(heads=0, q_heads=0), 0),
    (dict(dim=0, group=1), 0), (dict(batch=0, parts=None, q=None, lengths=None, ws=None), 0),
])
def test_attend_refusals(lib, kw, want):
    assert _attend(lib, **kw) == want


def test_attend_workspace_bytes(lib):
    f = lib.lp_cache_attend_workspace_bytes
    assert f(0, 1, 8, 8, 128) >= 0 and f(2, 1, 32, 8, 128) >= 2 * 32 * 4
    for bad in ((-1, 1, 8, 8, 128), (1, -1, 8, 8, 128), (1, 1, -8, 8, 128), (1, 1, 8, -8, 128),
                (1, 1, 8, 8, -1), (1, 1, 8, 8, 1025), (1, 1 << 30, 1 << 30, 8, 64),
                (1 << 40, 1, 8, 8, 64)):
        assert f(*bad) == -1


def _evict(lib, **kw):
    a = dict(parts=_parts(), n_parts=2, bits=8, n_slots=64, page=16, heads=8, dim=128, group=128,
             weights=FAKE, wb=512, wh=64, batch=2, blocks=FAKE, blocks_stride=4, max_blocks=4,
             block=16, lengths=FAKE, keep=32, first=4, recent=8, new=FAKE + 64, ws=FAKE,
             ws_bytes=1 << 40, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.lp_cache_evict(*a.values())


@pytest.mark.parametrize("kw, want", [
    (dict(n_parts=-1), 1), (dict(n_parts=9), 1), (dict(bits=3), 1), (dict(n_slots=-1), 1),
    (dict(page=0), 1), (dict(heads=-1), 1), (dict(dim=-1), 1), (dict(group=0), 1),
    (dict(group=48), 1), (dict(bits=4, dim=9, group=9), 1), (dict(batch=-1), 1),
    (dict(max_blocks=-1), 1), (dict(block=0), 1), (dict(blocks_stride=3), 1),
    (dict(keep=-1, first=0, recent=0), 1), (dict(first=-1), 1), (dict(recent=-1), 1),
    (dict(first=33), 1), (dict(first=25), 1), (dict(parts=None), 1), (dict(weights=None), 1),
    (dict(blocks=None), 1), (dict(lengths=None), 1), (dict(new=None), 1), (dict(new=FAKE), 1),
    (dict(new=FAKE + 4), 1), (dict(lengths=FAKE + 2), 1), (dict(weights=FAKE + 1), 1),
    (dict(ws=None), 1), (dict(ws=FAKE + 8), 1), (dict(ws_bytes=0), 1),
    (dict(parts=_parts(codes=None)), 1), (dict(parts=_parts(params=FAKE + 2)), 1),
    (dict(parts=_parts(param_head_stride=2)), 1),
    (dict(dim=1 << 30, group=1 << 30), 4), (dict(batch=1 << 31), 4), (dict(heads=1 << 31), 4),
    (dict(max_blocks=1 << 20, block=1 << 11, blocks_stride=1 << 20), 4),
    (dict(batch=0), 0), (dict(batch=0, parts=None, weights=None, lengths=None, new=None), 0),
])
def test_evict_refusals(lib, kw, want):
    assert _evict(lib, **kw) == want


def test_evict_workspace_bytes(lib):
    f = lib.lp_cache_evict_workspace_bytes
    assert f(0, 8, 100) >= 0 and f(2, 8, 100) >= 2 * 8 * 100 * 4
    for bad in ((-1, 8, 100), (1, -8, 100), (1, 8, -1), (1 << 20, 1 << 20, 1), (1, 1, 1 << 31)):
        assert f(*bad) == -1


def _verify(lib, **kw):
    a = dict(logits=FAKE, dt=2, B=8, cols=64, stride=64, bm=None, bm_rows=0, words=0, bm_stride=0,
             vocab=-1, needs=None, per=4, drafts=FAKE, probs=FAKE, ps=192, pr=64, u=FAKE,
             temp=None, t=1.0, seed=1, offset=2, seeds=None, tokens=FAKE, accepted=FAKE, ws=FAKE,
             ws_bytes=1 << 40, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.lp_verify_drafts(*a.values())


MASK = dict(bm=FAKE, bm_rows=8, words=2, bm_stride=2)


@pytest.mark.parametrize("kw, want", [
    (dict(dt=3), 2), (dict(dt=-1), 2), (dict(B=-4), 1), (dict(cols=-1), 1), (dict(stride=63), 1),
    (dict(per=0), 1), (dict(per=3), 1), (dict(vocab=65), 1), (dict(needs=FAKE), 1),
    (dict(MASK, bm_rows=7), 1), (dict(MASK, words=-1), 1), (dict(MASK, bm_stride=1), 1),
    (dict(MASK, vocab=64, words=1), 1), (dict(MASK, words=1 << 60, bm_stride=1 << 60), 1),
    (dict(MASK, bm=FAKE + 2), 1),
    (dict(logits=None), 1), (dict(logits=FAKE + 1), 1), (dict(stride=1 << 60), 1),
    (dict(drafts=None), 1), (dict(drafts=FAKE + 4), 1), (dict(u=None), 1), (dict(u=FAKE + 2), 1),
    (dict(probs=FAKE + 2), 1), (dict(temp=FAKE + 2), 1), (dict(seeds=FAKE + 4), 1),
    (dict(tokens=None), 1), (dict(tokens=FAKE + 4), 1), (dict(accepted=None), 1),
    (dict(accepted=FAKE + 2), 1), (dict(ws=None), 1), (dict(ws=FAKE + 8), 1), (dict(ws_bytes=0), 1),
    (dict(B=514, per=257), 4), (dict(B=1 << 28), 4), (dict(cols=1 << 31, stride=1 << 31), 4),
    (dict(B=0), 0), (dict(B=0, logits=None, drafts=None, tokens=None, ws=None), 0),
])
def test_verify_refusals(lib, kw, want):
    assert _verify(lib, **kw) == want


def test_verify_workspace_bytes(lib):
    f = lib.lp_verify_drafts_workspace_bytes
    assert f(0, 0, 5) >= 0 and f(2, 8, 128256) >= 8 * 16
    for bad in ((7, 1, 1), (0, -1, 1), (0, 1, -1), (0, 1 << 40, 1), (0, 1, 1 << 31)):
        assert f(*bad) == -1


def _cache(slots=32, heads=2, dim=64, bits=8, parts=2):
    groups, tail = (1, ()) if bits == 8 else (2, (2,))
    codes = torch.zeros(parts, slots, heads, dim * bits // 8, dtype=torch.uint8)
    params = torch.zeros(parts, slots, heads, groups, *tail,
                         dtype=torch.float32 if bits == 8 else torch.bfloat16)
    return ops.QuantCache(OnGpu(codes), OnGpu(params), dim=dim, bits=bits)


def _gpu(*shape, dtype=torch.float32):
    return OnGpu(torch.zeros(*shape, dtype=dtype))


INT = torch.int32


@pytest.mark.parametrize("kw, error, match", [
    (dict(cache=_cache(parts=1)), ValueError, "two parts"),
    (dict(q=_gpu(2, 1, 4, 64, dtype=torch.float64)), TypeError, "q must be float32"),
    (dict(q=torch.zeros(2, 1, 4, 64)), ValueError, "q must be on"),
    (dict(q=_gpu(2, 1, 4, 32)), ValueError, "q must be"),
    (dict(q=_gpu(2, 64)), ValueError, "q must be"),
    (dict(q=_gpu(2, 1, 3, 64)), ValueError, "multiple"),
    (dict(blocks=_gpu(2, 3)), TypeError, "blocks must be int32"),
    (dict(blocks=torch.zeros(2, 3, dtype=INT)), ValueError, "blocks must be on"),
    (dict(blocks=_gpu(3, dtype=INT)), ValueError, "blocks must be"),
    (dict(blocks=_gpu(3, 3, dtype=INT)), ValueError, "blocks must have 2"),
    (dict(block_size=0), ValueError, "block_size"),
    (dict(lengths=_gpu(2)), TypeError, "lengths must be int32"),
    (dict(lengths=_gpu(3, dtype=INT)), ValueError, "lengths must be"),
    (dict(n_rows=_gpu(2, 1, dtype=INT)), ValueError, "n_rows must be"),
    (dict(window=0), ValueError, "window"),
    (dict(weights=_gpu(2, 2, 47)), ValueError, "weights must be"),
    (dict(weights=_gpu(2, 1, 48)), ValueError, "weights must be"),
    (dict(weights=_gpu(2, 2, 48, dtype=torch.float64)), TypeError, "weights must be"),
    (dict(weights=OnGpu(torch.zeros(2, 1, 48).expand(2, 2, 48))), ValueError, "expanded"),
    (dict(weights=OnGpu(torch.zeros(2, 48, 2).transpose(1, 2))), ValueError, "contiguous"),
    (dict(out=_gpu(2, 1, 4, 32)), ValueError, "out must be"),
    (dict(out=OnGpu(torch.zeros(2, 1, 1, 64).expand(2, 1, 4, 64))), ValueError, "out must be"),
])
def test_attend_binding_refusals(kw, error, match):
    a = dict(cache=_cache(), q=_gpu(2, 1, 4, 64), blocks=_gpu(2, 3, dtype=INT),
             lengths=_gpu(2, dtype=INT), out=_gpu(2, 1, 4, 64), block_size=16,
             workspace=_gpu(4096, dtype=torch.uint8))
    if "q" in kw:
        a["out"] = kw["q"]
    a.update(kw)
    with pytest.raises(error, match=match):
        ops.cache_attend(a.pop("cache"), a.pop("q"), a.pop("blocks"), a.pop("lengths"), **a)


@pytest.mark.parametrize("kw, error, match", [
    (dict(keep=-1), ValueError, "keep"), (dict(first=-1), ValueError, "first"),
    (dict(first=9, recent=9), ValueError, "keep"),
    (dict(weights=_gpu(2, 2, 40)), ValueError, "weights must be"),
    (dict(weights=_gpu(2, 2, 48, dtype=torch.bfloat16)), TypeError, "weights must be"),
    (dict(blocks=_gpu(2, 3)), TypeError, "blocks"),
    (dict(lengths=_gpu(1, dtype=INT)), ValueError, "lengths"),
    (dict(out=_gpu(2)), TypeError, "out must be int32"),
])
def test_evict_binding_refusals(kw, error, match):
    a = dict(weights=_gpu(2, 2, 48), blocks=_gpu(2, 3, dtype=INT), lengths=_gpu(2, dtype=INT),
             keep=16, first=0, recent=0, block_size=16, out=_gpu(2, dtype=INT))
    a.update(kw)
    with pytest.raises(error, match=match):
        ops.cache_evict(_cache(), a.pop("weights"), a.pop("blocks"), a.pop("lengths"),
                        a.pop("keep"), **a)


@pytest.mark.parametrize("kw, error, match", [
    (dict(drafts=_gpu(6, dtype=torch.int64)), ValueError, "drafts must be"),
    (dict(drafts=_gpu(2, 3, dtype=INT)), TypeError, "drafts must be int64"),
    (dict(logits=_gpu(2, 3, 40)), ValueError, "must match drafts"),
    (dict(logits=_gpu(7, 40)), ValueError, "must have 8 rows"),
    (dict(logits=_gpu(8, 40, dtype=torch.float64)), TypeError, "float32"),
    (dict(uniforms=_gpu(2, 3, dtype=torch.float64)), TypeError, "uniforms must be"),
    (dict(uniforms=_gpu(2, 4)), ValueError, "like drafts"),
    (dict(uniforms=torch.zeros(2, 3)), ValueError, "same device"),
    (dict(needs=_gpu(8, dtype=torch.uint8)), ValueError, "needs a bitmask"),
    (dict(probs=_gpu(2, 3, 39)), ValueError, "draft_probs must be"),
    (dict(probs=_gpu(2, 4, 40)), ValueError, "draft_probs must be"),
    (dict(probs=_gpu(2, 3, 40, dtype=torch.bfloat16)), TypeError, "draft_probs must be"),
    (dict(probs=OnGpu(torch.zeros(2, 40, 3).transpose(1, 2))), ValueError, "contiguous"),
    (dict(seeds=_gpu(2, dtype=torch.int64)), ValueError, "seeds must be"),
    (dict(temperature=torch.zeros(3)), ValueError, "temperature must have"),
    (dict(out=(_gpu(2, 4), _gpu(2, dtype=INT))), ValueError, "out must be"),
])
def test_verify_binding_refusals(kw, error, match):
    a = dict(logits=_gpu(8, 40), drafts=_gpu(2, 3, dtype=torch.int64), uniforms=_gpu(2, 3),
             probs=None, needs=None, seeds=None, temperature=1.0,
             out=(_gpu(2, 4, dtype=torch.int64), _gpu(2, dtype=INT)))
    a.update(kw)
    with pytest.raises(error, match=match):
        ops.verify_drafts(a["logits"], a["drafts"], a["uniforms"], draft_probs=a["probs"],
                          row_needs_mask=a["needs"], seeds=a["seeds"],
                          temperature=a["temperature"], out=a["out"])


def test_definitions_by_hand():
    # two tokens of equal score, one of them hidden from the first row
    kv = np.zeros((2, 4, 1, 2))
    kv[1, :, 0] = [[1, 0], [3, 0], [5, 0], [7, 0]]
    q = np.ones((1, 2, 1, 2))
    out, _, w, _ = attended(kv, q, np.array([[1, 0]], np.int32), [3], 2)
    # tokens in slots 2, 3, 0: row 0 sees two of them, row 1 three
    np.testing.assert_allclose(out[0, :, 0, 0], [6.0, 13 / 3])
    np.testing.assert_allclose(w[0, 0], [5 / 6, 5 / 6, 1 / 3, 0])
    assert evicted(6, np.array([9, 1, 3, 3, np.nan, 0], np.float32), 4, 1, 1).tolist() == [0, 2, 3, 5]
    assert evicted(4, np.ones(4, np.float32), 2, 0, 0).tolist() == [0, 1]
    assert evicted(4, np.full(4, np.nan, np.float32), 3, 0, 1).tolist() == [0, 1, 3]
    ok = np.ones((2, 2), bool)
    np.testing.assert_allclose(row_probs(np.array([0.0, np.log(3)]), ok[0], 1.0), [0.25, 0.75])
    x = np.array([[0.0, np.log(3)], [0.0, np.log(3)]])
    none = lambda n: np.zeros(2)  # noqa: E731
    got = verified(x, ok, [0], np.array([[0.5, 0.5]]), [0.4], 1.0, none)
    assert got[0].tolist() == [0, 1] and got[1] == 1       # 0.2 < 0.25
    got = verified(x, ok, [0], np.array([[0.5, 0.5]]), [0.6], 1.0, none)
    assert got[0].tolist() == [1, -1] and got[1] == 0      # what is left is on token 1
    got = verified(x, ok, [0], None, [0.2], 1.0, none)
    assert got[1] == 1
    got = verified(x, ok, [1], None, [0.8], 1.0, none)
    assert got[0].tolist() == [0, -1]                      # p without the draft


@pytest.mark.parametrize("index", [0, 1])
def test_launches_are_on_the_tensors_device(recorded, monkeypatch, index):
    """With another device current, a call is made with the tensors' device current, and that
    one is current again after it."""
    def gpu(*shape, dtype=torch.float32):
        return OnGpu(torch.zeros(*shape, dtype=dtype), index)

    for name in ("cache_attend", "cache_evict", "verify_drafts"):
        monkeypatch.setattr(ops, f"{name}_workspace_bytes", lambda *a: 8)
    cache = ops.QuantCache(gpu(2, 32, 2, 64, dtype=torch.uint8), gpu(2, 32, 2, 1), dim=64)
    ws = gpu(8, dtype=torch.uint8)
    table, lens = gpu(2, 2, dtype=INT), gpu(2, dtype=INT)
    weights = gpu(2, 2, 32)
    weights.__dict__["is_contiguous"] = lambda: True
    q = gpu(2, 1, 4, 64)
    ops.cache_attend(cache, q, table, lens, block_size=16, out=gpu(2, 1, 4, 64), workspace=ws,
                     weights=weights)
    ops.cache_evict(cache, weights, table, lens, 8, block_size=16, out=gpu(2, dtype=INT),
                    workspace=ws)
    ops.verify_drafts(gpu(8, 40), gpu(2, 3, dtype=torch.int64), gpu(2, 3), workspace=ws,
                      out=(gpu(2, 4, dtype=torch.int64), gpu(2, dtype=INT)))
    assert [name for name, _ in recorded.calls] == ["lp_cache_attend", "lp_cache_evict",
                                                    "lp_verify_drafts"]
    assert {device for _, device in recorded.calls} == {index}
    assert recorded.current == [0]
