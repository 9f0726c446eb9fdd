"""Arguments of the beam-search entry points that are refused on the host: nothing here
reaches a GPU.  Also pins of the plain definitions that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from beam_oracle import beam_candidates  # noqa: E402
from grammar_constrained_logit_gb300 import _lib, build, ops  # noqa: E402

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _beam(lib, **kw):
    a = dict(logits=FAKE, dt=2, batch=2, beams=4, cols=64, stride=64, bm=None, bm_rows=0, words=0,
             bm_stride=0, vocab=-1, needs=None, scores=FAKE, finished=None, pad=0, n=8, os=FAKE,
             ot=FAKE, op=FAKE, ws=FAKE, ws_bytes=1 << 20, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.lp_beam_select(*a.values())


MASK = dict(bm=FAKE, bm_rows=8, words=2, bm_stride=2)


@pytest.mark.parametrize("kw, want", [
    (dict(dt=3), 2), (dict(dt=-1), 2),
    (dict(batch=-1), 1), (dict(beams=0), 1), (dict(beams=-2), 1), (dict(cols=-1), 1),
    (dict(stride=63), 1), (dict(n=-1), 1), (dict(vocab=65), 1),
    (dict(logits=None), 1), (dict(scores=None), 1), (dict(os=None), 1), (dict(ot=None), 1),
    (dict(op=None), 1), (dict(ws=None), 1), (dict(ws_bytes=63), 1),
    (dict(ws=ctypes.c_void_p(0x10004)), 1), (dict(logits=ctypes.c_void_p(0x10001)), 1),
    (dict(stride=1 << 60), 1),
    (dict(needs=FAKE), 1),  # flags without a bitmask
    (dict(MASK, bm_rows=7), 1), (dict(MASK, words=-1), 1), (dict(MASK, bm_stride=1), 1),
    (dict(MASK, vocab=64, words=1), 1), (dict(MASK, words=1 << 60, bm_stride=1 << 60), 1),
    (dict(beams=257), 4), (dict(n=257), 4), (dict(batch=1 << 27), 4),
    (dict(cols=1 << 31, stride=1 << 31), 4),
    (dict(batch=1 << 20, cols=1 << 22, stride=1 << 22, ws_bytes=1 << 62), 4),
    (dict(batch=0), 0), (dict(n=0), 0),  # nothing to do
])
def test_beam_select_refusals(lib, kw, want):
    assert _beam(lib, **kw) == want


def test_beam_workspace_bytes(lib):
    f = lib.lp_beam_select_workspace_bytes
    # 8 bytes for each 256 16-bit or 128 f32 tokens of a row
    assert f(2, 8, 1024) == 256 and f(2, 8, 1025) == 320 and f(0, 8, 1024) == 512
    assert f(1, 0, 5) == 0 and f(1, 3, 0) == 24
    assert f(7, 1, 1) == -1 and f(0, -1, 1) == -1 and f(0, 1, -1) == -1
    assert f(0, 1 << 60, 1 << 40) == -1


def test_binding_refusals():
    lg, sc = torch.zeros(8, 64), torch.zeros(2, 4)
    with pytest.raises(ValueError, match="CUDA"):
        ops.beam_select(lg, sc)
    with pytest.raises(ValueError, match="batch, beams"):
        ops.beam_select(lg, sc.view(-1))
    with pytest.raises(TypeError, match="float32"):
        ops.beam_select(lg, sc.double())
    with pytest.raises(ValueError, match="must match scores"):
        ops.beam_select(torch.zeros(2, 3, 64), sc)


def test_candidates_by_hand():
    x = np.array([[0.0, 0.0, -np.inf], [np.log(3.0), 0.0, np.nan]])
    got = beam_candidates(x, np.array([-1.0, -1.0]))
    # beam 1: 3/4 and 1/4; beam 0: a half each, its two tokens tied in order
    assert [(k, t) for _, k, t in got] == [(1, 0), (0, 0), (0, 1), (1, 1)]
    np.testing.assert_allclose([s for s, _, _ in got],
                               -1 + np.log([0.75, 0.5, 0.5, 0.25]), rtol=1e-15)
    got = beam_candidates(x, np.array([-1.0, -0.5]), finished=[False, True], pad=7,
                          allowed=np.array([[False, True, True]] * 2))
    assert got == [(-0.5, 1, 7), (-1.0, 0, 1)]
    assert beam_candidates(x, np.array([-np.inf, np.nan])) == []
    got = beam_candidates(np.array([[np.inf, 3.0, np.inf]]), np.array([0.0]))
    assert [(k, t) for _, k, t in got] == [(0, 0), (0, 2)] and got[0][0] == -np.log(2.0)


# ---------------------------------------------------------------- reorder_states


def _state(**kw):
    s = _lib.State()
    s.data, s.row_stride, s.run_bytes, s.token_bytes = 0x10000, 64, 64, 0
    for d in range(3):
        s.outer[d], s.outer_stride[d] = 1, 0
    for k, v in kw.items():
        if k == "outer":
            for d in range(3):
                s.outer[d] = v[d]
        else:
            setattr(s, k, v)
    return s


def _reorder(lib, *states, n=None, batch=2, beams=4, parents=FAKE, start=None, stop=None):
    arr = (_lib.State * max(1, len(states)))(*states)
    return lib.lp_reorder_states(arr if states else None, len(states) if n is None else n, batch,
                                 beams, parents, start, stop, None)


@pytest.mark.parametrize("kw, args, want", [
    (dict(run_bytes=-1), {}, 1), (dict(token_bytes=-2), {}, 1), (dict(token_bytes=5), {}, 1),
    (dict(outer=(1, -1, 1)), {}, 1), (dict(data=None), {}, 1), (dict(row_stride=63), {}, 1),
    (dict(row_stride=0), {}, 1), (dict(row_stride=-63), {}, 1),
    ({}, dict(batch=-1), 1), ({}, dict(beams=0), 1), ({}, dict(parents=None), 1),
    ({}, dict(n=-1), 1),
    ({}, dict(beams=257), 4), ({}, dict(batch=1 << 26), 4),
    (dict(outer=(1 << 32, 1, 1)), {}, 4), (dict(outer=(1 << 20, 1 << 20, 1)), {}, 4),
    (dict(run_bytes=1 << 50, row_stride=1 << 50), {}, 4),
    ({}, dict(batch=0), 0), (dict(run_bytes=0), {}, 0), (dict(outer=(0, 1, 1), data=None), {}, 0),
])
def test_reorder_refusals(lib, kw, args, want):
    assert _reorder(lib, _state(**kw), **args) == want


def test_reorder_nothing(lib):
    assert _reorder(lib) == 0
    assert _reorder(lib, n=1) == 1  # a count without states


def test_state_reorder_binding_refusals():
    with pytest.raises(ValueError, match="CUDA"):
        ops.StateReorder([torch.zeros(8, 4)], 2, 4)
    with pytest.raises(ValueError, match="beams"):
        ops.StateReorder([], 2, 0)
    with pytest.raises(ValueError, match="batch, beams"):
        ops.reorder_states([], torch.zeros(4, dtype=torch.int32))
    ops.StateReorder([], 2, 4).reorder(torch.zeros(2, 4, dtype=torch.int32))  # nothing to move


class _Fake:
    """A CUDA tensor's geometry without one."""

    def __init__(self, t):
        self.t, self.is_cuda = t, True

    def __getattr__(self, name):
        return getattr(self.t, name)


def _geometry(t, rows, tokens):
    s = ops._state(_Fake(t), rows, tokens)
    return (s.row_stride, s.run_bytes, s.token_bytes, tuple(s.outer), tuple(s.outer_stride))


def test_state_geometry():
    """The bytes that a descriptor names, walked on the CPU, are the tensor's own."""
    base = torch.arange(2 * 6 * 5 * 3 * 4, dtype=torch.int16).view(2, 6, 5, 3, 4)
    views = [(base, 1, 2), (base, 1, 3), (base, 1, None), (base.transpose(2, 3), 1, 3),
             (base[:, :, 1:4], 1, 2), (base[0], 0, 1), (base[..., 1:3], 1, 2), (base[:, :, :1], 1, 2),
             (base.permute(4, 1, 0, 3, 2), 1, 4), (base[1, :, 2], 0, None), (base[0, :, :, 0], 0, 1),
             (base[0, :, 0, 0, 0], 0, None), (base[:, :, :, :1], 1, 3), (base[:, :, ::2], 1, 2)]
    flat = base.reshape(-1)
    for t, rows, tokens in views:
        row_stride, run, token, outer, strides = _geometry(t, rows, tokens)
        for r in range(t.size(rows)):
            want = t.select(rows, r)
            places = []
            for i in range(outer[0]):
                for j in range(outer[1]):
                    for k in range(outer[2]):
                        at = t.storage_offset() * 2 + r * row_stride + i * strides[0] + \
                            j * strides[1] + k * strides[2]
                        assert at % 2 == 0
                        places += range(at // 2, (at + run) // 2)
            assert sorted(flat[places].tolist()) == sorted(want.reshape(-1).tolist())
        if tokens is not None:
            T = t.size(tokens)
            assert token == -1 and outer[0] == T or run // token == T
    with pytest.raises(ValueError, match="expanded"):
        _geometry(torch.zeros(1, 4).expand(3, 4), 0, None)
    with pytest.raises(ValueError, match="rows'"):
        _geometry(base, 1, 1)
    with pytest.raises(ValueError, match="out of range"):
        _geometry(base, 5, None)
    with pytest.raises(ValueError, match="three"):
        _geometry(torch.zeros(4, 3, 6, 3, 6, 3, 6, 3)[:, :2, :5, :2, :5, :2, :5, :2], 0, None)


# ------------------------------------------------------------------------- cache


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("kw, want", [
    (dict(dt=3), 2), (dict(bits=5), 1), (dict(bits=16), 1), (dict(n_parts=-1), 1),
    (dict(n_parts=9), 1), (dict(n_slots=-1), 1), (dict(page=0), 1), (dict(heads=-1), 1),
    (dict(dim=-1), 1), (dict(group=0), 1), (dict(group=48), 1), (dict(bits=4, dim=9, group=9), 1),
    (dict(n=-1), 1), (dict(parts=None), 1), (dict(x=None), 1), (dict(slots=None), 1),
    (dict(part=dict(codes=None)), 1), (dict(part=dict(params=None)), 1),
    (dict(part=dict(params=0x10002)), 1), (dict(part=dict(param_slot_stride=6)), 1),
    (dict(x_data=None), 1), (dict(x_data=0x10001), 1),
    (dict(dim=1 << 40, group=1), 4), (dict(heads=1 << 40), 4),
    (dict(heads=1 << 30, dim=1 << 30, group=1, n=1 << 10), 4),
    (dict(n=0), 0), (dict(heads=0), 0), (dict(dim=0), 0), (dict(n_parts=0), 0)])
def test_cache_refusals(lib, write, kw, want):
    kw = dict(kw)
    part = kw.pop("part", None)
    a = dict(data=kw.pop("x_data")) if "x_data" in kw else None
    p, h = _lib.CachePart(), _lib.Heads()
    p.codes = p.params = h.data = 0x10000
    for k, v in (part or {}).items():
        setattr(p, k, v)
    for k, v in (a or {}).items():
        setattr(h, k, v)
    args = dict(parts=ctypes.byref(p), x=ctypes.byref(h), n_parts=1, bits=8, dt=2, n_slots=16,
                page=16, heads=2, dim=64, group=32, slots=FAKE, n=4, stream=None)
    assert set(kw) <= set(args)
    args.update(kw)
    assert (lib.lp_cache_write if write else lib.lp_cache_read)(*args.values()) == want


def test_cache_binding_refusals():
    codes, params = torch.zeros(2, 4, 2, 64, dtype=torch.uint8), torch.zeros(2, 4, 2, 1)
    with pytest.raises(ValueError, match="CUDA"):
        ops.QuantCache(codes, params, dim=64)
    with pytest.raises(ValueError, match="bits"):
        ops.QuantCache(codes, params, dim=64, bits=2)
    with pytest.raises(TypeError, match="uint8"):
        ops.QuantCache(codes.char(), params, dim=64)
    with pytest.raises(TypeError, match="bfloat16"):
        ops.QuantCache(codes, params, dim=128, bits=4)
    for kw in (dict(group=5), dict(bits=3), dict(bits=4, group=0)):
        with pytest.raises(ValueError):
            ops.QuantCache.allocate(4, 2, 64, device="cpu", **kw)


def test_quantised_by_hand():
    from beam_oracle import e4m3_values, held_values, quantised

    v = e4m3_values()
    assert v[0x7e] == 448 and v[1] == 2.0 ** -9 and v[0x38] == 1 and v[0xb8] == -1
    x = np.array([448.0, -1.0, 17.0, 19.0, 0.0, 2.0 ** -10, np.inf, np.nan], np.float32)
    code, scale, low = quantised(x, 8, 8)
    assert scale.tolist() == [1.0]
    # 17 and 19 lie half-way between neighbours: to the even ones; 2^-10 is half a step
    assert code[0, :7].tolist() == [448, -1, 16, 20, 0, 0, 448] and np.isnan(code[0, 7])
    x = np.array([-1.0, 14.0, 0.5, 1.5, -np.inf, np.nan], np.float32)
    code, scale, low = quantised(x, 4, 6)
    assert scale.tolist() == [1.0] and low.tolist() == [-1.0]
    assert code[0].tolist() == [0, 15, 2, 2, 0, 0]
    assert held_values(code, scale, low, 4).tolist() == [-1, 14, 1, 1, -1, -1]
