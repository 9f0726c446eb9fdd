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
    assert f(2, 8, 1024) == 64 and f(2, 8, 1025) == 128 and f(0, 8, 1024) == 128
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
