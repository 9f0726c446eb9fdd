"""Verification of drafts at the ends of the temperature's range."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from grammar_constrained_logit_gb300 import ops  # noqa: E402
from test_gpu_verify import check, make  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from grammar_constrained_logit_gb300 import _lib

    _lib.load()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V, keep", [(40, None), (40, 0.5), (4003, 0.3), (70001, None)])
def test_infinite_temperature(dtype, V, keep):
    """All candidates are equally likely: a draft is accepted where u q < 1 / candidates."""
    rng = np.random.default_rng(V)
    slots, rows = 24, 4
    temps = np.full(slots, 1.0, np.float32)
    x, allowed, temps, q, drafts, u = make(rng, slots, rows, V, V, dtype, keep=keep, temps=temps)
    temps[:] = np.inf
    temps[::5] = 0.7
    # near acceptance, on either side: u q from 0 to twice 1 / candidates
    n = allowed[:, :-1].sum(-1)
    at = np.take_along_axis(q, drafts[..., None], 2)[..., 0]
    even = rng.random((slots, rows - 1))
    tokens, accepted = check(x, allowed, temps, q, drafts,
                             np.minimum(even * 2 / (n * at), 0.999).astype(np.float32),
                             masked=keep is not None)
    hot = np.isinf(temps)
    assert 0 < accepted[hot].sum() < hot.sum() * (rows - 1)
    _, accepted = check(x, allowed, temps, None, drafts, (even * 2 / n).astype(np.float32),
                        masked=keep is not None)
    assert 0 < accepted[hot].sum() < hot.sum() * (rows - 1)


@pytest.mark.parametrize("heat", [float("inf"), 1e38, 1e-38, 1e-45])
def test_one_temperature_for_all(heat):
    """As a number, and as a tensor; drafts that are sure are accepted whatever it is."""
    rng = np.random.default_rng(9)
    x, _, _, _, drafts, u = make(rng, 6, 3, 900, 900, "f32", probs=False)
    drafts[:] = x[:, :-1].numpy().argmax(-1)
    u[:] = 0.0
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    args = (x.cuda(), dev(drafts), dev(u))
    tokens, accepted = ops.verify_drafts(*args, temperature=heat, seed=4)
    assert (accepted == 2).all() and (tokens[:, 2] >= 0).all()
    more = ops.verify_drafts(*args, temperature=torch.tensor([heat], device="cuda"), seed=4)
    assert torch.equal(tokens, more[0]) and torch.equal(accepted, more[1])
    plain = ops.sample(x.cuda().view(18, 900), temperature=heat, seed=4).view(6, 3)
    if heat > 1e-30:
        assert torch.equal(tokens[:, 2], plain[:, 2])
