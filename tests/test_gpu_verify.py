"""Verification of drafts against its definition in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from attend_oracle import row_probs, verified  # noqa: E402
from grammar_constrained_logit_gb300 import ops  # noqa: E402
from grammar_constrained_logit_gb300 import synthetic as syn  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from grammar_constrained_logit_gb300 import _lib

    _lib.load()


def gumbel(seed, row, offset, V):
    """The sampler's noise of one row, float64."""
    n = (V + 3) // 4
    c = torch.zeros(n, 4, dtype=torch.int64)
    c[:, 0] = torch.arange(n)
    c[:, 1], c[:, 2], c[:, 3] = row, offset & 0xffffffff, offset >> 32
    k = torch.tensor([[seed & 0xffffffff, (seed >> 32) & 0xffffffff]]).expand(n, 2)
    as32 = lambda t: torch.where(t >= 1 << 31, t - (1 << 32), t).to(torch.int32)  # noqa: E731
    w = ops.philox4x32_10(as32(c).cuda(), as32(k.contiguous()).cuda()).cpu().numpy()
    u = ((w.view(np.uint32).reshape(-1)[:V] >> 9).astype(np.float64) + 0.5) * 2.0 ** -23
    return -np.log(-np.log(u))


def make(rng, slots, rows, V, cols, dtype, *, probs=True, keep=None, temps=None, far=0.7):
    x = torch.from_numpy((rng.standard_normal((slots, rows, cols)) * 3).astype(np.float32))
    x = x.to(TYPES[dtype])
    allowed = np.ones((slots, rows, V), bool) if keep is None else \
        rng.random((slots, rows, V)) < keep
    temps = np.full(slots, 0.9, np.float32) if temps is None else temps
    near = x[:, :-1, :V].double().numpy() + far * rng.standard_normal((slots, rows - 1, V))
    near = np.where(allowed[:, :-1], near, -np.inf) / np.maximum(temps, 0.1)[:, None, None]
    near = np.exp(near - np.maximum(near.max(-1, keepdims=True), -1e30))
    near /= np.maximum(near.sum(-1, keepdims=True), 1e-300)
    q = near.astype(np.float32)
    drafts = np.zeros((slots, rows - 1), np.int64)
    for s in range(slots):
        for i in range(rows - 1):
            if near[s, i].sum() > 0:
                drafts[s, i] = rng.choice(V, p=near[s, i] / near[s, i].sum())
    u = rng.random((slots, rows - 1)).astype(np.float32)
    return x, allowed, temps, q if probs else None, drafts, u


def check(x, allowed, temps, q, drafts, u, *, needs=None, seed=5, offset=3, seeds=None, V=None,
          masked=True):
    """Every slot is as defined, unless one of its decisions hung on less than the rounding: of
    a probability 2e-5 at most (T >= 0.3: the largest |x - top| / T, below 100, times 2^-23,
    and the sum's error), of a score the same."""
    slots, rows, cols = x.shape
    V = cols if V is None else V
    mask = flags = None
    if masked:
        mask = torch.from_numpy(syn.pack_bits(allowed.reshape(slots * rows, V))).cuda()
        if needs is not None:
            flags = torch.from_numpy(needs.astype(np.uint8)).cuda()
            allowed = allowed | (needs == 0).reshape(slots, rows, 1)
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    tokens, accepted = ops.verify_drafts(
        x.cuda(), dev(drafts), dev(u), draft_probs=dev(q), bitmask=mask, row_needs_mask=flags,
        temperature=dev(temps), seed=seed, offset=offset, seeds=dev(seeds), vocab_size=V)
    assert tokens.dtype == torch.int64 and accepted.dtype == torch.int32
    tokens, accepted = tokens.cpu().numpy(), accepted.cpu().numpy()
    xs = x[:, :, :V].double().numpy()
    close = 0
    for s in range(slots):
        def noise(n):
            row = s * rows + n
            return gumbel(seed if seeds is None else int(seeds[row]), row, offset, V)

        want, n, margin = verified(xs[s], allowed[s], drafts[s], None if q is None else q[s],
                                   u[s], float(temps[s]), noise)
        if margin < 2e-5:
            close += 1
        else:
            assert accepted[s] == n, (s, accepted[s], n, margin)
            assert np.array_equal(tokens[s], want), (s, tokens[s], want, margin)
        n = accepted[s]
        assert np.array_equal(tokens[s, :n], drafts[s, :n]) and (tokens[s, n + 1:] == -1).all()
        assert tokens[s, n] == -1 or allowed[s, n, tokens[s, n]]
    assert close <= 1 + slots // 50
    return tokens, accepted


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("slots, rows, V, cols, keep", [
    (1, 4, 32000, 32000, None), (9, 5, 1003, 1003, None), (5, 3, 4097, 4101, 0.3),
    (16, 2, 50, 64, 0.5), (3, 9, 20011, 20011, 0.02), (2, 33, 700, 700, None),
    (4, 1, 5000, 5008, 0.5), (7, 4, 1, 1, None), (2, 2, 150001, 150016, 0.1)])
def test_shapes(dtype, probs, slots, rows, V, cols, keep):
    rng = np.random.default_rng(V + rows)
    made = make(rng, slots, rows, V, cols, dtype, probs=probs, keep=keep,
                temps=rng.uniform(0.5, 1.5, slots).astype(np.float32))
    needs = (rng.random(slots * rows) < 0.7) if keep else None
    check(*made, needs=needs, V=V, masked=keep is not None,
          seeds=rng.integers(-2 ** 63, 2 ** 63 - 1, slots * rows) if V % 2 else None,
          offset=2 ** 40 + 5)


def test_greedy_and_mixed():
    rng = np.random.default_rng(1)
    temps = np.array([0.0, 1.0, -2.0, np.nan, 0.3, 0.0], np.float32)
    x, allowed, temps, q, drafts, u = make(rng, 6, 4, 3001, 3001, "bf16", keep=0.4, temps=temps)
    best = np.where(allowed, x.double().numpy()[..., :3001], -np.inf).argmax(-1)
    drafts[0] = best[0, :3]          # all right
    drafts[5] = best[5, :3]
    drafts[5, 1] = (drafts[5, 1] + 1) % 3001
    for probs in (q, None):
        tokens, accepted = check(x, allowed, temps, probs, drafts, u)
        assert accepted[5] == 1 and tokens[5, 1] == best[5, 1]
        if probs is None:
            assert accepted[0] == 3 and tokens[0].tolist() == best[0].tolist()


def test_drafts_that_are_not_there():
    rng = np.random.default_rng(2)
    x, allowed, temps, q, drafts, u = make(rng, 8, 4, 999, 999, "f32")
    u[:] = 0.0  # what is there is accepted
    drafts[0, 0] = -1
    drafts[1, 1] = 999
    drafts[2, 2] = 2 ** 40
    drafts[3] = -1
    drafts[4, 0] = -(2 ** 62)
    _, accepted = check(x, allowed, temps, q, drafts, u, masked=False)
    assert accepted.tolist() == [0, 1, 2, 0, 0, 3, 3, 3]


def test_rows_without_a_candidate():
    """A mask that admits nothing refuses the draft and says -1; so do logits of -inf and NaN."""
    rng = np.random.default_rng(3)
    x, allowed, temps, q, drafts, u = make(rng, 5, 3, 500, 500, "f32", keep=0.5)
    u[:] = 0.0
    allowed[0, 1] = False
    allowed[1, 0] = False
    x[2, 1] = float("-inf")
    x[3, 2] = float("nan")
    allowed[4, 2] = False
    tokens, accepted = check(x, allowed, temps, q, drafts, u)
    assert accepted[:5].tolist()[0] == 1 and tokens[0].tolist() == [drafts[0, 0], -1, -1]
    assert tokens[1].tolist() == [-1, -1, -1] and accepted[1] == 0
    assert tokens[2, 1] == -1 and tokens[3, accepted[3]] == -1 or accepted[3] < 2


def test_infinities_and_nan():
    rng = np.random.default_rng(4)
    x, allowed, temps, q, drafts, u = make(rng, 4, 3, 300, 300, "f32", probs=False)
    x[0, 0, [5, 9]] = float("inf")   # share the mass: 1/2 each
    drafts[0, 0], u[0, 0] = 9, 0.49
    x[1, 0, 7] = float("nan")        # no candidate
    drafts[1, 0], u[1, 0] = 7, 0.0
    x[2, 0, :] = float("-inf")
    x[2, 0, 3] = 1.0                 # the only one
    drafts[2, 0], u[2, 0] = 3, 0.999
    u[3, 0] = float("nan")           # accepts nothing
    tokens, accepted = check(x, allowed, temps, None, drafts, u, masked=False)
    assert accepted[0] >= 1 and accepted[1] == 0 and accepted[2] >= 1 and accepted[3] == 0


def test_nothing_left():
    """The draft's probabilities above the target's everywhere: p draws after all."""
    rng = np.random.default_rng(5)
    x, allowed, temps, q, drafts, u = make(rng, 3, 2, 400, 400, "f32", far=0.0)
    q[:] = 1.0
    u[:] = 0.999999
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    tokens, accepted = ops.verify_drafts(x.cuda(), dev(drafts), dev(u), draft_probs=dev(q),
                                         temperature=dev(temps), seed=8)
    assert (accepted == 0).all()
    plain = ops.sample(x.cuda().view(6, 400), temperature=dev(np.repeat(temps, 2)), seed=8)
    assert torch.equal(tokens[:, 0], plain.view(3, 2)[:, 0])
    q[:] = float("nan")
    u[:] = 0.5
    tokens, accepted = ops.verify_drafts(x.cuda(), dev(drafts), dev(u), draft_probs=dev(q),
                                         temperature=dev(temps), seed=8)
    assert (accepted == 0).all() and torch.equal(tokens[:, 0], plain.view(3, 2)[:, 0])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows_that_all_accept_say_what_the_sampler_says(dtype):
    """The row after the accepted drafts draws as mask_and_sample_slots does."""
    rng = np.random.default_rng(6)
    slots, rows, V = 12, 4, 9001
    x, allowed, temps, q, drafts, u = make(rng, slots, rows, V, V, dtype, keep=0.2,
                                           temps=rng.uniform(0.4, 1.3, 12).astype(np.float32))
    u[:] = 0.0
    drafts[::3, 1:] = -1
    mask = torch.from_numpy(syn.pack_bits(allowed.reshape(-1, V))).cuda()
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    seeds = torch.randint(-2 ** 62, 2 ** 62, (slots * rows,), device="cuda")
    tokens, accepted = ops.verify_drafts(x.cuda(), dev(drafts), dev(u), draft_probs=dev(q),
                                         bitmask=mask, temperature=dev(temps), seeds=seeds,
                                         offset=11)
    ids = ops.mask_and_sample_slots(x.cuda(), mask, rows, temperature=dev(temps), seeds=seeds,
                                    offset=11).view(slots, rows)
    n = accepted.long()[:, None]
    assert n.view(-1).tolist() == [1 if s % 3 == 0 else 3 for s in range(slots)]
    assert torch.equal(tokens.gather(1, n), ids.gather(1, n))
    one, zero = ops.verify_drafts(x.cuda()[:, :1], dev(drafts[:, :0].copy()),
                                  dev(u[:, :0].copy()), temperature=dev(temps), seed=4)
    assert (zero == 0).all()
    assert torch.equal(one.view(-1), ops.sample(x.cuda()[:, 0].contiguous(), dev(temps), seed=4))


def test_what_is_said_follows_the_target():
    """Over many seeds, what a slot says first is distributed as p, whatever the draft: a
    chi-squared statistic of 7 degrees of freedom stays below 24.3 (one in a thousand)."""
    rng = np.random.default_rng(7)
    V, slots = 8, 20000
    logits = rng.standard_normal(V).astype(np.float32)
    p = row_probs(logits.astype(np.float64), np.ones(V, bool), 1.0)
    x = torch.from_numpy(logits).cuda().expand(slots, 2, V).contiguous()
    other = rng.dirichlet(np.ones(V))
    for q in (other, None):
        drafts = rng.choice(V, size=(slots, 1), p=other) if q is not None else \
            np.full((slots, 1), 2)
        u = torch.rand(slots, 1, device="cuda")
        probs = None if q is None else torch.tensor(q, device="cuda", dtype=torch.float32)
        tokens, _ = ops.verify_drafts(
            x, torch.from_numpy(drafts).cuda(), u, seed=123,
            draft_probs=None if q is None else probs.expand(slots, 1, V))
        seen = np.bincount(tokens[:, 0].cpu().numpy(), minlength=V)
        assert ((seen - slots * p) ** 2 / (slots * p)).sum() < 24.3


def test_strides_and_out():
    rng = np.random.default_rng(8)
    x, allowed, temps, q, drafts, u = make(rng, 3, 4, 777, 777, "bf16", keep=0.5)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    mask = torch.from_numpy(syn.pack_bits(allowed.reshape(-1, 777))).cuda()
    want = ops.verify_drafts(x.cuda(), dev(drafts), dev(u), draft_probs=dev(q), bitmask=mask,
                             temperature=dev(temps), seed=3)
    wide = torch.full((12, 801), 50.0, device="cuda", dtype=torch.bfloat16)
    wide[:, 3:780] = x.cuda().view(12, 777)
    room = torch.full((3, 5, 800), 1.0, device="cuda")
    room[:, 1:4, 5:782] = dev(q)
    out = (torch.full((3, 4), 9, dtype=torch.int64, device="cuda"),
           torch.full((3,), 9, dtype=torch.int32, device="cuda"))
    got = ops.verify_drafts(wide[:, 3:780], dev(drafts), dev(u), draft_probs=room[:, 1:4, 5:782],
                            bitmask=mask, temperature=dev(temps), seed=3, out=out)
    assert got is out and all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.empty(ops.verify_drafts_workspace_bytes(torch.bfloat16, 12, 777),
                     dtype=torch.uint8, device="cuda").fill_(0xff)
    again = ops.verify_drafts(x.cuda(), dev(drafts), dev(u), draft_probs=dev(q), bitmask=mask,
                              temperature=dev(temps), seed=3, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(again, want))
