"""How exact attention over the quantised cache is, over a whole call: the norm of what it is off
by, against 64 bits.

An element's bound has to allow for the largest error that arithmetic admits; the norm over
thousands of elements does not, so fewer bits than are claimed show in it.  Independent errors
add in squares:

  * the result's rounding: what rounding the 64-bit result to its type leaves, which depends on
    where in their binades the values lie.  The kernel rounds values that are a little off, so
    its N roundings are others of the same spread; the root of the mean square of N errors that
    are even over a step spreads by 0.45 / sqrt(N) of itself, below 0.8% for the 4096 elements
    and more here: 5% is allowed;
  * a weight's rounding where it meets its value, w = 2^-11 (bf16) or 2^-22: with values of
    either sign, w / sqrt(6) of the output, in 4 bits of the codes' part, twice that and less.
    w is allowed;
  * sums on tensor cores.  A product of 16 cuts its 17 addends at 2^-24 of the largest, to zero:
    e = sqrt(17 / 3) 2^-24 of it at the root of the mean square.  A score has dim / 16 such steps
    in two pieces, at most 32, and partial sums of up to 4 times its deviation, which is 1 here:
    sqrt(32) * 4 e = 3.2e-6, which is what a weight is off by, relatively.  What is added up over
    tokens is cut within 16 of them, sqrt(2) * 1.5 e, and rounded from there on: n / 16 sums, the
    root of the mean square of whose roundings is 2^-24 / sqrt(3) of them, that grow as the root
    of what they are made of: sqrt(n / 32) * 2^-24 / sqrt(3), 1.2e-6 for 40000.  In squares
    3.5e-6; 4e-6 is allowed.

What is cut is lost toward zero, so it also shows as a part of the result itself, <got, want> over
<want, want> less 1, where N roundings average out to 1 / sqrt(N) of them.  The sums of 16 tokens leave no more than the
rest does.  The kernel of many rows (8 bits with one scale a head, 16-bit queries) goes on for 8192
tokens, 512 products or 1024 in two pieces, each of which takes half a unit of 2^-23 of the sum's
binade, 0.7 * 2^-24 of the sum, and half of that over its growth: 2.1e-5.

A weight that is added up is rounded to 32 bits, so the last is its bound for all types."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from attend_oracle import WEIGHT, held  # noqa: E402
from grammar_constrained_logit_gb300 import ops  # noqa: E402
from test_gpu_attend import TYPES, filled, table  # noqa: E402

pytestmark = pytest.mark.gpu

SUMS = 4e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from grammar_constrained_logit_gb300 import _lib

    _lib.load()


def even(total, heads, dim, bits, group):
    """A cache of keys and values that are even about zero, of deviation 1."""
    cache = filled(total, heads, dim, bits, group, page=16)
    g = torch.Generator("cuda").manual_seed(dim + bits)
    x = [torch.randn(total, heads, dim, device="cuda", generator=g) for _ in range(2)]
    ops.cache_write(cache, x, torch.arange(total, device="cuda"))
    return cache


def exactly(cache, q, blocks, lengths, size, window=None):
    """(out, weights) in 64 bits."""
    kv = torch.from_numpy(held(cache)).cuda()
    batch, rows, q_heads, dim = q.shape
    shared = q_heads // cache.heads
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    weights = torch.zeros(batch, cache.heads, blocks.shape[1] * size, dtype=torch.float64,
                          device="cuda")
    for b, n in enumerate(lengths):
        t = np.arange(n)
        at = torch.from_numpy(blocks[b].astype(np.int64)[t // size] * size + t % size).cuda()
        k, v = (p[at].repeat_interleave(shared, 1) for p in kv)
        x = torch.einsum("rhd,thd->hrt", q[b].double(), k) / math.sqrt(dim)
        end = n - (rows - 1) + torch.arange(rows, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")
        hidden = (t >= end) if window is None else (t >= end) | (t < end - window)
        p = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
        out[b] = torch.einsum("hrt,thd->rhd", p, v)
        weights[b, :, :n] = p.view(cache.heads, shared * rows, n).sum(1)
    return out, weights


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def close(cache, q, blocks, lengths, size, dtype, window=None):
    q = q.to(TYPES[dtype])
    w = torch.zeros(q.size(0), cache.heads, blocks.shape[1] * size, device="cuda")
    got = ops.cache_attend(cache, q, torch.from_numpy(blocks).cuda(),
                           torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                           block_size=size, window=window, weights=w)
    want, weights = exactly(cache, q, blocks, lengths, size, window)
    rounding = 1.05 * off(want.to(q.dtype), want)
    bound = math.sqrt(rounding ** 2 + WEIGHT[dtype] ** 2 + SUMS ** 2)
    assert off(got, want) < bound, (off(got, want), bound)
    assert off(w, weights) < SUMS, off(w, weights)
    along = float((got.double() * want).sum() / (want * want).sum()) - 1
    return along, rounding / math.sqrt(want.numel())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bits, dim, group", [
    (8, 128, 128), (8, 128, 32), (8, 64, 64), (8, 80, 16), (8, 256, 128), (8, 72, 72),
    (4, 128, 32), (4, 128, 16), (4, 128, 128), (4, 64, 32), (4, 80, 16), (4, 96, 96),
    (4, 192, 64), (4, 256, 32), (4, 112, 16)])
def test_norm(bits, dim, group, dtype):
    """A token a sequence with four queries a head, and drafts with a window."""
    rng = np.random.default_rng(dim + group)
    lengths = [700, 33, 257, 640]
    total = (sum(-(-n // 16) for n in lengths) + 1) * 16
    cache = even(total, 4, dim, bits, group)
    blocks = table(rng, lengths, 16, total)
    g = torch.Generator("cuda").manual_seed(dim)
    for rows, window in ((1, None), (5, None), (3, 127)):
        q = torch.randn(4, rows, 16, dim, device="cuda", generator=g)
        close(cache, q, blocks, lengths, 16, dtype, window)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bits, dim, group", [(8, 128, 128), (8, 64, 64), (8, 128, 32),
                                              (4, 128, 32), (4, 128, 128)])
@pytest.mark.parametrize("window", [None, 300])
def test_norm_of_many_rows(bits, dim, group, dtype, window):
    """As many queries as the tensor-memory kernels take."""
    rng = np.random.default_rng(31)
    lengths = [500, 130, 700, 256, 300]
    total = (sum(-(-n // 16) for n in lengths) + 1) * 16
    cache = even(total, 8, dim, bits, group)
    g = torch.Generator("cuda").manual_seed(32)
    q = torch.randn(5, 97, 24, dim, device="cuda", generator=g)
    close(cache, q, table(rng, lengths, 16, total), lengths, 16, dtype, window)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("bits, dim, group", [(8, 128, 32), (4, 128, 32), (4, 64, 16),
                                              (8, 128, 128), (8, 64, 64)])
def test_norm_over_many_tokens(bits, dim, group, dtype):
    """So many rows that a worker or block goes through hundreds of tiles of tokens."""
    lengths = [40000]
    total = 40016
    cache = even(total, 4, dim, bits, group)
    g = torch.Generator("cuda").manual_seed(33)
    q = torch.randn(1, 500, 16, dim, device="cuda", generator=g)
    along, spread = close(cache, q, table(np.random.default_rng(34), lengths, 16, total), lengths,
                          16, dtype)
    cut = SUMS if dtype == "f32" or bits == 4 or group < dim else 2.1e-5
    assert abs(along) < cut + 4 * spread, (along, spread)
