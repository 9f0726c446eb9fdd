"""The example's whole search on the package's operators against the same search on their
plain definitions."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from beam_oracle import beam_candidates, held_values, quantised, reordered  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(ROOT, "examples", "constrained_beam_search.py")
    spec = importlib.util.spec_from_file_location("constrained_beam_search", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class PlainCache:
    """Holds, for each slot, the codes' values and their scaling in the tensors' place."""

    @classmethod
    def allocate(cls, slots, heads, dim, *, bits, device):
        c = cls()
        c.bits, c.group = bits, dim if bits == 8 or dim % 32 else 32
        c.codes = torch.zeros(2, slots, heads, dim, dtype=torch.float64)
        c.params = torch.zeros(2, slots, heads, 2 * (dim // c.group), dtype=torch.float32)
        return c


class PlainReorder:
    def __init__(self, states, batch, beams):
        self.states = [(s, 0, None) if isinstance(s, torch.Tensor) else s for s in states]

    def reorder(self, parents, start=None, stop=None):
        p = parents.cpu().numpy()
        for t, rows, tokens in self.states:
            if tokens is None:
                there = t.movedim(rows, 0)[:, None]
                lo = hi = None
            else:
                there = t.movedim((rows, tokens), (0, 1))
                lo, hi = start.tolist(), stop.tolist()
            there.copy_(torch.from_numpy(reordered(there.cpu().numpy(), p, lo, hi)))


class Plain:
    QuantCache, StateReorder = PlainCache, PlainReorder

    @staticmethod
    def cache_write(cache, xs, slots):
        for part, x in enumerate(xs):
            code, scale, low = quantised(x.cpu().numpy(), cache.bits, cache.group)
            at = slots.cpu()
            cache.codes[part, at] = torch.from_numpy(code.reshape(x.shape))
            cache.params[part, at] = torch.from_numpy(np.concatenate((scale, low), -1))

    @staticmethod
    def cache_read(cache, slots, *, dtype):
        at, out = slots.cpu(), []
        for part in range(2):
            c = cache.codes[part, at].numpy()
            s, m = np.split(cache.params[part, at].numpy(), 2, -1)
            v = held_values(c.reshape(*c.shape[:-1], -1, cache.group), s, m, cache.bits)
            out.append(torch.from_numpy(v).to(dtype).cuda())
        return out

    @staticmethod
    def beam_select(logits, scores, n, *, bitmask, row_needs_mask, finished, pad_id, vocab_size):
        x, s = logits.double().cpu().numpy(), scores.cpu().numpy()
        batch, beams = s.shape
        words = bitmask.cpu().numpy().view(np.uint8)
        allowed = np.unpackbits(words, axis=1, bitorder="little")[:, :vocab_size] != 0
        allowed |= (row_needs_mask.cpu().numpy() == 0)[:, None]
        f = finished.cpu().numpy()
        out = (np.full((batch, n), -np.inf, np.float32), np.full((batch, n), -1, np.int64),
               np.full((batch, n), -1, np.int32))
        for b in range(batch):
            r = slice(b * beams, (b + 1) * beams)
            best = beam_candidates(x[r, :vocab_size], s[b], allowed=allowed[r], finished=f[b],
                                   pad=pad_id)[:n]
            for i, (v, k, t) in enumerate(best):
                out[0][b, i], out[1][b, i], out[2][b, i] = v, t, k
        return tuple(torch.from_numpy(o).cuda() for o in out)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("batch, beams, steps", [(1, 1, 6), (2, 4, 12), (3, 5, 9)])
def test_search_as_on_the_plain_definitions(example, bits, batch, beams, steps):
    model = example.Decoder(seed=batch)
    g = torch.Generator().manual_seed(beams)
    prompts = torch.randint(4, model.vocab, (batch, 5), generator=g).cuda()
    got = example.search(model, prompts, beams, steps, bits)
    want = example.search(model, prompts, beams, steps, bits, ops=Plain)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    # a step adds a score rounded to 32 bits and a log of a sum good to 4e-6 (the bound that
    # the selection's own tests derive); the caches hold the same values on both sides
    fine = torch.isfinite(want[1])
    assert torch.equal(fine, torch.isfinite(got[1]))
    off = (got[1][fine] - want[1][fine]).abs()
    assert bool((off <= steps * (4e-6 + 2.0 ** -23 * want[1][fine].abs())).all())


def test_search_keeps_to_the_grammar(example):
    model = example.Decoder(seed=9)
    prompts = torch.randint(4, model.vocab, (4, 3)).cuda()
    tokens, scores, ended = example.search(model, prompts, 6, 15, 4)
    grammar = example.Grammar(model.vocab)
    assert bool((scores[:, :-1] >= scores[:, 1:]).all()) and bool(ended.any())
    for row, done in zip(tokens.view(-1, 15).tolist(), ended.view(-1).tolist()):
        state = grammar.START
        for t in row:
            if state == grammar.DONE:
                assert t == grammar.END
                continue
            word = int(grammar.rows[state][t // 32]) & 0xffffffff
            assert word >> (t % 32) & 1, (row, t)
            state = grammar.advance(state, t)
        assert (state == grammar.DONE) == done
