#!/usr/bin/env python
"""Beam search under a grammar, with its cache held in 4 or 8 bits.

A small random decoder stands in for a model, and a state machine over token classes for a
grammar engine.  Each step of the search is what a serving loop would do:

  1. the new token's keys and values are quantised into the cache     (cache_write)
  2. the rows' history is read back for attention                     (cache_read)
  3. the host fills the grammar's bitmask for each live beam, and it is uploaded
     on a copy stream                                                 (BitmaskStager)
  4. the best continuations are selected over beams and vocabulary    (beam_select)
  5. caches and histories follow the beams, in place; the prompt, which all beams
     of a request share, stays where it is                            (StateReorder)

    python examples/constrained_beam_search.py [--bits 4|8] [--beams K] [--batch B]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from grammar_constrained_logit_gb300 import ops as lp  # noqa: E402


class Grammar:
    """Items in brackets: "[", then item tokens separated by commas, "]", then the end.
    Token 0 ends, 1 opens, 2 closes, 3 separates, the others are items (each item only
    after a separator or an opening)."""

    END, OPEN, CLOSE, COMMA = range(4)
    START, WANT_ITEM, HAVE_ITEM, CLOSED, DONE = range(5)

    def __init__(self, vocab: int):
        self.vocab, self.words = vocab, (vocab + 31) // 32
        items = torch.ones(self.words * 32, dtype=torch.bool)
        items[:4] = False
        items[vocab:] = False
        allowed = torch.zeros(5, self.words * 32, dtype=torch.bool)
        allowed[self.START, self.OPEN] = True
        allowed[self.WANT_ITEM] = items
        allowed[self.HAVE_ITEM, [self.CLOSE, self.COMMA]] = True
        allowed[self.CLOSED, self.END] = True
        bits = allowed.view(5, self.words, 32).to(torch.int64) << torch.arange(32)
        bits = bits.sum(-1)
        self.rows = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)

    def advance(self, state: int, token: int) -> int:
        if token == self.END:
            return self.DONE
        return {self.OPEN: self.WANT_ITEM, self.COMMA: self.WANT_ITEM,
                self.CLOSE: self.CLOSED}.get(token, self.HAVE_ITEM)


class Decoder:
    """A pre-norm transformer decoder with random weights, in 32 bits."""

    def __init__(self, vocab=1003, layers=2, heads=4, dim=32, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.vocab, self.layers, self.heads, self.dim = vocab, layers, heads, dim
        width = heads * dim

        def w(*shape):
            return (torch.randn(*shape, generator=g) / math.sqrt(shape[0])).to(device)

        self.embed = torch.randn(vocab, width, generator=g).to(device)
        self.qkv = [w(width, 3 * width) for _ in range(layers)]
        self.out = [w(width, width) for _ in range(layers)]
        self.up = [w(width, 2 * width) for _ in range(layers)]
        self.down = [w(2 * width, width) for _ in range(layers)]
        self.head = w(width, vocab) * 3.0

    def step(self, tokens, position, attend):
        """Logits [rows, vocab] after one token a row; ``attend(layer, q, k, v)`` stores
        the token's keys and values and returns the attention's output."""
        at = torch.arange(self.heads * self.dim, device=tokens.device)
        x = self.embed[tokens] + torch.sin(position * 0.1 * (at + 1).float())
        for i in range(self.layers):
            h = torch.nn.functional.layer_norm(x, x.shape[-1:])
            q, k, v = (h @ self.qkv[i]).view(-1, 3, self.heads, self.dim).unbind(1)
            x = x + attend(i, q, k, v).flatten(1) @ self.out[i]
            h = torch.nn.functional.layer_norm(x, x.shape[-1:])
            x = x + torch.relu(h @ self.up[i]) @ self.down[i]
        return torch.nn.functional.layer_norm(x, x.shape[-1:]) @ self.head


def search(model: Decoder, prompts: torch.Tensor, beams: int, steps: int, bits: int = 4, ops=lp):
    """Beam search from ``prompts`` int64 [batch, length].  Returns (tokens [batch, beams,
    steps], scores [batch, beams], ended [batch, beams]), best first."""
    batch, prompt = prompts.shape
    rows, length = batch * beams, prompt + steps
    dev = prompts.device
    grammar = Grammar(model.vocab)
    # slot of token t of row r: r * length + t, so a row's history is contiguous
    caches = [ops.QuantCache.allocate(rows * length, model.heads, model.dim, bits=bits, device=dev)
              for _ in range(model.layers)]
    history = torch.zeros(rows, steps, dtype=torch.int64, device=dev)
    states = [(t.unflatten(1, (rows, length)), 1, 2) for c in caches for t in (c.codes, c.params)]
    mover = ops.StateReorder(states, batch, beams)
    said = ops.StateReorder([history], batch, beams)
    first_slot = torch.arange(rows, device=dev)[:, None] * length
    start = torch.full((batch,), prompt, dtype=torch.int32, device=dev)
    stop = start.clone()
    stager = lp.BitmaskStager(rows, grammar.words, device=dev)

    def attend_at(position):
        read = (first_slot + torch.arange(position + 1, device=dev)).view(-1)
        write = (first_slot[:, 0] + position).contiguous()

        def attend(layer, q, k, v):
            ops.cache_write(caches[layer], (k, v), write)
            ks, vs = ops.cache_read(caches[layer], read, dtype=torch.float32)
            ks, vs = (t.view(rows, position + 1, model.heads, model.dim) for t in (ks, vs))
            p = torch.einsum("rhd,rthd->rht", q, ks) / math.sqrt(model.dim)
            return torch.einsum("rht,rthd->rhd", p.softmax(-1), vs)

        return attend

    for t in range(prompt):  # every beam of a request reads the same prompt
        token = prompts[:, t].repeat_interleave(beams)
        logits = model.step(token, t, attend_at(t))
    scores = torch.full((batch, beams), float("-inf"), device=dev)
    scores[:, 0] = 0.0  # the first step continues one beam; the others do not exist yet
    ended = torch.zeros(batch, beams, dtype=torch.bool, device=dev)
    grammar_state = [Grammar.START] * rows

    for t in range(steps):
        host_mask, host_flags = stager.host()
        for r, s in enumerate(grammar_state):
            host_flags[r] = s != Grammar.DONE
            if s != Grammar.DONE:
                host_mask[r] = grammar.rows[s]
        mask, flags = stager.upload()
        scores, tokens, parents = ops.beam_select(
            logits, scores, beams, bitmask=mask, row_needs_mask=flags, finished=ended,
            pad_id=Grammar.END, vocab_size=model.vocab)
        stager.consumed()

        mover.reorder(parents, start, stop)  # tokens [prompt, what is written so far)
        said.reorder(parents)
        there = parents >= 0  # fewer candidates than beams: the place stays empty
        ended = ended.gather(1, parents.clamp_min(0).long()) & there
        ended |= tokens == Grammar.END
        history[:, t] = tokens.view(-1).clamp_min(0)

        token_list, parent_list = tokens.view(-1).tolist(), parents.view(-1).tolist()
        was = grammar_state
        grammar_state = [
            was[r // beams * beams + p] if tok < 0 or was[r // beams * beams + p] == Grammar.DONE
            else grammar.advance(was[r // beams * beams + p], tok)
            for r, (tok, p) in enumerate(zip(token_list, (max(p, 0) for p in parent_list)))]
        if t + 1 < steps:
            logits = model.step(history[:, t], prompt + t, attend_at(prompt + t))
            stop += 1
    return history.view(batch, beams, steps), scores, ended


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--bits", type=int, default=4, choices=(4, 8))
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--steps", type=int, default=12)
    a = ap.parse_args()
    model = Decoder()
    prompts = torch.randint(4, model.vocab, (a.batch, 5), device="cuda")
    tokens, scores, ended = search(model, prompts, a.beams, a.steps, a.bits)
    for b in range(a.batch):
        print(f"request {b}:")
        for k in range(a.beams):
            said = [{0: ".", 1: "[", 2: "]", 3: ","}.get(t, str(t)) for t in tokens[b, k].tolist()]
            print(f"  {scores[b, k].item():9.4f} {'ended ' if ended[b, k] else 'going '}",
                  " ".join(said))


if __name__ == "__main__":
    main()
