#!/usr/bin/env python
"""Speculative decoding under a grammar, over a quantised cache of bounded size.

A small random decoder stands in for a model, its first embedding alone for a drafter, and a
state machine over token classes for a grammar engine.  Each step is what a serving loop would
do:

  1. the drafter says a few tokens ahead, each drawn under the grammar's mask
  2. the model takes all of them at once: their keys and values are quantised into the cache
                                                                     (cache_write)
     and every row attends to the cache's codes, adding up each token's attention weight
                                                                     (cache_attend)
  3. drafts are accepted or refused so that what is said follows the model's distribution
     under the mask, and one token more is drawn                     (verify_drafts)
  4. what was refused is forgotten: the sequence's length says so
  5. a sequence that outgrew its budget keeps its first tokens, its last ones, and of those
     between the ones that were attended to most, each head its own  (cache_evict)

    python examples/speculative_decoding.py [--bits 4|8] [--batch B] [--drafts K] [--budget T]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for path in (ROOT, os.path.join(ROOT, "examples")):
    if path not in sys.path:
        sys.path.insert(0, path)

from constrained_beam_search import Decoder, Grammar  # noqa: E402
from grammar_constrained_logit_gb300 import ops as lp  # noqa: E402

FIRST, RECENT = 2, 6  # tokens that always stay


def draft(model: Decoder, grammar: Grammar, last, states, count, g):
    """``count`` drafts for each sequence: (tokens [batch, count] (-1 after the end), the
    probabilities they were drawn from, the grammar's states before each row)."""
    tokens, probs, before = [], [], [list(states)]
    for _ in range(count):
        x = torch.nn.functional.layer_norm(model.embed[last], model.embed.shape[-1:])
        allowed = torch.stack([grammar.rows[s] if s != Grammar.DONE else
                               torch.zeros_like(grammar.rows[0]) for s in before[-1]])
        bits = (allowed[:, :, None] >> torch.arange(32)) & 1
        kept = bits.flatten(1)[:, :model.vocab].bool().to(last.device)
        p = torch.softmax((x @ model.head).masked_fill(~kept, float("-inf")), -1).nan_to_num(0.0)
        noise = torch.rand(p.shape, generator=g).to(p.device)
        t = (p / -torch.log(noise)).argmax(-1)
        ended = torch.tensor([s == Grammar.DONE for s in before[-1]], device=last.device)
        tokens.append(torch.where(ended, -1, t))
        probs.append(p)
        last = t
        said = tokens[-1].tolist()
        before.append([s if s == Grammar.DONE else grammar.advance(s, k)
                       for s, k in zip(before[-1], said)])
    return torch.stack(tokens, 1), torch.stack(probs, 1), before


def generate(model: Decoder, prompts: torch.Tensor, steps: int, drafts: int = 3, bits: int = 8,
             budget: int = 24, temperature: float = 0.8, seed: int = 0, ops=lp):
    """Continues ``prompts`` int64 [batch, length] by ``steps`` verifications.  Returns what
    each sequence says, and how many of its drafts were accepted."""
    batch, prompt = prompts.shape
    rows, dev = drafts + 1, prompts.device
    room = max(budget, prompt) + rows  # places of a sequence: the budget, and a step's rows
    grammar = Grammar(model.vocab)
    caches = [ops.QuantCache.allocate(batch * room, model.heads, model.dim, bits=bits, device=dev)
              for _ in range(model.layers)]
    weights = [torch.zeros(batch, model.heads, room, device=dev) for _ in range(model.layers)]
    blocks = torch.arange(batch, dtype=torch.int32, device=dev)[:, None]  # a block a sequence
    lengths = torch.zeros(batch, dtype=torch.int32, device=dev)
    position = torch.zeros(batch, dtype=torch.int64, device=dev)  # goes on through evictions
    place = torch.arange(room, device=dev)
    stager = lp.BitmaskStager(batch * rows, grammar.words, device=dev)
    g = torch.Generator().manual_seed(seed)

    def forward(tokens, lengths):
        """Logits [batch, n, vocab] after n tokens a sequence, the first at `lengths`."""
        n = tokens.size(1)
        at = lengths[:, None] + torch.arange(n, device=dev)
        slots = (blocks * room + at).view(-1).long()

        def attend(layer, q, k, v):
            ops.cache_write(caches[layer], (k, v), slots)
            return ops.cache_attend(caches[layer], q.view(batch, n, model.heads, -1), blocks,
                                    lengths + n, block_size=room,
                                    weights=weights[layer]).flatten(0, 1)

        where = (position[:, None] + torch.arange(n, device=dev)).view(-1, 1)
        return model.step(tokens.reshape(-1), where, attend).view(batch, n, -1)

    if prompt > 1:
        forward(prompts[:, :-1].contiguous(), lengths)
    lengths, position = lengths + (prompt - 1), position + (prompt - 1)
    last = prompts[:, -1]
    states = [Grammar.START] * batch
    said: list = [[] for _ in range(batch)]
    accepted = [0] * batch

    for step in range(steps):
        guesses, probs, before = draft(model, grammar, last, states, drafts, g)
        logits = forward(torch.cat((last[:, None], guesses.clamp_min(0)), 1), lengths)
        host_mask, host_flags = stager.host()
        for b in range(batch):
            for r in range(rows):
                host_flags[b * rows + r] = before[r][b] != Grammar.DONE
                if before[r][b] != Grammar.DONE:
                    host_mask[b * rows + r] = grammar.rows[before[r][b]]
        mask, flags = stager.upload()
        tokens, count = ops.verify_drafts(
            logits, guesses, torch.rand(guesses.shape, generator=g).to(dev), draft_probs=probs,
            bitmask=mask, row_needs_mask=flags, temperature=temperature, seed=seed, offset=step,
            vocab_size=model.vocab)
        stager.consumed()

        # the last token said has no place in the cache yet: it is the next step's first row
        lengths = lengths + 1 + count
        position = position + 1 + count
        last = tokens.gather(1, count.long()[:, None])[:, 0].clamp_min(0)
        for w in weights:  # what was refused has no weight
            w.masked_fill_((place >= lengths[:, None])[:, None], 0.0)
        for b, (row, n) in enumerate(zip(tokens.tolist(), count.tolist())):
            for t in row[:n + 1]:
                if states[b] != Grammar.DONE and t >= 0:
                    said[b].append(t)
                    states[b] = grammar.advance(states[b], t)
            accepted[b] += n
        for layer, cache in enumerate(caches):
            left = ops.cache_evict(cache, weights[layer], blocks, lengths, budget, first=FIRST,
                                   recent=RECENT, block_size=room)
        lengths = left
    return said, accepted


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--bits", type=int, default=8, choices=(4, 8))
    ap.add_argument("--batch", type=int, default=3)
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--budget", type=int, default=24)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    model = Decoder()
    prompts = torch.randint(4, model.vocab, (a.batch, 12), device="cuda")
    said, accepted = generate(model, prompts, a.steps, a.drafts, a.bits, a.budget)
    for b, row in enumerate(said):
        text = [{0: ".", 1: "[", 2: "]", 3: ","}.get(t, str(t)) for t in row]
        print(f"request {b}: {accepted[b]} drafts accepted:", " ".join(text))


if __name__ == "__main__":
    main()
