"""Operators over the cache and over drafted tokens as measured cases: attention that reads the
cache's codes, eviction by accumulated attention weight, and verification of drafts.

``run`` computes each operator in its plain form (elementary torch operations) or, where
``own`` is true, through this package's entry points, on the same inputs.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
PAGE = 16  # slots of a page: the pages of a sequence lie anywhere in the cache
NEG = float("-inf")


# ------------------------------------------------------------------ the cases


def _attend(name, batch, rows, tokens, heads, shared, dim, bits, group, dtype, ragged=True,
            paged=True, window=0, weights=False):
    return {"name": name, "op": "attend", "batch": batch, "rows": rows, "tokens": tokens,
            "heads": heads, "shared": shared, "dim": dim, "bits": bits, "group": group,
            "dtype": dtype, "ragged": ragged, "paged": paged, "window": window,
            "weights": weights}


def _evict(name, batch, tokens, keep, first, recent, heads, dim, bits, group, ragged=True,
           paged=True):
    return {"name": name, "op": "evict", "batch": batch, "tokens": tokens, "keep": keep,
            "first": first, "recent": recent, "heads": heads, "dim": dim, "bits": bits,
            "group": group, "ragged": ragged, "paged": paged}


def _verify(name, slots, rows, vocab, cols, dtype, probs=True, keep=1.0, greedy=0.0, ragged=False):
    return {"name": name, "op": "verify", "slots": slots, "rows": rows, "vocab": vocab,
            "cols": cols, "dtype": dtype, "probs": probs, "keep": keep, "greedy": greedy,
            "ragged": ragged}


def listed():
    return [
        # one request early in its answer: a single token, latency alone counts
        _attend("attend one token", 1, 1, 250, 8, 4, 128, 8, 128, "bf16", ragged=False),
        # a serving batch's decoding step, sequences of all lengths on pages
        _attend("attend batch 8-bit", 32, 1, 8192, 8, 4, 128, 8, 128, "bf16"),
        # a few long documents in a 4-bit cache, eight query heads to each of its heads
        _attend("attend long 4-bit", 4, 1, 65536, 8, 8, 128, 4, 32, "bf16"),
        # drafted tokens to verify, a sliding window, heads of an odd number and width
        _attend("attend drafts window", 24, 5, 3001, 5, 3, 80, 4, 16, "f16", window=1024),
        # a prompt's next chunk over what the cache holds of it
        _attend("attend prompt chunk", 1, 1024, 16384, 8, 4, 128, 8, 128, "bf16", ragged=False),
        # a cache that is about to evict: every step adds its weights up; a model in 32 bits
        _attend("attend with weights", 16, 1, 4096, 8, 1, 64, 8, 64, "f32", paged=False,
                weights=True),
        # one request that reached its budget: little to move, latency alone counts
        _evict("evict one request", 1, 640, 512, 4, 64, 8, 128, 8, 128, ragged=False),
        # a serving batch cut to half, sequences of all lengths on pages
        _evict("evict batch", 32, 4096, 2048, 4, 256, 8, 128, 8, 128),
        # a few long documents cut to a quarter in a 4-bit cache
        _evict("evict long 4-bit", 4, 65536, 16384, 16, 1024, 8, 128, 4, 32, ragged=False),
        # one request's drafts: latency alone counts
        _verify("verify one slot", 1, 4, 32000, 32000, "f32"),
        # a full batch of eight rows a slot under a JSON-like grammar, logits padded to a width
        _verify("verify grammar batch", 64, 8, 128256, 128512, "bf16", keep=0.1),
        # drafts looked up in the prompt, which have no probabilities; some slots are greedy
        # and some have fewer drafts; rows that start at odd addresses
        _verify("verify looked up", 48, 5, 65519, 65519, "f16", probs=False, greedy=0.25,
                ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _cache_of(rng):
    heads, dim, bits = (rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 80, 96, 128, 192, 256]),
                        rng.choice([8, 4]))
    groups = (dim, dim, dim, 64, 32) if bits == 8 else (16, 32, 32, 64, dim)
    return heads, dim, bits, rng.choice([g for g in groups if dim % g == 0])


def draw(rng):
    op = rng.choice(["attend", "attend", "evict", "verify"])
    if op == "attend":
        heads, dim, bits, group = _cache_of(rng)
        shared = rng.choice([1, 2, 3, 4, 7, 8])
        rows = _log(rng, 16, 512) if rng.random() < 0.2 else rng.choice([1, 1, 1, 2, 4, 5, 8])
        batch = _log(rng, 1, max(1, 64 // rows))
        # bounded by the cache that is read, and by the products
        token = heads * (2 * dim * bits // 8 + dim // group * 8 + 9)
        most = min(250_000_000 // (batch * token),
                   1024 * 15800 * 32 * 128 // (batch * rows * heads * shared * dim), 65536)
        return {k: v for k, v in _attend(
            "", batch, rows, _log(rng, min(rows, most), most), heads, shared, dim, bits, group,
            rng.choice(["bf16", "f16", "f32"]), rng.random() < 0.7, rng.random() < 0.7,
            rng.choice([0, 0, 0, 127, 1024]), rng.random() < 0.3).items() if k != "name"}
    if op == "evict":
        heads, dim, bits, group = _cache_of(rng)
        batch = _log(rng, 1, 48)
        tokens = _log(rng, 16, min(65536, 16 * 4096 * 8 * 128 // (batch * heads * dim)))
        keep = max(8, int(tokens * rng.uniform(0.1, 1.1)))
        first = rng.choice([0, 4, 4])
        recent = int((keep - first) * rng.choice([0.0, 0.1, 0.5, 1.0]))
        return {k: v for k, v in _evict(
            "", batch, tokens, keep, first, recent, heads, dim, bits, group,
            rng.random() < 0.6, rng.random() < 0.7).items() if k != "name"}
    dtype = rng.choice(["f32", "f16", "bf16"])
    vocab, rows = _log(rng, 1000, 202048), rng.randint(1, 9)
    most = 64 * 8 * 128256 // (vocab * rows) // (SIZE[dtype] // 2)
    cols = rng.choice([vocab, -(-vocab // 256) * 256, vocab + rng.randrange(1, 64)])
    return {k: v for k, v in _verify(
        "", _log(rng, 1, max(1, min(128, most))), rows, vocab, cols, dtype, rng.random() < 0.7,
        rng.choice([1.0, 1.0, 0.5, 0.1]), rng.choice([0.0, 0.0, 0.3]),
        rng.random() < 0.4).items() if k != "name"}


# ----------------------------------------------------------------- the inputs


def _lengths(case):
    """Tokens of each sequence, the same for every seed (a seed shuffles the sequences), so
    that the work of a pass is known from the case."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    T = case["tokens"]
    if not case["ragged"]:
        return [T] * case["batch"]
    return [T] + [r.randint(min(T, case.get("rows", 1)), T) for _ in range(case["batch"] - 1)]


def _quantise(x, bits, group):
    """[n, heads, dim] float32 -> codes and what they are scaled by, as a cache holds them."""
    n, H, D = x.shape
    x = x.view(n, H, -1, group)
    if bits == 8:
        scale = (x.abs().amax(-1) * (1 / 448)).clamp_min(2.0 ** -126)
        y = (x * (1.0 / scale)[..., None]).clamp(-448.0, 448.0)
        return y.to(torch.float8_e4m3fn).view(torch.uint8).view(n, H, D), scale
    lo, hi = x.amin(-1), x.amax(-1)
    scale = ((hi * 0.5 - lo * 0.5) * (1 / 7.5)).clamp_min(2.0 ** -126).to(torch.bfloat16)
    low = lo.to(torch.bfloat16)
    y = (x - low.float()[..., None]) * (1.0 / scale.float())[..., None]
    code = y.clamp(0.0, 15.0).round().to(torch.uint8).view(n, H, D // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), torch.stack((scale, low), -1)


def _prepare_cache(s, case, seed, g):
    """Codes and params of keys and values, and where the sequences' tokens lie in them."""
    B, H, D, bits = case["batch"], case["heads"], case["dim"], case["bits"]
    lens = _lengths(case)
    random.Random(seed).shuffle(lens)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["block"] = PAGE if case["paged"] else case["tokens"]
    width = -(-max(lens) // s["block"])
    held = np.array([-(-n // s["block"]) for n in lens])
    total = int(held.sum()) + 2
    blocks = np.full((B, width), -1, np.int32)
    blocks[np.arange(width)[None, :] < held[:, None]] = \
        np.random.RandomState(seed % (1 << 31)).permutation(total)[:total - 2]
    s["blocks"] = torch.from_numpy(blocks).cuda()
    n = total * s["block"]
    s["codes"] = torch.empty(2, n, H, D * bits // 8, dtype=torch.uint8, device="cuda")
    s["params"] = (torch.empty(2, n, H, D // case["group"], device="cuda") if bits == 8 else
                   torch.empty(2, n, H, D // case["group"], 2, dtype=torch.bfloat16,
                               device="cuda"))
    # keys have channels that are large for every token, values have not
    channels = torch.randn(H, D, device="cuda", generator=g)
    channels = torch.where(channels > 1.5, 3.0 * channels, 0.0)
    for part in range(2):
        x = torch.randn(n, H, D, device="cuda", generator=g)
        s["codes"][part], s["params"][part] = _quantise(x if part else x + channels, bits,
                                                        case["group"])
    if own:
        from grammar_constrained_logit_gb300 import ops

        def shape(t):
            return t.unflatten(1, (total, PAGE)) if case["paged"] else t

        s["cache"] = ops.QuantCache(shape(s["codes"]), shape(s["params"]), dim=D, bits=bits)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    dev = {"device": "cuda", "generator": g}
    s = {"case": case}
    if case["op"] == "verify":
        S, R, V, cols = case["slots"], case["rows"], case["vocab"], case["cols"]
        s["logits"] = torch.empty(S, R, cols, dtype=TYPES[case["dtype"]], device="cuda")
        s["logits"].normal_(0.0, 3.0, generator=g)
        s["bitmask"] = s["needs"] = s["probs"] = None
        kept = None
        if case["keep"] < 1.0:
            words = (V + 31) // 32
            bits = torch.zeros(S * R, words, dtype=torch.int64, device="cuda")
            for i in range(32):
                bits |= (torch.rand(S * R, words, **dev) < case["keep"]).to(torch.int64) << i
            s["bitmask"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
            s["needs"] = (torch.rand(S * R, **dev) < 0.9).to(torch.uint8)
            token = torch.arange(V, device="cuda")
            kept = (bits[:, token >> 5] >> (token & 31)) & 1 == 1
            kept = (kept | (s["needs"] == 0)[:, None]).view(S, R, V)[:, :-1]
        s["temperature"] = torch.where(torch.rand(S, **dev) < case["greedy"], 0.0,
                                       0.6 + 0.6 * torch.rand(S, **dev))
        # a drafter that is near the target; looked-up drafts are often right, too
        near = s["logits"][:, :-1, :V].float()
        near = near + 0.7 * torch.randn(near.shape, **dev)
        if kept is not None:
            near = torch.where(kept, near, NEG)
        near = torch.softmax(near / s["temperature"].clamp_min(0.1)[:, None, None], -1)
        s["drafts"] = torch.zeros(S, R - 1, dtype=torch.int64, device="cuda")
        if R > 1:
            flat = near.reshape(S * (R - 1), V)
            noise = torch.empty_like(flat).exponential_(1.0, generator=g)
            s["drafts"] = (flat / noise).argmax(1).view(S, R - 1)
        if case["probs"]:
            s["probs"] = near.contiguous()
        else:
            sure = torch.rand(S, R - 1, **dev) < 0.6
            s["drafts"] = torch.where(sure, s["logits"][:, :-1, :V].float().argmax(-1),
                                      s["drafts"])
        if case["ragged"]:  # places without a draft
            there = torch.rand(S, 1, **dev) * 1.5 * R
            s["drafts"] = torch.where(torch.arange(R - 1, device="cuda") < there, s["drafts"], -1)
        s["uniforms"] = torch.rand(S, R - 1, **dev)
        s["seeds"] = torch.randint(0, 1 << 62, (S * R,), **dev)
        return s
    _prepare_cache(s, case, seed, g)
    B, H = case["batch"], case["heads"]
    width = s["blocks"].size(1) * s["block"]
    if case["op"] == "attend":
        q = torch.empty(B, case["rows"], H * case["shared"], case["dim"],
                        dtype=TYPES[case["dtype"]], device="cuda")
        s["q"] = q.normal_(0.0, 1.25, generator=g)
        s["weights"] = torch.rand(B, H, width, **dev) if case["weights"] else None
    else:
        # attention's weight is uneven: a few tokens have most of it
        s["seen"] = torch.randn(B, H, width, **dev).mul_(2.0).exp_()
        s["weights"] = torch.empty_like(s["seen"])
    return s


# ------------------------------------------------------------- the plain forms


def _values(codes, params, case):
    """The values that codes stand for, in 32 bits: [..., heads, dim]."""
    shape = codes.shape[:-1]
    if case["bits"] == 8:
        y = codes.view(torch.float8_e4m3fn).float().view(*shape, -1, case["group"])
        return (y * params[..., None]).flatten(-2)
    y = torch.stack((codes & 15, codes >> 4), -1).float().view(*shape, -1, case["group"])
    return (params[..., 1:].float() + y * params[..., :1].float()).flatten(-2)


def _places(s):
    """The slot of each token of each sequence."""
    at = torch.arange(s["block"], device="cuda")
    return (s["blocks"].long()[:, :, None] * s["block"] + at).flatten(1)


def _attended(s):
    case = s["case"]
    B, R, H, D = (case[k] for k in ("batch", "rows", "heads", "dim"))
    slots = _places(s)
    at = torch.arange(slots.size(1), device="cuda")
    held = at < s["lengths"][:, None]
    slots = torch.where(held, slots, 0)
    k = _values(s["codes"][0][slots], s["params"][0][slots], case)
    q = s["q"].float().view(B, R, H, -1, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    del k
    # row r of R sees what was there before it, and itself
    end = s["lengths"][:, None] - (R - 1 - torch.arange(R, device="cuda"))
    see = at < end[:, :, None]
    if case["window"]:
        see &= at >= end[:, :, None] - case["window"]
    x = x.view(B, H, -1, R, slots.size(1)).masked_fill_(~see[:, None, None], NEG)
    top = x.amax(-1, keepdim=True).clamp_min(-3e38)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total > 0, total, 1.0)
    if s["weights"] is not None:
        s["weights"] += p.sum((2, 3))
    v = _values(s["codes"][1][slots], s["params"][1][slots], case)
    v = v.masked_fill_(~held[..., None, None], 0.0)
    out = torch.matmul(p.flatten(2, 3), v.transpose(1, 2)).view(B, H, -1, R, D)
    return out.permute(0, 3, 1, 2, 4).reshape(B, R, -1, D).to(s["q"].dtype)


def _evicted(s):
    case, n = s["case"], s["lengths"].long()[:, None, None]
    B, H, keep = case["batch"], case["heads"], case["keep"]
    slots, w = _places(s), s["weights"]
    at = torch.arange(w.size(2), device="cuda")
    # the first and the last ones stay, then those of most weight, ties to the earliest
    worth = torch.where((at < case["first"]) | (at >= n - case["recent"]), math.inf, w)
    worth = torch.where(at < n, worth, NEG)
    kept = worth.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    left = n.clamp_max(keep)
    there = at[:kept.size(2)] < left
    kept = torch.where(there, kept, at.numel()).sort(-1).values.clamp_max(at.numel() - 1)
    where = there.expand(B, H, -1)
    row = torch.arange(B, device="cuda")[:, None, None].expand(where.shape)
    head = torch.arange(H, device="cuda")[:, None].expand(where.shape)[where]
    to = slots[row, at[:kept.size(2)].expand(where.shape)][where]
    source = slots[row, kept][where]
    s["codes"][:, to, head] = s["codes"][:, source, head]
    s["params"][:, to, head] = s["params"][:, source, head]
    moved = torch.where(where, w.gather(2, kept), 0.0)
    moved = torch.nn.functional.pad(moved, (0, at.numel() - moved.size(2)))
    w.copy_(torch.where(at < n, moved, w))
    return left.view(-1).to(torch.int32)


def _high(a, m):
    """The upper 32 bits of a * m, of numbers below 2^32 in int64."""
    return (a * (m >> 16) + ((a * (m & 0xffff)) >> 16)) >> 16


def _round(c, k, i):
    """One of Philox4x32's ten rounds (Salmon et al., SC'11)."""
    k0, k1 = (k[0] + i * 0x9E3779B9) & 0xffffffff, (k[1] + i * 0xBB67AE85) & 0xffffffff
    return (_high(c[2], 0xCD9E8D57) ^ c[1] ^ k0, (c[2] * 0xCD9E8D57) & 0xffffffff,
            _high(c[0], 0xD2511F53) ^ c[3] ^ k1, (c[0] * 0xD2511F53) & 0xffffffff)


def _gumbel(seed, row, vocab):
    """The sampler's noise of rows `row` keyed by `seed`: word (v & 3) of the block v >> 2."""
    block = torch.arange((vocab + 3) // 4, device="cuda").expand(row.numel(), -1)
    zero = torch.zeros_like(block)
    k = (seed & 0xffffffff)[:, None], ((seed >> 32) & 0xffffffff)[:, None]
    c = block, zero + row[:, None], zero, zero
    c = _round(_round(_round(_round(_round(c, k, 0), k, 1), k, 2), k, 3), k, 4)
    c = _round(_round(_round(_round(_round(c, k, 5), k, 6), k, 7), k, 8), k, 9)
    u = ((torch.stack(c, -1).flatten(1)[:, :vocab] >> 9).double() + 0.5) * 2.0 ** -23
    return -torch.log(-torch.log(u))


def _verified(s):
    case = s["case"]
    S, R, V = case["slots"], case["rows"], case["vocab"]
    # 64 bits: an acceptance hangs on the last places of its two probabilities
    x = s["logits"][:, :, :V].double()
    token = torch.arange(V, device="cuda")
    if s["bitmask"] is not None:
        bits = (s["bitmask"][:, token >> 5] >> (token & 31).to(torch.int32)) & 1
        kept = (bits == 1) | (s["needs"] == 0)[:, None]
        x = torch.where(kept.view(S, R, V), x, NEG)
    heat = s["temperature"].double()[:, None, None]
    top = x.amax(-1, keepdim=True)
    first = torch.where(x == top, token, V).amin(-1, keepdim=True)  # ties to the lowest
    p = torch.exp((x - top) / torch.where(heat > 0, heat, 1.0))
    p = p / p.sum(-1, keepdim=True)
    p = torch.where(heat > 0, p, (token == first).double())
    drafts, slot = s["drafts"], torch.arange(S, device="cuda")
    there = (drafts >= 0) & (drafts < V)
    at = drafts.clamp(0, V - 1)[..., None]
    mine = p[:, :-1].gather(2, at)[..., 0]
    theirs = s["probs"].gather(2, at)[..., 0] if s["probs"] is not None else 1.0
    taken = there & (s["uniforms"].double() * theirs < mine)
    count = taken.to(torch.int64).cumprod(1).sum(1)
    # the row after the accepted ones draws: from what the draft left where it was refused
    last = p[slot, count]
    refused = torch.nn.functional.pad(there, (0, 1))[slot, count]
    less = torch.zeros_like(last)
    if R > 1:
        i = count.clamp_max(R - 2)
        less = (s["probs"][slot, i].double() if s["probs"] is not None else
                (token == drafts[slot, i][:, None]).double())
    rest = torch.where(refused[:, None], (last - less).clamp_min(0.0), last)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, last)
    row = slot * R + count
    score = torch.log(rest) + _gumbel(s["seeds"][row], row, V)
    drawn = torch.where(score == score.amax(-1, keepdim=True), token, V).amin(-1)
    place = torch.arange(R, device="cuda")
    said = torch.nn.functional.pad(drafts, (0, 1))
    said = torch.where(place < count[:, None], said, -1)
    said = torch.where(place == count[:, None], drawn[:, None], said)
    return said, count.to(torch.int32)


def run(state):
    s, case = state, state["case"]
    if own:
        from grammar_constrained_logit_gb300 import ops

    if case["op"] == "attend":
        if own:
            out = ops.cache_attend(s["cache"], s["q"], s["blocks"], s["lengths"],
                                   block_size=s["block"], window=case["window"] or None,
                                   weights=s["weights"])
        else:
            out = _attended(s)
        return [out] if s["weights"] is None else [out, s["weights"]]
    if case["op"] == "evict":
        # what the steps since the last eviction added up: an eviction changes it in place
        s["weights"].copy_(s["seen"])
        if own:
            left = ops.cache_evict(s["cache"], s["weights"], s["blocks"], s["lengths"],
                                   case["keep"], first=case["first"], recent=case["recent"],
                                   block_size=s["block"])
        else:
            left = _evicted(s)
        return [left, s["weights"], s["codes"], s["params"]]
    if own:
        return ops.verify_drafts(s["logits"], s["drafts"], s["uniforms"], draft_probs=s["probs"],
                                 bitmask=s["bitmask"], row_needs_mask=s["needs"],
                                 temperature=s["temperature"], seeds=s["seeds"],
                                 vocab_size=case["vocab"])
    return _verified(s)


# ------------------------------------------------------------------- the work


def _token_bytes(case):
    """Of a token's codes and params, for one head of one part."""
    return case["dim"] * case["bits"] // 8 + case["dim"] // case["group"] * 4


def work(case):
    if case["op"] == "verify":
        S, R, V, e = case["slots"], case["rows"], case["vocab"], SIZE[case["dtype"]]
        # memory is read in sectors of 32 bytes: the share that holds a kept token
        touched, mask = 1.0, 0.0
        if case["keep"] < 1.0:
            touched = 0.1 + 0.9 * (1 - (1 - case["keep"]) ** (32 // e))
            mask = 0.9 * V / 8
        # every row once, and the draft's probabilities of the row that draws in its place
        probs = S * 4 * V * touched if case["probs"] and R > 1 else 0
        return {"bytes": S * R * (touched * V * e + mask) + probs + S * R * 40,
                "flops": 4.0 * S * R * V * case["keep"]}
    lens = _lengths(case)
    H, token = case["heads"], case["heads"] * 2 * _token_bytes(case)
    if case["op"] == "attend":
        R, W = case["rows"], case["window"]
        ends = [[max(0, n - (R - 1 - r)) for r in range(R)] for n in lens]
        seen = sum(min(e, W) if W else e for es in ends for e in es)
        read = sum(n - (max(0, es[0] - W) if W else 0) for n, es in zip(lens, ends))
        q = case["batch"] * R * H * case["shared"] * case["dim"] * SIZE[case["dtype"]]
        return {"bytes": read * token + 2 * q + read // 4 +
                (read * H * 8 if case["weights"] else 0),
                "flops": 4.0 * seen * H * case["shared"] * case["dim"]}
    # tokens that move: the kept ones behind the first that goes
    kept = [min(n, case["keep"]) for n in lens]
    moved = sum(k - min(k, case["first"]) for n, k in zip(lens, kept) if n > k)
    return {"bytes": 2.0 * moved * token + sum(lens) * H * (4 + 8) + sum(kept) * H * 4,
            "flops": 4.0 * sum(lens) * H}


# ------------------------------------------------------------ in 64 bits, apart


def exact(case, seed):
    if case["op"] != "attend":
        return None  # whole numbers, and bytes that move
    s = prepare(case, seed)
    D, R, size, bits = case["dim"], case["rows"], case["group"], case["bits"]
    byte = torch.arange(256, device="cuda")
    if bits == 8:  # sign, four bits of exponent, three of fraction; 127 is no number
        e, m = (byte >> 3) & 15, (byte & 7).double()
        value = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.double() - 10))
        value = torch.where(byte >= 128, -value, value)[:, None]
    else:
        value = torch.stack((byte % 16, byte // 16), 1).double()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    weights = None if s["weights"] is None else s["weights"].double()
    for b, n in enumerate(s["lengths"].tolist()):
        lo = max(0, n - R + 1 - case["window"]) if case["window"] else 0
        t = torch.arange(lo, n, device="cuda")
        slot = s["blocks"][b].long()[t // s["block"]] * s["block"] + t % s["block"]
        end = n - R + 1 + torch.arange(R, device="cuda")[:, None]
        hidden = t >= end
        if case["window"]:
            hidden |= t < end - case["window"]
        for h in range(case["heads"]):
            k, v = (value[s["codes"][p, slot, h].long()].reshape(n - lo, -1, size)
                    for p in range(2))
            ks, vs = (s["params"][p, slot, h].double() for p in range(2))
            if bits == 8:
                k, v = k * ks[..., None], v * vs[..., None]
            else:
                k, v = ks[..., 1:] + k * ks[..., :1], vs[..., 1:] + v * vs[..., :1]
            mine = slice(h * case["shared"], (h + 1) * case["shared"])
            x = torch.einsum("rgd,td->grt", s["q"][b, :, mine].double(), k.reshape(-1, D))
            x = (x / math.sqrt(D)).masked_fill(hidden, NEG)
            p = torch.softmax(x, -1)
            p = torch.where(hidden.all(-1)[:, None], 0.0, p)
            out[b, :, mine] = torch.einsum("grt,td->rgd", p, v.reshape(-1, D))
            if weights is not None:
                weights[b, h, lo:n] += p.sum((0, 1))
    return [out] if weights is None else [out, weights]
