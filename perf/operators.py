"""The beam-search operators as measured cases: selection over beams and vocabulary, the
reordering of states, and the cache quantised as it is written and read back.

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
LARGEST = 3.3895313892515355e38  # the largest bf16: what is beyond it counts as an infinity
TINY = 2.0 ** -126


# ------------------------------------------------------------------ the cases


def _beam(name, batch, beams, vocab, cols, n, dtype, keep=1.0, alive="all", finished=0.0):
    return {"name": name, "op": "beam", "batch": batch, "beams": beams, "vocab": vocab,
            "cols": cols, "n": n, "dtype": dtype, "keep": keep, "alive": alive,
            "finished": finished}


def _reorder(name, batch, beams, tokens, layers, heads, dim, kind, layout, ragged):
    return {"name": name, "op": "reorder", "batch": batch, "beams": beams, "tokens": tokens,
            "layers": layers, "heads": heads, "dim": dim, "kind": kind, "layout": layout,
            "ragged": ragged}


def _cache(name, op, n, heads, dim, bits, group, dtype, fused=False, padded=0.0):
    return {"name": name, "op": op, "n": n, "heads": heads, "dim": dim, "bits": bits,
            "group": group, "dtype": dtype, "fused": fused, "padded": padded}


def listed():
    return [
        # the first step of one request: only its first beam is alive, latency alone counts
        _beam("beam first step", 1, 4, 32000, 32000, 8, "f32", alive="first"),
        # a few requests under a JSON-like grammar, vocabulary padded to the logits' width
        _beam("beam grammar", 8, 4, 128256, 128512, 8, "bf16", keep=0.01, finished=0.1),
        # rows that start at odd addresses, ended hypotheses, an odd number of beams
        _beam("beam odd vocabulary", 24, 5, 65519, 65519, 10, "f16", alive="some", finished=0.1),
        # retrieval by generated identifiers: many beams over a constrained vocabulary
        _beam("beam many", 4, 64, 32000, 32000, 128, "bf16", keep=0.1),
        # a full serving batch over the largest vocabulary
        _beam("beam full batch", 128, 8, 202048, 202048, 16, "f16"),
        # one request after a short answer: a few small tensors, latency alone counts
        _reorder("reorder one request", 1, 4, 256, 2, 8, 128, "bf16", "tokens", False),
        # caches laid out heads first, with answers of different lengths after their prompts
        _reorder("reorder heads first", 16, 5, 1000, 4, 8, 128, "bf16", "heads", True),
        # a serving batch's 8-bit cache with its scales: the largest thing a step moves
        _reorder("reorder 8-bit cache", 32, 4, 2048, 8, 8, 128, "q8", "tokens", True),
        # one decoded token a row
        _cache("write one token a row", "write", 32, 8, 128, 8, 128, "bf16", fused=True),
        # a long prompt's keys and values, out of the fused projection
        _cache("write long prompt", "write", 32768, 8, 128, 8, 128, "bf16", fused=True,
               padded=0.02),
        # a prompt's chunk that attends to its own quantised values; heads of an odd width
        _cache("write and read 4-bit", "both", 6001, 5, 80, 4, 16, "f32"),
        # a long shared prefix read back for the next prompts
        _cache("read 4-bit prefix", "read", 131072, 8, 128, 4, 32, "bf16", padded=0.01),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["beam", "beam", "reorder", "cache"])
    if op == "beam":
        dtype = rng.choice(["f32", "f16", "bf16"])
        vocab = _log(rng, 1000, 202048)
        beams = rng.choice([1, 2, 3, 4, 5, 8, 10, 16, 32, 64])
        most = 1024 * 202048 * 2 // (vocab * SIZE[dtype] * beams)
        batch = _log(rng, 1, max(1, min(256, most)))
        cols = rng.choice([vocab, -(-vocab // 256) * 256, vocab + rng.randrange(1, 64)])
        return {k: v for k, v in _beam(
            "", batch, beams, vocab, cols, rng.choice([beams, 2 * beams]), dtype,
            rng.choice([1.0, 1.0, 0.5, 0.1, 0.01]), rng.choice(["all", "all", "some", "first"]),
            rng.choice([0.0, 0.0, 0.2])).items() if k != "name"}
    if op == "reorder":
        heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 128])
        kind, layers = rng.choice(["bf16", "q8", "q4"]), rng.randint(1, 8)
        batch, beams = _log(rng, 1, 48), rng.choice([2, 3, 4, 5, 8, 10, 16])
        size = dim * 2 if kind == "bf16" else dim + 4 if kind == "q8" else dim // 2 + dim // 4
        most = 128 * 2048 * 8 * 132 * 8 // (batch * beams * heads * size * layers)
        return {k: v for k, v in _reorder(
            "", batch, beams, _log(rng, 1, max(1, min(4096, most))), layers, heads, dim, kind,
            rng.choice(["tokens", "heads"]), rng.random() < 0.6).items() if k != "name"}
    what, bits = rng.choice(["write", "both", "read"]), rng.choice([8, 4])
    if bits == 4 and what == "write":
        what = "both"
    heads, dim = rng.choice([1, 2, 5, 8, 16]), rng.choice([64, 72, 80, 96, 128, 192, 256, 576])
    group = rng.choice([g for g in (8, 16, 32, 64, 128, dim) if dim % g == 0])
    dtype = rng.choice(["f32", "f16", "bf16"])
    most = 131072 * 8 * 128 * 2 // (heads * dim * SIZE[dtype])
    return {k: v for k, v in _cache(
        "", what, _log(rng, 1, most // (2 if what == "both" else 1)), heads, dim, bits, group,
        dtype, rng.random() < 0.5, rng.choice([0.0, 0.02])).items() if k != "name"}


# ----------------------------------------------------------------- the inputs


def _pattern(case):
    """What a reorder's batches do: (parents, start, stop) of each, the same for every seed
    (a seed shuffles the batches), so that the work of a pass is known from the case."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    K, T = case["beams"], case["tokens"]
    weights = [0.6 ** j for j in range(K)]  # the better half of the beams has most successors
    made = []
    for _ in range(case["batch"]):
        stop = r.randint(1, T) if case["ragged"] else (T + 1) // 2
        start = r.randint(0, stop) // 2 if case["ragged"] else 0
        made.append((r.choices(range(K), weights, k=K), start, stop))
    return made


def _slots(case, seed):
    n, r = case["n"], np.random.RandomState(seed % (1 << 31))
    pages = -(-n // PAGE) + 3
    order = r.permutation(pages)
    at = np.arange(n)
    slots = order[at // PAGE].astype(np.int64) * PAGE + at % PAGE
    if case["padded"]:
        slots[r.rand(n) < case["padded"]] = -1  # padding of the batch: no slot
    return pages * PAGE, torch.from_numpy(slots).cuda()


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    dev = {"device": "cuda", "generator": g}
    s = {"case": case}
    if case["op"] == "beam":
        B, K, V, cols = case["batch"], case["beams"], case["vocab"], case["cols"]
        R = B * K
        s["logits"] = torch.empty(R, cols, dtype=TYPES[case["dtype"]], device="cuda")
        s["logits"].normal_(0.0, 2.5, generator=g)
        scores = -torch.rand(B, K, **dev) * 12.0 - 1.0
        scores = scores.sort(1, descending=True).values
        if case["alive"] == "first":
            scores[:, 1:] = NEG
        elif case["alive"] == "some":
            scores = torch.where(torch.rand(B, K, **dev) < 0.15, NEG, scores)
        s["scores"] = scores.contiguous()
        s["bitmask"] = s["needs"] = s["finished"] = None
        if case["keep"] < 1.0:
            words = (V + 31) // 32
            bits = torch.zeros(R, words, dtype=torch.int64, device="cuda")
            for i in range(32):
                bits |= (torch.rand(R, words, **dev) < case["keep"]).to(torch.int64) << i
            s["bitmask"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
            s["needs"] = (torch.rand(R, **dev) < 0.9).to(torch.uint8)
        if case["finished"]:
            s["finished"] = (torch.rand(R, **dev) < case["finished"]).to(torch.uint8)
    elif case["op"] == "reorder":
        B, K, T, H, D = (case[k] for k in ("batch", "beams", "tokens", "heads", "dim"))
        R = B * K
        made = _pattern(case)
        random.Random(seed).shuffle(made)
        s["parents"] = torch.tensor([m[0] for m in made], dtype=torch.int32, device="cuda")
        s["start"] = torch.tensor([m[1] for m in made], dtype=torch.int32, device="cuda")
        s["stop"] = torch.tensor([m[2] for m in made], dtype=torch.int32, device="cuda")

        def shape(*rest):
            return (2, R, T, H, *rest) if case["layout"] == "tokens" else (2, R, H, T, *rest)

        def make(dtype, *rest):
            if dtype == torch.uint8:
                return torch.randint(0, 256, shape(*rest), dtype=dtype, **dev)
            t = torch.empty(shape(*rest), dtype=dtype, device="cuda")
            return t.normal_(0.0, 1.0, generator=g)

        at = 2 if case["layout"] == "tokens" else 3
        # (tensor, axis of the rows, axis of the tokens): keys and values of each layer
        s["states"] = []
        for _ in range(case["layers"]):
            if case["kind"] == "bf16":
                s["states"].append((make(torch.bfloat16, D), 1, at))
            elif case["kind"] == "q8":
                s["states"].append((make(torch.uint8, D), 1, at))
                s["states"].append((make(torch.float32, 1), 1, at))
            else:
                s["states"].append((make(torch.uint8, D // 2), 1, at))
                s["states"].append((make(torch.bfloat16, D // 16, 2), 1, at))
        # and the tokens that each row has said
        s["states"].append((torch.randint(0, 32000, (R, T), **dev), 0, 1))
        if own:
            from grammar_constrained_logit_gb300 import ops

            s["mover"] = ops.StateReorder(s["states"], B, K)
    else:
        H, D, G = case["heads"], case["dim"], case["dim"] // case["group"]
        total, s["slots"] = _slots(case, seed)
        s["codes"] = torch.zeros(2, total, H, D * case["bits"] // 8, dtype=torch.uint8,
                                 device="cuda")
        s["params"] = (torch.zeros(2, total, H, G, device="cuda") if case["bits"] == 8 else
                       torch.zeros(2, total, H, G, 2, dtype=torch.bfloat16, device="cuda"))
        dtype = TYPES[case["dtype"]]
        if case["op"] == "read":
            for part in range(2):
                codes, params = _quantise(torch.randn(total, H, D, **dev), case)
                s["codes"][part], s["params"][part] = codes, params
        elif case["fused"]:  # keys and values are columns of one projection's output
            kv = torch.empty(case["n"], 2 * H * D, dtype=dtype, device="cuda")
            kv.normal_(0.0, 1.0, generator=g)
            s["x"] = [kv[:, :H * D].view(-1, H, D), kv[:, H * D:].view(-1, H, D)]
        else:
            s["x"] = [torch.empty(case["n"], H, D, dtype=dtype, device="cuda").normal_(
                0.0, 1.0, generator=g) for _ in range(2)]
        if own:
            from grammar_constrained_logit_gb300 import ops

            s["cache"] = ops.QuantCache(s["codes"], s["params"], dim=D, bits=case["bits"])
    return s


# ------------------------------------------------------------- the plain forms


def _select(s):
    case = s["case"]
    B, K, V, n = (case[k] for k in ("batch", "beams", "vocab", "n"))
    x = s["logits"][:, :V].float() + 0.0
    kept = x > NEG
    token = torch.arange(V, device="cuda")
    if s["bitmask"] is not None:
        bits = (s["bitmask"][:, token >> 5] >> (token & 31).to(torch.int32)) & 1
        kept &= (bits == 1) | (s["needs"] == 0)[:, None]
    x = torch.where(kept, x, NEG)
    top = x.amax(1, keepdim=True).double()
    # 64 bits: the order of two beams' candidates hangs on their sums' last places
    z = torch.where(kept, torch.exp(x.double() - top), 0.0).sum(1, keepdim=True).log()
    # a row's best tokens, ties to the lowest: the logit's order and the token in one number
    i = x.view(torch.int32).to(torch.int64)
    key = torch.where(i < 0, -(i + (1 << 31)), i) * (1 << 31) + (V - 1 - token)
    best = key.topk(min(n, V), dim=1).indices
    score = s["scores"].view(-1, 1).double()
    live = kept.gather(1, best) & (score > NEG)
    cand = torch.where(live, score + (x.gather(1, best).double() - top - z), NEG)
    if s["finished"] is not None:  # an ended hypothesis goes on as it is
        ended = (s["finished"] != 0)[:, None]
        first = torch.arange(best.size(1), device="cuda") == 0
        cand = torch.where(ended, torch.where(first & (score > NEG), score, NEG), cand)
        best = torch.where(ended, 0, best)
    cand, order = cand.view(B, -1).sort(dim=1, descending=True, stable=True)
    cand, order = cand[:, :n], order[:, :n]
    there = cand > NEG
    return (cand.float(), torch.where(there, best.view(B, -1).gather(1, order), -1),
            torch.where(there, order // min(n, V), -1).to(torch.int32))


def _move(t, rows, tokens, source, held):
    """One state after a reorder: `source` has each row's new row, `held` the (row, token)s
    that take part."""
    there = t.movedim((rows, tokens), (0, 1))
    new = torch.where(held.view(held.shape + (1,) * (t.dim() - 2)),
                      there.index_select(0, source), there)
    there.copy_(new)
    return t


def _reordered(s):
    case = s["case"]
    B, K, T = case["batch"], case["beams"], case["tokens"]
    source = (s["parents"].long() + torch.arange(B, device="cuda")[:, None] * K).view(-1)
    at = torch.arange(T, device="cuda")
    held = (at >= s["start"][:, None]) & (at < s["stop"][:, None])
    held = held.repeat_interleave(K, 0)
    return [_move(t, rows, tokens, source, held) for t, rows, tokens in s["states"]]


def _quantise(x, case):
    """[n, heads, dim] -> codes and what they are scaled by."""
    n, H, D = x.shape
    x = x.float().reshape(n, H, -1, case["group"])
    fine = x.abs() <= LARGEST
    if case["bits"] == 8:
        scale = (torch.where(fine, x.abs(), 0.0).amax(-1) * (1 / 448)).clamp_min(TINY)
        y = (x * (1.0 / scale)[..., None]).clamp(-448.0, 448.0)
        return y.to(torch.float8_e4m3fn).view(torch.uint8).view(n, H, D), scale
    lo = torch.where(fine, x, math.inf).amin(-1)
    hi = torch.where(fine, x, -math.inf).amax(-1)
    lo, hi = torch.where(lo <= hi, lo, 0.0), torch.where(lo <= hi, hi, 0.0)
    scale = ((hi * 0.5 - lo * 0.5) * (1 / 7.5)).clamp_min(TINY).to(torch.bfloat16)
    low = lo.to(torch.bfloat16)
    y = (x - low.float()[..., None]) * (1.0 / scale.float())[..., None]
    code = y.clamp(0.0, 15.0).round().to(torch.uint8).view(n, H, D // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), torch.stack((scale, low), -1)


def _values(codes, params, case):
    """The values that codes stand for, in 32 bits: [n, heads, dim]."""
    n, H = codes.shape[:2]
    if case["bits"] == 8:
        y = codes.view(torch.float8_e4m3fn).float().view(n, H, -1, case["group"])
        return (y * params[..., None]).view(n, H, -1)
    y = torch.stack((codes & 15, codes >> 4), -1).float().view(n, H, -1, case["group"])
    return (params[..., 1:].float() + y * params[..., :1].float()).view(n, H, -1)


def _written(s):
    case, slots = s["case"], s["slots"]
    taken = slots >= 0
    at = slots[taken]
    (k, ks), (v, vs) = _quantise(s["x"][0][taken], case), _quantise(s["x"][1][taken], case)
    s["codes"][0, at], s["params"][0, at] = k, ks
    s["codes"][1, at], s["params"][1, at] = v, vs


def _read(s, part):
    at = s["slots"].clamp_min(0)
    y = _values(s["codes"][part, at], s["params"][part, at], s["case"])
    return torch.where((s["slots"] >= 0)[:, None, None], y, 0.0).to(TYPES[s["case"]["dtype"]])


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from grammar_constrained_logit_gb300 import ops

    if op == "beam":
        if own:
            return ops.beam_select(s["logits"], s["scores"], s["case"]["n"],
                                   bitmask=s["bitmask"], row_needs_mask=s["needs"],
                                   finished=s["finished"], pad_id=0,
                                   vocab_size=s["case"]["vocab"])
        return _select(s)
    if op == "reorder":
        if own:
            s["mover"].reorder(s["parents"], s["start"], s["stop"])
            return [t for t, _, _ in s["states"]]
        return _reordered(s)
    if op != "read":
        if own:
            ops.cache_write(s["cache"], s["x"], s["slots"])
        else:
            _written(s)
        if op == "write":  # 8 bits: the cache's own buffers, seen as the type that they hold
            return [s["codes"].view(torch.float8_e4m3fn), s["params"]]
    if own:
        back = ops.cache_read(s["cache"], s["slots"], dtype=TYPES[s["case"]["dtype"]])
    else:
        back = [_read(s, 0), _read(s, 1)]
    return [*back, s["params"]] if op == "both" else back


# ------------------------------------------------------------------- the work


def work(case):
    if case["op"] == "beam":
        B, K, V, e = case["batch"], case["beams"], case["vocab"], SIZE[case["dtype"]]
        live = {"all": K, "some": 0.85 * K, "first": 1}[case["alive"]] * (1 - case["finished"])
        # memory is read in sectors of 32 bytes: the share that holds a kept token
        touched, mask = 1.0, 0.0
        if case["keep"] < 1.0:
            touched = 0.1 + 0.9 * (1 - (1 - case["keep"]) ** (32 // e))
            mask = 0.9 * V / 8
        return {"bytes": B * live * (touched * V * e + mask) + B * K * 6 + B * case["n"] * 16,
                "flops": 4.0 * B * live * V * case["keep"]}
    if case["op"] == "reorder":
        H, D = case["heads"], case["dim"]
        token = {"bf16": 2 * D, "q8": D + 4, "q4": D // 2 + D // 16 * 4}[case["kind"]]
        token = 2 * case["layers"] * H * token + 8
        moved = 0
        for parents, start, stop in _pattern(case):
            there = [(p, k) for k, p in enumerate(parents) if p != k]
            moved += (len({p for p, _ in there}) + len(there)) * (stop - start)
        return {"bytes": max(1, moved * token) + case["batch"] * (case["beams"] + 2) * 4,
                "flops": 0}
    n, H, D = case["n"] * (1 - case["padded"]), case["heads"], case["dim"]
    x = H * D * SIZE[case["dtype"]]
    kept = H * (D * case["bits"] // 8 + D // case["group"] * 4)
    out = case["n"] * x  # a padded token's values are written as zeros
    back = {"write": 0, "read": n * kept + out, "both": out}[case["op"]]
    there = 0 if case["op"] == "read" else n * (x + kept)
    return {"bytes": 2 * (back + there) + case["n"] * 8, "flops": 2 * 4.0 * n * H * D}


# ------------------------------------------------------------ in 64 bits, apart


def exact(case, seed):
    if case["op"] == "reorder":
        return None  # moves bytes, computes nothing
    s = prepare(case, seed)
    if case["op"] == "beam":
        B, K, V, n = (case[k] for k in ("batch", "beams", "vocab", "n"))
        if B * K * V > 3e7:
            return None
        x = s["logits"][:, :V].double().cpu().numpy()
        scores = s["scores"].double().cpu().numpy().reshape(-1)
        if s["bitmask"] is not None:
            words = np.ascontiguousarray(s["bitmask"].cpu().numpy()).view(np.uint8)
            bits = np.unpackbits(words, axis=1, bitorder="little")[:, :V]
            x[(bits == 0) & (s["needs"].cpu().numpy() != 0)[:, None]] = NEG
        ended = s["finished"].cpu().numpy() if s["finished"] is not None else np.zeros(B * K)
        out = np.full((B, n), NEG)
        for b in range(B):
            pool = []
            for r in range(b * K, b * K + K):
                if not scores[r] > NEG:
                    continue
                if ended[r]:
                    pool.append(scores[r:r + 1])
                    continue
                row = x[r][x[r] > NEG]
                if row.size:
                    most = row.max()
                    total = math.log(np.exp(row - most).sum()) + most
                    pool.append(scores[r] + np.sort(row)[::-1][:n] - total)
            best = np.sort(np.concatenate(pool))[::-1][:n] if pool else np.zeros(0)
            out[b, :best.size] = best
        return out, None, None
    D, size, bits = case["dim"], case["group"], case["bits"]
    if case["n"] * case["heads"] * D > 2e7:
        return None
    slots = s["slots"].cpu().numpy()
    ok = slots >= 0
    codes = [None, None]
    params = s["params"].double().cpu().numpy()
    if case["op"] == "read":
        held = s["codes"].cpu().numpy()
        for p in range(2):
            c = held[p]
            if bits == 8:
                e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
                y = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
                codes[p] = np.where(c & 128, -y, y)
            else:
                y = np.empty(c.shape[:2] + (D,))
                y[..., 0::2], y[..., 1::2] = c % 16, c // 16
                codes[p] = y
    else:
        total = s["codes"].shape[1]
        one = np.float32(1.0)
        for p in range(2):
            # which code a value gets is defined in 32-bit arithmetic, so that every reader
            # and writer of a cache agrees on it: followed here step by step up to the rounding
            x = s["x"][p].float().cpu().numpy()[ok].reshape(ok.sum(), case["heads"], -1, size)
            codes[p] = np.zeros((total, case["heads"], D))
            if bits == 8:
                scale = np.maximum(np.abs(x).max(-1) * np.float32(1 / 448), np.float32(TINY))
                y = (x * (one / scale)[..., None]).astype(np.float64)
                with np.errstate(divide="ignore"):
                    step = 2.0 ** (np.clip(np.floor(np.log2(np.abs(y))), -6, 8) - 3)
                params[p, slots[ok]] = np.maximum(np.abs(x.astype(np.float64)).max(-1) / 448, TINY)
                y = np.clip(np.rint(y / step) * step, -448, 448)
                codes[p][slots[ok]] = y.reshape(ok.sum(), -1, D)
            else:
                # the pair is held in bf16: its rounding is part of the definition
                def short(a):
                    a = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
                    a = (a + 0x7fff + ((a >> 16) & 1)) & 0xffff0000
                    return a.astype(np.uint32).view(np.float32)

                half = np.float32(0.5)
                scale = (x.max(-1) * half - x.min(-1) * half) * np.float32(1 / 7.5)
                scale, low = short(np.maximum(scale, np.float32(TINY))), short(x.min(-1))
                y = (x - low[..., None]) * (one / scale)[..., None]
                y = np.rint(np.clip(y.astype(np.float64), 0, 15))
                params[p, slots[ok], ..., 0], params[p, slots[ok], ..., 1] = scale, low
                codes[p][slots[ok]] = y.reshape(ok.sum(), -1, D)
        if case["op"] == "write":
            return [np.stack(codes), params]
    back = []
    for p in range(2):
        y = codes[p][slots * ok].reshape(slots.size, case["heads"], -1, size)
        q = params[p][slots * ok]
        y = y * q[..., None] if bits == 8 else q[..., 1:] + y * q[..., :1]
        back.append(np.where(ok[:, None, None], y.reshape(slots.size, -1, D), 0.0))
    return [*back, params] if case["op"] == "both" else back
