"""Plain 64-bit definitions of attention over the cache, eviction and verification of drafts,
on the CPU, for their tests."""
import numpy as np

from beam_oracle import e4m3_values

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
# what a weight is rounded to before it meets a value: 11 bits for bf16, 22 for the others
WEIGHT = {"f32": 2.0 ** -22, "f16": 2.0 ** -22, "bf16": 2.0 ** -11}


def values(codes, params, bits, group):
    """codes uint8 [..., bytes], params [..., groups(, 2)] -> float64 [..., dim]."""
    if bits == 8:
        v = e4m3_values()[codes]
        v = v.reshape(*v.shape[:-1], -1, group) * params.astype(np.float64)[..., None]
    else:
        v = np.stack((codes & 15, codes >> 4), -1).astype(np.float64)
        v = v.reshape(*codes.shape[:-1], -1, group)
        p = params.astype(np.float64)
        v = p[..., 1:] + v * p[..., :1]
    return v.reshape(*v.shape[:-2], -1)


def held(cache):
    """The cache's values, float64 [parts, slots, heads, dim]."""
    codes, params = cache.codes, cache.params
    if codes.dim() == 5:
        codes, params = codes.flatten(1, 2), params.flatten(1, 2)
    return values(codes.cpu().numpy(), params.float().cpu().numpy(), cache.bits, cache.group)


def reach(cache):
    """What a weight's rounding is multiplied by, at most: |code * scale| of the values.  In 4
    bits that is the value less its group's low, which comes to it unrounded: the weight of a
    token is rounded where it meets the code, p s c, so it is off by its rounding times s c,
    however near the value l + s c is to zero."""
    v = held(cache)[1]
    if cache.bits == 8:
        return np.abs(v)
    p = cache.params if cache.codes.dim() == 4 else cache.params.flatten(1, 2)
    low = p[1, ..., 1].double().cpu().numpy()
    return np.abs(v - np.repeat(low, cache.group, -1))


def slots_of(blocks, b, n, size, total):
    """Slots of a sequence's n tokens; -1 outside the cache."""
    t = np.arange(n)
    s = blocks[b].astype(np.int64)[t // size] * size + t % size if n else np.zeros(0, np.int64)
    return np.where((s >= 0) & (s < total), s, -1)


def attended(kv, q, blocks, lengths, size, *, n_rows=None, scale=None, window=None, dtype="f32",
             reach=None):
    """(out, how far it may be off, weights [batch, heads, tokens], how far those may be).

    An element of the output is sum_t p_t v_t.  With d the error of a score, a weight's
    relative error is below 2 d (its own and the sum's); it is rounded where it meets the
    value's code (`reach`); the sums over n tokens, of codes' parts and of lows' parts, add n
    roundings of 2^-24; and the result is rounded once.  A score is a sum of dim
    products in 32 bits, of which tensor cores cut off bits (2^-23 a step, at most), a product
    with the scale and one with its group's params; an exponential is off by 2^-21.  A
    weight that is small beside the row's largest product of weight and scale is rounded to
    1.5 * 2^-39 of that (2^-32 for 16-bit queries, whose largest product is held at 2^8 to
    2^15), times codes up to 448; a scale below 2^-60, as of a value of zeros, counts as
    2^-60 there."""
    batch, rows, q_heads, dim = q.shape
    slots, heads = kv.shape[1], kv.shape[2]
    shared = q_heads // heads
    scale = dim ** -0.5 if scale is None else scale
    most = blocks.shape[1] * size
    out, off = np.zeros(q.shape), np.zeros(q.shape)
    weights, woff = np.zeros((batch, heads, most)), np.zeros((batch, heads, most))
    for b in range(batch):
        L = min(max(int(lengths[b]), 0), most)
        n = rows if n_rows is None else min(max(int(n_rows[b]), 0), rows)
        at = slots_of(blocks, b, L, size, slots)
        for r in range(n):
            end = max(0, L - (n - 1 - r))
            lo = max(0, end - window) if window else 0
            t = np.arange(lo, end)
            t = t[at[lo:end] >= 0]
            if t.size == 0:
                continue
            for j in range(q_heads):
                h = j // shared
                k, v = kv[0, at[t], h], kv[1, at[t], h]
                x = (k * q[b, r, j]).sum(-1) * scale
                most_x = (np.abs(k) * np.abs(q[b, r, j])).sum(-1) * abs(scale)
                with np.errstate(invalid="ignore"):
                    p = np.exp(x - x.max())
                p /= p.sum()
                d = (dim + 8) * 2.0 ** -23 * most_x.max() + 2.0 ** -21
                out[b, r, j] = p @ v
                mass = p @ np.abs(v)
                far = mass if reach is None else p @ reach[at[t], h]
                small = t.size * 448 * (2.0 ** -38 if dtype == "f32" else 2.0 ** -32) * \
                    max(np.nanmax(p[:, None] * np.abs(v)), p.max() * 2.0 ** -60)
                rel = 2 * d + (t.size + 64) * 2.0 ** -24
                off[b, r, j] = rel * (mass + far) + WEIGHT[dtype] * far + small + \
                    HALF_STEP[dtype] * np.abs(out[b, r, j])
                weights[b, h, t] += p
                woff[b, h, t] += p * (2 * d + (t.size + 64) * 2.0 ** -24) + 2.0 ** -149
    return out, off, weights, woff


def evicted(n, weights, keep, first, recent):
    """The places that a head of n tokens keeps, in order."""
    if n <= keep:
        return np.arange(n)
    lo, hi = first, n - recent
    w = weights[lo:hi].astype(np.float64)
    # NaN is the least; ties go to the lowest place
    order = sorted(range(lo, hi), key=lambda t: (np.isnan(w[t - lo]),
                                                 -w[t - lo] if w[t - lo] == w[t - lo] else 0, t))
    kept = list(range(lo)) + order[:keep - first - recent] + list(range(hi, n))
    return np.array(sorted(kept), np.int64)


def row_probs(x, allowed, temperature):
    """Target probabilities of one row, float64; all zeros without a candidate."""
    ok = (x > -np.inf) & allowed
    p = np.zeros(x.size)
    if not ok.any():
        return p
    top = x[ok].max()
    if not temperature > 0:
        p[np.flatnonzero(ok & (x == top))[0]] = 1.0
        return p
    with np.errstate(invalid="ignore"):
        d = np.where(x == top, 0.0, x - top) / temperature
    p[ok] = np.exp(d[ok])
    return p / p.sum()


def verified(x, allowed, drafts, probs, uniforms, temperature, noise):
    """One slot: (tokens, accepted, margin): x float64 [rows, V]; noise(row) its Gumbel noise.
    margin: how far the nearest decision was from going the other way, relative."""
    R, V = x.shape
    margin, n, refused = np.inf, 0, False
    for i in range(R - 1):
        v = int(drafts[i])
        if not 0 <= v < V:
            break
        p = row_probs(x[i], allowed[i], temperature)[v]
        a = float(uniforms[i]) * (1.0 if probs is None else float(probs[i, v]))
        if p > 0 or a > 0:
            margin = min(margin, abs(p - a) / max(p, a))
        if not a < p:
            refused = True
            break
        n += 1
    p = row_probs(x[n], allowed[n], temperature)
    r = p
    if refused:
        q = np.zeros(V)
        if probs is None:
            q[int(drafts[n])] = 1.0
        else:
            q = probs[n, :V].astype(np.float64)
        r = np.where(p - q > 0, p - q, 0.0)  # NaN counts as 0
        if not (r > 0).any():
            r, margin = p, 0.0 if (p > 0).any() and temperature > 0 else margin
        # rounded to 32 bits, p - q may be this far off, relative to itself
        if (r > 0).any():
            margin = min(margin, 1.0)
    token = -1
    if (r > 0).any():
        if not temperature > 0:
            token = int(np.argmax(p))
        else:
            with np.errstate(divide="ignore"):
                score = np.log(r) + noise(n)
            order = np.argsort(-score, kind="stable")
            token = int(order[0])
            if order.size > 1 and score[order[1]] > -np.inf:
                margin = min(margin, score[token] - score[order[1]])
    out = np.full(R, -1, np.int64)
    out[:n] = drafts[:n]
    out[n] = token
    return out, n, margin
