"""Plain 64-bit definitions of the beam-search operators, on the CPU, for their tests."""
import numpy as np


def beam_candidates(x, scores, *, allowed=None, finished=None, pad=0):
    """Candidates of one batch entry, best first: a list of (score, beam, token).
    x float64 [beams, V]; scores [beams]; allowed bool [beams, V] or None."""
    out = []
    for k in range(x.shape[0]):
        s = float(scores[k])
        if not s > -np.inf:
            continue
        if finished is not None and finished[k]:
            out.append((s, k, -1))
            continue
        ok = x[k] > -np.inf  # false for NaN
        if allowed is not None:
            ok &= allowed[k]
        v = np.flatnonzero(ok)
        if v.size == 0:
            continue
        m = x[k, v].max()
        if m == np.inf:
            v = v[x[k, v] == np.inf]
            lp = np.full(v.size, -np.log(float(v.size)))
        else:
            d = x[k, v] - m
            lp = d - np.log(np.exp(d).sum())
        out += [(s + lp[i], k, int(v[i])) for i in np.argsort(-lp, kind="stable")
                if s + lp[i] > -np.inf]
    out.sort(key=lambda c: (-c[0], c[1], c[2]))
    return [(s, k, pad if t < 0 else t) for s, k, t in out]


def check_beam(got, x, scores, n, *, allowed=None, finished=None, pad=0, tol=None):
    """Compares a selection with the definition.  Scores agree within

        2^-24 |score|  (one rounding to 32 bits)  +  4e-6  (the error of log S)

    where log S's bound adds, relative to S: 2^-22 of an exponential by the hardware's
    approximation, 2^-23 sum_i p_i t_i <= 2^-23 ln V of its argument's two roundings
    (below 1.5e-6 for V < 2^18), 20 additions of 2^-24 (1.2e-6) and the join's 2^-23.
    Where neighbours in the true order are further apart than twice that, beam and token
    are the definition's; nearer ones may trade places, unless they are of one beam."""
    gs, gt, gp = (np.asarray(a) for a in got)
    batch, beams = scores.shape
    for b in range(batch):
        r = slice(b * beams, (b + 1) * beams)
        want = beam_candidates(x[r], scores[b], pad=pad,
                               allowed=None if allowed is None else allowed[r],
                               finished=None if finished is None else finished[b])
        true = {(k, t): s for s, k, t in want}
        m = min(n, len(want))
        assert (gt[b, m:] == -1).all() and (gp[b, m:] == -1).all()
        assert np.isneginf(gs[b, m:]).all()
        picked = [(int(gp[b, i]), int(gt[b, i])) for i in range(m)]
        assert len(set(picked)) == m, "a candidate twice"
        for i in range(m):
            s = want[i][0]
            off = (2.0 ** -24 * abs(s) + 4e-6) if np.isfinite(s) else 0.0
            assert picked[i] in true, (b, i, picked[i])
            assert gs[b, i] == s or abs(float(gs[b, i]) - s) <= off, (b, i, gs[b, i], s)
            if picked[i] != want[i][1:]:
                # only a neighbour within the rounding may stand here, and of another beam
                assert abs(true[picked[i]] - s) <= 2 * off, (b, i, picked[i], want[i])
        for k in set(p for p, _ in picked):  # one beam's candidates keep their exact order
            mine = [t for p, t in picked if p == k]
            assert mine == [t for _, p, t in want if p == k][:len(mine)], (b, k)


def reordered(rows, parents, start=None, stop=None):
    """rows [batch * beams, tokens, ...] after a reorder."""
    batch, beams = parents.shape
    out = rows.copy()
    T = rows.shape[1]
    for b in range(batch):
        lo = 0 if start is None else min(max(int(start[b]), 0), T)
        hi = T if stop is None else min(max(int(stop[b]), 0), T)
        for k in range(beams):
            p = int(parents[b, k])
            if 0 <= p < beams and lo < hi:
                out[b * beams + k, lo:hi] = rows[b * beams + p, lo:hi]
    return out


LARGEST, TINY = np.float32(3.3895313892515355e38), np.float32(2.0 ** -126)


def to_bf16(x):
    """float32 -> the nearest bf16, as float32 (finite values)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000).astype(np.uint32).view(np.float32)


def e4m3_values():
    """What the 256 codes stand for."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


def quantised(x, bits, group):
    """x float32 [..., dim] -> (the value of each code before scaling, scale, low), the
    definition's 32-bit steps; scale and low [..., groups]."""
    x = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, group)
    fine = np.abs(x) <= LARGEST
    with np.errstate(all="ignore"):
        if bits == 8:
            scale = np.maximum(np.where(fine, np.abs(x), 0).max(-1) * np.float32(1 / 448), TINY)
            y = x * (np.float32(1) / scale)[..., None]
            grid = np.sort(e4m3_values()[:127])  # 0 .. 448
            a = np.minimum(np.abs(y), np.float32(448)).astype(np.float64)
            i = np.clip(np.searchsorted(grid, a), 1, 126)
            lo, hi = grid[i - 1], grid[i]
            up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))  # ties: an even code
            code = np.copysign(np.where(up, hi, lo), y)
            code[np.isnan(y)] = np.nan
            return code, scale, np.zeros_like(scale)
        lo = np.where(fine, x, np.inf).min(-1)
        hi = np.where(fine, x, -np.inf).max(-1)
        none = ~(lo <= hi)
        lo, hi = np.where(none, 0, lo).astype(np.float32), np.where(none, 0, hi).astype(np.float32)
        half = np.float32(0.5)
        scale = to_bf16(np.maximum((hi * half - lo * half) * np.float32(1 / 7.5), TINY))
        low = to_bf16(lo)
        y = (x - low[..., None]) * (np.float32(1) / scale)[..., None]
        code = np.rint(np.clip(y, 0, 15)).astype(np.float64)
        code[np.isnan(y)] = 0
        return code, scale, low


def held_values(code, scale, low, bits):
    """The float32 values that codes stand for, [..., dim]: rounded once."""
    s, m = scale.astype(np.float64)[..., None], low.astype(np.float64)[..., None]
    v = (code * s if bits == 8 else m + code * s).astype(np.float32)
    return v.reshape(*v.shape[:-2], -1)
