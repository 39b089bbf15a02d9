"""Plain 64-bit references of the 8-bit paged cache and of the prompts'
attention, and the error bounds their GPU results are held to."""
import numpy as np

import operator_refs as ref

TOP = 448.0
LEAST = 2.0 ** -100


def rotate(x, r, table, rot, interleaved):
    """x [T, H, hs] turned by the angles at rows r of table [P, rot], in the type
    of both (float64, or float32 with each operation rounded by itself); rows
    outside of it give zeros.  Returns the values and the magnitudes that meet
    in each."""
    y, mag = x.copy(), np.abs(x)
    if rot:
        ok = (r >= 0) & (r < len(table))
        cs = table[np.where(ok, r, 0)][:, None] if len(table) else np.zeros((len(r), 1, rot), x.dtype)
        c, s = cs[..., :rot // 2], cs[..., rot // 2:rot]
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        xa, xb = x[..., a], x[..., b]
        y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
        mag[..., a], mag[..., b] = np.abs(xa * c) + np.abs(xb * s), np.abs(xb * c) + np.abs(xa * s)
        y[~ok], mag[~ok] = 0, 0
    return y, mag


def codes(x):
    """Nearest e4m3 values, ties to even, of float64 x."""
    x = np.clip(x, -TOP, TOP)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 1e-300))), -6) - 3)
    return np.round(x / step) * step


def append(cache, scales, k, v, table, starts, lens, bs):
    """Append k (rotated), v [T, H, hs] to cache float64 [nb, 2, bs, H, hs] of
    e4m3 values and scales [nb, 2, H], in place, in the type of k, v and scales:
    float64, or float32 with the definition's roundings.  Returns bool arrays of the entries and scales written, and of the older entries that
    shrank."""
    nb = len(cache)
    wrote, scaled, shrunk = np.zeros(cache.shape, bool), np.zeros(scales.shape, bool), np.zeros(cache.shape, bool)
    for b in range(len(lens)):
        n, length = int(starts[b + 1] - starts[b]), max(int(lens[b]), 0)
        ctx = length - n
        pos = max(ctx, 0)
        while pos < length:
            page, off = pos // bs, pos % bs
            cnt = min(bs - off, length - pos)
            blk = int(table[b, page]) if page < table.shape[1] else -1
            if 0 <= blk < nb:
                t0 = int(starts[b]) + pos - ctx
                x = np.stack([k[t0:t0 + cnt], v[t0:t0 + cnt]])                      # [2, tokens, H, hs]
                one = x.dtype.type
                need = np.clip(np.abs(x).max((1, 3)) / one(TOP), one(LEAST), one(2.0 ** 120))
                if off:
                    old = np.clip(scales[blk], one(LEAST), one(2.0 ** 121))
                    (ma, ea), (mb, eb) = np.frexp(old), np.frexp(need)
                    times = np.maximum(eb - ea + (mb > ma), 0)
                    need = np.ldexp(old, times)
                    grown = times > 0
                    cache[blk, :, :off] = codes(np.ldexp(cache[blk, :, :off], -times[:, None, :, None]))
                    shrunk[blk, :, :off] |= grown[:, None, :, None]
                    scales[blk] = np.where(grown, need, scales[blk])
                    scaled[blk] |= grown
                else:
                    scales[blk], scaled[blk] = need, True
                inverse = (one(1) / need)[:, None, :, None]
                cache[blk, :, off:off + cnt] = codes((x * inverse).astype(np.float64))
                wrote[blk, :, off:off + cnt] = True
            pos += cnt
    return wrote, scaled, shrunk


def attend(q, k, v, see, scale, rounding, floor):
    """Softmax attention of rows q [n, dk] over keys [m, dk] / values [m, dv]
    with visibility see [n, m]: (out, lse, out_tol, lse_tol) in float64.

    Bounds.  Scores are binary32 sums of dk exact products, so a logit is off
    by at most (dk + 4) 2^-24 times the sum of its products' magnitudes, plus
    2^-22 of its own size and of its distance to the row's maximum (scalings,
    the shift, the value scale's logarithm, exp2's argument).  A weight is off
    by that relatively, by `rounding` (half a step of the type that it is
    multiplied in) and by 2^-22 for exp2; sums of m weights add m 2^-24 each in
    the numerator and the denominator.  Weights below that type's normal range
    are off by at most `floor` of the largest value's size each.  The output is
    rounded to bf16 once: half a step is 2^-8 of its size.
    """
    n, m = see.shape
    out, lse = np.zeros((n, v.shape[1])), np.full(n, -np.inf)
    otol, ltol = np.zeros((n, v.shape[1])), np.zeros(n)
    seen = see.any(0)[:, None]
    kk, vv = np.where(seen, k, 0), np.where(seen, v, 0)
    logit = np.where(see, (q @ kk.T) * scale, -np.inf)
    size = (np.abs(q) @ np.abs(kk).T) * abs(scale)
    for i in range(n):
        s = see[i]
        if not s.any():
            continue
        x = logit[i, s]
        top = x.max()
        p = np.exp(x - top)
        tot = p.sum()
        lse[i] = top + np.log(tot)
        vals = vv[s]
        out[i] = p @ vals / tot
        eps = (q.shape[1] + 4) * 2.0 ** -24 * size[i, s] + 2.0 ** -22 * (np.abs(x) + 2 * (top - x) + 32)
        mean = (p * eps).sum() / tot
        mag = (p[:, None] * np.abs(vals)).sum(0) / tot
        rel = (p[:, None] * np.abs(vals) * (eps[:, None] + rounding)).sum(0) / tot
        wide = (s.sum() + 64) * 2.0 ** -23
        otol[i] = (2.0 ** -8 * np.abs(out[i]) + rel + (mean + wide) * (mag + np.abs(out[i]))
                   + s.sum() * floor) * 1.01 + 1e-30
        ltol[i] = mean + wide + 2.0 ** -22 * (abs(lse[i]) + abs(top) + 16)
    return out, lse, otol, ltol


causal, tree, bf16, e4m3 = ref.causal, ref.tree, ref.bf16, ref.e4m3
