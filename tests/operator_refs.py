"""Plain 64-bit references of the operators around the cache, on the CPU, and
the error bounds their GPU results are held to."""
import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e4m3(b):
    """e4m3 bytes -> float64 (NaN codes give NaN)."""
    b = np.asarray(b, np.uint8).astype(np.int64)
    e, m = b >> 3 & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def codes(data):
    """Packed e2m1 bytes [..., n] -> float64 [..., 2n]."""
    data = np.asarray(data)
    return E2M1[np.stack([data & 15, data >> 4], -1).reshape(*data.shape[:-1], -1)]


def nvfp4(data, scale):
    """Codes and block scales -> float64; a NaN scale counts as 0, as the
    attention operators define."""
    return codes(data) * np.repeat(np.nan_to_num(e4m3(scale), nan=0.0), 16, -1)


def kv_rows(cache, layout, blk, off, head, hs):
    """(k, v) float64 [hs] of one cache entry; cache: flat bytes."""
    out = []
    for side in (0, 1):
        base = blk * layout.block_stride + side * layout.side_stride
        d = base + layout.data_offset + off * layout.data_token_stride + head * layout.data_head_stride
        s = base + layout.scale_offset + off * layout.scale_token_stride + head * layout.scale_head_stride
        out.append(nvfp4(cache[d:d + hs // 2], cache[s:s + hs // 16]))
    return out


def kv_positions(cache, layout, table_row, n, bs, num_blocks, head, hs):
    """k, v [n, hs] of a request's positions and which of them exist."""
    k, v, ok = np.zeros((n, hs)), np.zeros((n, hs)), np.zeros(n, bool)
    for p in range(n):
        if p // bs >= len(table_row):
            continue
        blk = int(table_row[p // bs])
        if 0 <= blk < num_blocks:
            ok[p] = True
            k[p], v[p] = kv_rows(cache, layout, blk, p % bs, head, hs)
    return k, v, ok


def mla_positions(cache, table_row, n, bs, num_blocks, bstr, estr):
    """(keys [n, 576], values [n, 512], exists) of nvfp4_ds_mla entries."""
    k, ok = np.zeros((n, 576)), np.zeros(n, bool)
    for p in range(n):
        if p // bs >= len(table_row):
            continue
        blk = int(table_row[p // bs])
        if 0 <= blk < num_blocks:
            ok[p] = True
            e = cache[blk * bstr + p % bs * estr:][:352]
            k[p, :512] = nvfp4(e[:256], e[320:352])
            k[p, 512:] = e4m3(e[256:320])
    return k, k[:, :512].copy(), ok


def attend(q, k, v, see, scale, gk=1.0, gv=1.0):
    """Softmax attention of rows q [n, dk] over keys [m, dk] / values [m, dv]
    with visibility see [n, m]: (out, lse, out_tol, lse_tol) in float64.

    Bounds.  Scores are binary32 sums of dk exact products, so a logit is off
    by at most (dk + 4) 2^-24 times the sum of its products' magnitudes, plus
    2^-22 of its own size and of its distance to the row's maximum (two scalings, the shift,
    exp2's argument).  A weight is off by that relatively, by 2^-11 for its
    rounding to binary16 and by 2^-22 for exp2; sums of m weights add m 2^-24
    each in the numerator and the denominator.  Weights below binary16's
    normal range (2^-20 of the maximum) are off by 2^-25 / 2^6 of it at most.
    The output is rounded to bf16 once: half a step is 2^-8 of its size.
    """
    n, m = see.shape
    out, lse = np.zeros((n, v.shape[1])), np.full(n, -np.inf)
    otol, ltol = np.zeros((n, v.shape[1])), np.zeros(n)
    with np.errstate(all="ignore"):
        logit = np.where(see, (q @ np.where(see.any(0)[:, None], k, 0).T) * scale * gk, -np.inf)
        size = (np.abs(q) @ np.abs(np.where(see.any(0)[:, None], k, 0)).T) * abs(scale * gk)
    for i in range(n):
        s = see[i]
        if not s.any():
            continue
        x = logit[i, s]
        top = x.max()
        p = np.exp(x - top)
        tot = p.sum()
        lse[i] = top + np.log(tot)
        vals = v[s] * gv
        out[i] = p @ vals / tot
        eps = (q.shape[1] + 4) * 2.0 ** -24 * size[i, s] + 2.0 ** -22 * (np.abs(x) + 2 * (top - x) + 16)
        mean = (p * eps).sum() / tot
        mag = (p[:, None] * np.abs(vals)).sum(0) / tot
        rel = (p[:, None] * np.abs(vals) * (eps[:, None] + 2.0 ** -11)).sum(0) / tot
        wide = (s.sum() + 64) * 2.0 ** -23
        otol[i] = (2.0 ** -8 * np.abs(out[i]) + rel + (mean + wide) * (mag + np.abs(out[i]))
                   + s.sum() * 2.0 ** -31 * np.abs(vals).max()) * 1.01 + 1e-30
        ltol[i] = mean + wide + 2.0 ** -22 * (abs(lse[i]) + abs(top) + 16)
    return out, lse, otol, ltol


def causal(n, length, window=None, sinks=0):
    """Visibility [n, length] of the last n positions of a sequence."""
    i = np.arange(length - n, length)[:, None]
    j = np.arange(length)[None]
    see = (j <= i) & (i >= 0)
    if window is not None:
        see &= (j < sinks) | (i - j < window)
    return see


def tree(n, length, mask):
    """Visibility of n drafted tokens; mask bool [n, columns]."""
    see = np.zeros((n, max(length, 0)), bool)
    ctx = length - n
    for i in range(n):
        if ctx + i < 0:
            continue
        for j in range(length):
            d = j - ctx
            see[i, j] = d < 0 or (d < mask.shape[1] and bool(mask[i, d]))
    return see


def norm_rope(x, w, positions, cos_sin, rot, eps, interleaved):
    """float64 norm and rotation of x [T, H, hs], and a bound of the error of
    a binary32 computation rounded to bf16: 2^-8 of the value, and 2^-20 of
    the magnitudes that meet in it (sum of squares, square root, division,
    three products and a sum: well below 16 roundings of 2^-24)."""
    x = x.astype(np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    mag = np.abs(y)
    if rot:
        ok = (positions >= 0) & (positions < len(cos_sin))
        cs = cos_sin[np.where(ok, positions, 0)][:, None].astype(np.float64)
        c, s = cs[..., :rot // 2], cs[..., rot // 2:rot]
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
        mag[..., a] = np.abs(ya * c) + np.abs(yb * s)
        mag[..., b] = np.abs(yb * c) + np.abs(ya * s)
        y[~ok], mag[~ok] = 0, 0
    return y, 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * mag + 1e-37


# ---------------------------------------------------------------------------
# page bookkeeping, the definitions step by step
# ---------------------------------------------------------------------------
def pages(n, bs):
    return -(-n // bs) if n > 0 else 0


def _grant(valid_need, refs):
    """Requests [(valid, need)] in order -> (granted, page lists)."""
    free = [int(i) for i in np.nonzero(refs == 0)[0]]
    upto, got = 0, []
    for valid, need in valid_need:
        if not valid:
            got.append(None)
            continue
        got.append(free[upto:upto + need] if upto + need <= len(free) else None)
        upto += need
    return got


def fork(table, lens, refs, parents, children, bs, caches):
    before = lens.copy()
    seen, asks = set(), []
    for p, c in zip(parents, children):
        ok = 0 <= p < len(lens) and 0 <= c < len(lens) and p != c and before[c] == 0 and before[p] >= 0 \
            and pages(int(before[p]), bs) <= table.shape[1] and c not in seen
        if ok:
            seen.add(c)
        asks.append((ok, int(ok and before[p] % bs != 0)))
    got = _grant(asks, refs)
    status = np.zeros(len(asks), np.int32)
    olds = table.copy()
    for i, (p, c) in enumerate(zip(parents, children)):
        if got[i] is None:
            continue
        status[i] = 1
        full = int(before[p]) // bs
        for j in range(full):
            table[c, j] = olds[p, j]
            if 0 <= olds[p, j] < len(refs):
                refs[olds[p, j]] += 1
        if got[i]:
            table[c, full] = got[i][0]
            refs[got[i][0]] += 1
            if 0 <= olds[p, full] < len(refs):
                for cache in caches:
                    cache[got[i][0]] = cache[olds[p, full]]
        lens[c] = before[p]
    return status


def extend(table, lens, refs, rows, new, bs):
    seen, asks = set(), []
    for r, n in zip(rows, new):
        ok = 0 <= r < len(lens) and 0 <= lens[r] <= n and pages(int(n), bs) <= table.shape[1] and r not in seen
        if ok:
            seen.add(r)
        asks.append((ok, pages(int(n), bs) - pages(int(lens[r]), bs) if ok else 0))
    got = _grant(asks, refs)
    status = np.zeros(len(asks), np.int32)
    for i, (r, n) in enumerate(zip(rows, new)):
        if got[i] is None:
            continue
        status[i] = 1
        have = pages(int(lens[r]), bs)
        for j, page in enumerate(got[i]):
            table[r, have + j] = page
            refs[page] += 1
        lens[r] = n
    return status


def free(table, lens, refs, rows, bs):
    for r in rows:
        if not 0 <= r < len(lens):
            continue
        for j in range(min(pages(int(lens[r]), bs), table.shape[1])):
            page = table[r, j]
            if 0 <= page < len(refs) and refs[page] > 0:
                refs[page] -= 1
            table[r, j] = -1
        lens[r] = 0


def compact(table, lens, refs, bs, caches):
    live = refs > 0
    n = int(live.sum())
    holes = [i for i in range(n) if not live[i]]
    movers = [i for i in range(len(refs) - 1, n - 1, -1) if live[i]]
    page_map = np.where(live, np.arange(len(refs)), -1).astype(np.int32)
    for h, m in zip(holes, movers):
        page_map[m] = h
        refs[h], refs[m] = refs[m], 0
        for cache in caches:
            cache[h] = cache[m]
    for r in range(len(lens)):
        for j in range(min(pages(int(lens[r]), bs), table.shape[1])):
            if 0 <= table[r, j] < len(refs):
                table[r, j] = page_map[table[r, j]]
    return page_map


def bf16(a):
    """float array -> (bf16 torch tensor, its exact float64 values)."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t, t.to(torch.float64).numpy()
