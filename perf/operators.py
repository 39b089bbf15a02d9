"""Cases and plain forms of the attention, rotation and page operators around the
quantized paged KV cache.

A case names an operator (`op`) and its sizes; sequence lengths of a batch are
drawn from the case's own `lens` number, contents from the seed.  With `own`
False, `run` computes the operator with elementary torch operations in 32
bits, rounded once at the end; with `own` True it calls this repository's
package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decoded token: launch latency is what counts
        dict(name="qk_one_token", op="qk", tokens=1, heads=32, kv_heads=8, hs=128, rot=128, interleaved=False),
        # a prefill chunk's queries and keys
        dict(name="qk_prefill", op="qk", tokens=16384, heads=32, kv_heads=8, hs=128, rot=128, interleaved=False),
        # one user decoding behind a short window
        dict(name="window_one_token", op="window", batch=1, qmax=1, lmin=1037, lmax=1037, heads=32, kv_heads=8,
             hs=128, block=16, window=512, sinks=4, lens=1),
        # a decode batch with contexts of 1 Ki to 32 Ki tokens behind a 4 Ki window
        dict(name="window_decode", op="window", batch=64, qmax=1, lmin=1024, lmax=32768, heads=32, kv_heads=8,
             hs=128, block=16, window=4096, sinks=4, lens=2),
        # ragged prefill chunks over cached contexts
        dict(name="window_prefill", op="window", batch=3, qmax=4096, lmin=4096, lmax=8192, heads=32, kv_heads=8,
             hs=128, block=16, window=2048, sinks=4, lens=3),
        # eight drafted tokens of one user
        dict(name="tree_one_request", op="tree", batch=1, qmax=8, lmin=1021, lmax=1021, heads=32, kv_heads=8,
             hs=128, block=16, lens=4),
        # up to 64 drafted tokens for each of 16 requests
        dict(name="tree_batch", op="tree", batch=16, qmax=64, lmin=2048, lmax=16384, heads=32, kv_heads=8,
             hs=128, block=16, lens=5),
        # one decoded token over the 352-byte latent cache
        dict(name="mla_one_token", op="mla", batch=1, qmax=1, lmin=4096, lmax=4096, heads=16, block=64, lens=6),
        # up to 32 drafted tokens for each of 16 requests over the latent cache
        dict(name="mla_tree_batch", op="mla", batch=16, qmax=32, lmin=2048, lmax=16384, heads=16, block=64, lens=7),
        # four beams from one prompt, 32 layers
        dict(name="fork_beams", op="fork", caches=32, parents=1, children=4, blocks=256, page=18432, block=16,
             lmin=100, lmax=1000, lens=8),
        # 64 prompts with eight samples each, 32 layers of the latent cache
        dict(name="fork_batch", op="fork", caches=32, parents=64, children=8, blocks=2048, page=22528, block=64,
             lmin=64, lmax=1500, lens=9),
        # half of the requests end; the pages of the others move together
        dict(name="compact_pages", op="compact", caches=16, rows=128, blocks=8192, page=22528, block=64, lmin=512,
             lmax=6000, lens=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "window", "window", "tree", "mla", "fork", "compact"])
    lens = rng.randrange(1 << 30)
    if op == "qk":
        hs = rng.choice([64, 80, 96, 128, 192, 256])
        kv = rng.choice([1, 2, 4, 8])
        return dict(op=op, tokens=_log(rng, 1, 8000), heads=kv * rng.choice([1, 2, 3, 4]), kv_heads=kv, hs=hs,
                    rot=rng.choice([hs, hs // 2 // 16 * 16]), interleaved=rng.random() < 0.4)
    if op == "fork":
        return dict(op=op, caches=rng.randint(1, 32), parents=_log(rng, 1, 40), children=rng.randint(1, 8),
                    blocks=rng.randint(1000, 2000), page=rng.choice([18432, 22528, 41984, 5640]),
                    block=rng.choice([16, 48, 64]), lmin=1, lmax=384, lens=lens)
    if op == "compact":
        return dict(op=op, caches=rng.randint(1, 16), rows=_log(rng, 4, 100), blocks=rng.randint(5000, 8000),
                    page=rng.choice([18432, 22528, 5640]), block=rng.choice([64, 80]), lmin=1, lmax=4000, lens=lens)
    lmax = _log(rng, 40, 8000)
    lmin = max(1, lmax // rng.randint(1, 8))
    if op == "mla":
        return dict(op=op, batch=_log(rng, 1, 16), qmax=_log(rng, 1, 24), lmin=lmin, lmax=lmax,
                    heads=rng.choice([8, 16, 16, 20, 32]), block=rng.choice([16, 48, 64]), lens=lens)
    kv = rng.choice([1, 2, 4, 8])
    case = dict(op=op, batch=_log(rng, 1, 16), qmax=_log(rng, 1, 48), lmin=lmin, lmax=lmax,
                heads=kv * rng.choice([1, 2, 3, 4, 8]), kv_heads=kv, hs=rng.choice([64, 80, 96, 128, 256]),
                block=rng.choice([16, 16, 24, 64]), lens=lens)
    if op == "window":
        case.update(window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 7, 40]))
        if rng.random() < 0.4:                          # a prefill chunk
            case.update(batch=rng.randint(1, 3), qmax=_log(rng, 100, 2000))
    while work(case)["flops"] > 3e11:                   # no dearer than the listed ones
        case["qmax"] = (case["qmax"] + 1) // 2
    return case


def _lengths(case):
    """(query lengths, total key lengths) of a batch: the first request has the
    longest query, the others any."""
    r = random.Random(case["lens"])
    q = [case["qmax"]] + [r.randint((case["qmax"] + 1) // 2, case["qmax"]) for _ in range(case["batch"] - 1)]
    return q, [r.randint(case["lmin"], case["lmax"]) + n for n in q]


def _row_lengths(case):
    """Tokens of each request that owns pages; each keeps to its share of them."""
    r = random.Random(case["lens"])
    n = case["parents"] if case["op"] == "fork" else case["rows"]
    share = (case["blocks"] - (n * case["children"] if case["op"] == "fork" else 0)) // n
    return [min(r.randint(case["lmin"], case["lmax"]), share * case["block"]) for _ in range(n)]


def _sum_min(lo, hi, w):
    """Sum of min(x, w) over lo <= x < hi."""
    m = min(max(w, lo), hi)
    return (m - lo) * (lo + m - 1) // 2 + (hi - m) * w


def _mask_pairs(case):
    """Visible (query, key) pairs of one head, the keys that any query of a
    request sees, and the queries."""
    q, l = _lengths(case)
    if case["op"] == "window":
        w, s = case["window"], case["sinks"]
        pairs = sum(_sum_min(t - n + 1, t + 1, w + s) for n, t in zip(q, l))
        return pairs, sum(min(t, w + n - 1 + s) for n, t in zip(q, l)), sum(q)
    return sum(n * (t - n) + n * (1 + n // 7) for n, t in zip(q, l)), sum(l), sum(q)


def work(case):
    op = case["op"]
    if op == "qk":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["hs"]
        return dict(bytes=4 * n + 4 * case["tokens"] * case["rot"], flops=8 * n)
    if op == "fork":
        lens = _row_lengths(case)
        n = sum(t % case["block"] != 0 for t in lens) * case["children"]
        rd = sum(t % case["block"] != 0 for t in lens)
        pages = sum(-(-t // case["block"]) for t in lens)
        return dict(bytes=case["caches"] * case["page"] * (n + rd) + 4 * pages * (1 + case["children"]), flops=0)
    if op == "compact":
        pages = sum(-(-t // case["block"]) for t in _row_lengths(case)[::2])
        moved = pages - pages * pages // case["blocks"]
        return dict(bytes=2 * moved * case["caches"] * case["page"] + 16 * case["blocks"], flops=0)
    pairs, keys, t = _mask_pairs(case)
    if op == "mla":
        return dict(bytes=352 * keys + 2 * t * case["heads"] * (576 + 512), flops=2 * 1088 * pairs * case["heads"])
    return dict(bytes=keys * case["kv_heads"] * case["hs"] * 9 // 8 + 4 * t * case["heads"] * case["hs"],
                flops=4 * case["hs"] * pairs * case["heads"])


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _fp4_pool(g, n=1 << 16):
    """Bytes of 2 codes and block scales as the quantizer makes them of
    normally distributed values."""
    x = torch.randn(n, 16, generator=g, device=DEV)
    sf = (x.abs().amax(1) / 6).to(torch.float8_e4m3fn)
    y = x / sf.float()[:, None]
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.bucketize(y.abs(), mid) + 8 * (y < 0)
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8).reshape(-1), sf.view(torch.uint8)


def _pick(pool, shape, g):
    return pool[torch.randint(0, pool.numel(), shape, generator=g, device=DEV, dtype=torch.int32)]


def _paged(case, seed):
    """Block table over shuffled pages, starts and lengths of a batch."""
    q, l = _lengths(case)
    bs = case["block"]
    pages = torch.tensor([-(-t // bs) for t in l])
    nb = int(pages.sum()) + 3
    starts = torch.tensor([0] + q).cumsum(0)
    return dict(block_table=_table(pages, nb, seed).to(DEV), query_starts=starts.int().to(DEV), seq_lens=_i32(l),
                blocks=nb, tokens=sum(q), max_query_len=max(q), max_seq_len=max(l))


def _table(pages, blocks, seed):
    """int32 table of rows that own pages[i] of the shuffled blocks, -1 behind them."""
    order = torch.randperm(blocks, generator=torch.Generator().manual_seed(seed)).int()
    owned = torch.arange(int(pages.max()) + 1)[None] < pages[:, None]
    table = torch.full(owned.shape, -1, dtype=torch.int32)
    table[owned] = order[:int(pages.sum())]
    return table


def _tree(case, seed, tokens):
    """bool [tokens, qmax]: every drafted token sees itself and its ancestors.
    A token's parent is one of the six before it, or the context."""
    n = case["qmax"]
    i = torch.arange(n)
    low = (i - 6).clamp(min=-1)
    r = torch.rand(case["batch"], n, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
    parent = low + (r * (i - low)).long()
    step = torch.zeros(case["batch"], n, n + 1, dtype=torch.float64).scatter_(2, parent[..., None] + 1, 1.0)[..., 1:]
    one = torch.eye(n, dtype=torch.float64)
    seen = torch.linalg.solve_triangular(one - step, one.expand_as(step), upper=False) > 0.5    # I + P + P^2 + ...
    q = torch.tensor(_lengths(case)[0])
    return (seen & (i < q[:, None, None]))[i < q[:, None]].reshape(tokens, n).to(DEV)


def _rows(case, seed):
    """Requests that own shuffled pages: table, lengths and reference counts."""
    lens = _row_lengths(case)
    pages = torch.tensor([-(-t // case["block"]) for t in lens] + [0] * (
        case["parents"] * case["children"] if case["op"] == "fork" else 0))
    table = _table(pages, case["blocks"], seed)
    refs = torch.zeros(case["blocks"] + 1, dtype=torch.int32)
    refs[table.long().flatten()] = 1                                # -1 falls on the place behind the last
    return dict(block_table=table.to(DEV), seq_lens=_i32(lens + [0] * (len(pages) - len(lens))),
                ref_counts=refs[:-1].contiguous().to(DEV))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(op=op, case=case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)

    if op == "qk":
        hs, rot = case["hs"], case["rot"]
        qkv = normal(case["tokens"], case["heads"] + 2 * case["kv_heads"], hs)     # one fused projection's output
        s["q"], s["k"] = qkv[:, :case["heads"]], qkv[:, case["heads"]:case["heads"] + case["kv_heads"]]
        s["q_weight"] = (1 + 0.1 * torch.randn(hs, generator=g, device=DEV)).to(torch.bfloat16)
        s["k_weight"] = (1 + 0.1 * torch.randn(hs, generator=g, device=DEV)).to(torch.bfloat16)
        inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        ang = torch.arange(32768, dtype=torch.float64, device=DEV)[:, None] * inv
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        s["positions"] = torch.randint(0, 32768, (case["tokens"],), generator=g, device=DEV)
        return s
    if op in ("fork", "compact"):
        s.update(_rows(case, seed))
        cache = torch.randint(0, 256, (case["caches"], case["blocks"], case["page"]), generator=g, device=DEV,
                              dtype=torch.uint8)
        s["cache"], s["caches"] = cache, list(cache.unbind(0))                     # one cache a layer
        n = case["parents"] if op == "fork" else case["rows"]
        if op == "fork":
            s["parent_rows"] = torch.arange(n, device=DEV, dtype=torch.int32).repeat_interleave(case["children"])
            s["child_rows"] = torch.arange(n, n + n * case["children"], device=DEV, dtype=torch.int32)
        else:
            s["rows"] = torch.arange(1, n, 2, device=DEV, dtype=torch.int32)       # every second request ends
        return s
    s.update(_paged(case, seed))
    data, scales = _fp4_pool(g)
    nb, bs = s["blocks"], case["block"]
    if op == "mla":
        s["cache"] = torch.cat([_pick(data, (nb, bs, 256), g),
                                _pick(normal(1 << 16).float().to(torch.float8_e4m3fn).view(torch.uint8), (nb, bs, 64), g),
                                _pick(scales, (nb, bs, 32), g)], 2)
        s["q"] = (1.2 * normal(s["tokens"], case["heads"], 576).float()).to(torch.bfloat16)
        s["softmax_scale"] = 192 ** -0.5
        s["tree_mask"] = _tree(case, seed, s["tokens"])
        return s
    h, hs = case["kv_heads"], case["hs"]
    s["cache"] = torch.cat([_pick(data, (nb, 2, bs * h * hs // 2), g), _pick(scales, (nb, 2, bs * h * hs // 16), g)],
                           2).view(nb, 2, bs, h, hs // 2 + hs // 16)
    s["q"] = (1.5 * normal(s["tokens"], case["heads"], hs).float()).to(torch.bfloat16)
    s["k_scale"] = torch.tensor([0.75], device=DEV)
    s["v_scale"] = torch.tensor([1.25], device=DEV)
    s["softmax_scale"] = hs ** -0.5
    if op == "tree":
        s["tree_mask"] = _tree(case, seed, s["tokens"])
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    op = state["op"]
    if own:
        return _own(state)
    if op == "qk":
        return _plain_qk(state)
    if op == "fork":
        return _plain_fork(state)
    if op == "compact":
        return _plain_compact(state)
    return _plain_attention(state)


def _own(s):
    import gather_concat_cache_amd as gc
    op, case = s["op"], s["case"]
    if op == "qk":
        q, k = gc.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["cos_sin"], eps=1e-6,
                               interleaved=case["interleaved"])
        return dict(q=q, k=k)
    if op == "fork":
        table, lens, refs = s["block_table"].clone(), s["seq_lens"].clone(), s["ref_counts"].clone()
        status = gc.fork_requests(s["caches"], case["block"], table, lens, refs, s["parent_rows"], s["child_rows"])
        return dict(block_table=table, seq_lens=lens, ref_counts=refs, status=status, cache=s["cache"])
    if op == "compact":
        table, lens, refs = s["block_table"].clone(), s["seq_lens"].clone(), s["ref_counts"].clone()
        gc.free_requests(case["block"], table, lens, refs, s["rows"])
        page_map = gc.compact_pages(s["caches"], case["block"], table, lens, refs)
        return dict(block_table=table, seq_lens=lens, ref_counts=refs, page_map=page_map, cache=s["cache"])
    if op == "mla":
        out, lse = gc.tree_attention_nvfp4_ds_mla(s["q"], s["cache"], s["block_table"], s["query_starts"], s["seq_lens"],
                                                  s["tree_mask"], s["max_seq_len"], s["softmax_scale"], return_lse=True)
    elif op == "tree":
        out, lse = gc.tree_attention_nvfp4_kv(s["q"], s["cache"], s["k_scale"], s["v_scale"], s["block_table"],
                                              s["query_starts"], s["seq_lens"], s["tree_mask"], s["max_seq_len"],
                                              s["softmax_scale"], return_lse=True)
    else:
        out, lse = gc.attention_nvfp4_kv(s["q"], s["cache"], s["k_scale"], s["v_scale"], s["block_table"],
                                         s["query_starts"], s["seq_lens"], s["max_seq_len"], s["softmax_scale"],
                                         window=case["window"], num_sinks=case["sinks"], return_lse=True)
    return dict(out=out, lse=lse)


def _plain_qk(s):
    case = s["case"]
    rot = case["rot"]
    cs = s["cos_sin"][s["positions"]][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16)

    return dict(q=one(s["q"], s["q_weight"]), k=one(s["k"], s["k_weight"]))


def _plain_fork(s):
    bs = s["case"]["block"]
    table, lens, refs = s["block_table"].clone(), s["seq_lens"].clone(), s["ref_counts"].clone()
    parent, child = s["parent_rows"].long(), s["child_rows"].long()
    n = lens[parent]
    full, need = n // bs, (n % bs != 0)
    upto = need.int().cumsum(0)
    free = torch.argsort((refs > 0).int(), stable=True)          # free pages first, lowest ids first
    ok = upto <= (refs == 0).sum()
    take = ok & need
    last = table[parent].gather(1, full.long().clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    new = torch.where(take, free[(upto - 1).clamp(min=0).long()].int(), last)
    col = torch.arange(table.shape[1], device=table.device)[None]
    shared = (col < full[:, None]) & ok[:, None]
    row = torch.where(shared, table[parent], table[child])
    row = torch.where((col == full[:, None]) & take[:, None], new[:, None], row)
    spare = torch.cat([refs, refs.new_zeros(1)])                  # one more place for what is not counted
    spare.index_add_(0, torch.where(shared, table[parent], refs.numel()).flatten().long(),
                     torch.ones(shared.numel(), dtype=torch.int32, device=refs.device))
    spare.index_add_(0, torch.where(take, new, refs.numel()).long(), torch.ones_like(new))
    src, dst = torch.where(take, last, 0).long(), torch.where(take, new, 0).long()
    s["cache"][:, dst] = s["cache"][:, src]
    table[child] = row
    lens[child] = torch.where(ok, n, lens[child])
    return dict(block_table=table, seq_lens=lens, ref_counts=spare[:-1].contiguous(), status=ok.int(), cache=s["cache"])


def _plain_compact(s):
    bs = s["case"]["block"]
    table, lens, refs = s["block_table"].clone(), s["seq_lens"].clone(), s["ref_counts"].clone()
    nb = refs.numel()
    col = torch.arange(table.shape[1], device=table.device)[None]
    rows = s["rows"].long()
    owned = col < ((lens[rows] + bs - 1) // bs)[:, None]
    spare = torch.cat([refs, refs.new_zeros(1)])
    spare.index_add_(0, torch.where(owned, table[rows], nb).flatten().long(),
                     torch.full((owned.numel(),), -1, dtype=torch.int32, device=refs.device))
    refs = spare[:-1].contiguous()
    table[rows] = torch.where(owned, -1, table[rows])
    lens[rows] = 0
    live = refs > 0
    ids = torch.arange(nb, device=refs.device)
    count = live.sum()
    before = live.long().cumsum(0) - live.long()
    holes = ids[~live & (ids < count)]
    movers = ids[live & (ids >= count)].flip(0)                   # the highest page takes the lowest hole
    page_map = torch.where(live, ids, -1).int()
    page_map[movers] = holes.int()
    s["cache"][:, holes] = s["cache"][:, movers]
    refs[holes] = refs[movers]
    refs[movers] = 0
    owned = col < ((lens + bs - 1) // bs)[:, None]
    table = torch.where(owned, page_map[table.clamp(min=0).long()], table)
    return dict(block_table=table, seq_lens=lens, ref_counts=refs, page_map=page_map, cache=s["cache"])


def _decode(data, scale):
    """Codes [..., n/2] and e4m3 scales [..., n/16] -> float [..., n]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=data.device)
    pair = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], 1)             # byte -> (low, high)
    v = pair[data.int()].flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scale.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _plain_attention(s):
    case, op = s["case"], s["op"]
    bs, qs, lens = case["block"], s["query_starts"], s["seq_lens"]
    table, n = s["block_table"], s["max_query_len"]
    qlen = qs[1:] - qs[:-1]
    ctx = (lens - qlen)[:, None]
    t = torch.arange(s["tokens"], device=DEV, dtype=torch.int32)
    req = torch.searchsorted(qs, t, right=True).int() - 1                          # request of each token
    row = (t - qs[req]).long()
    req = req.long()
    # the positions that any query of a request can see
    if op == "window":
        w, sinks = case["window"], case["sinks"]
        first = (ctx - (w - 1)).clamp(min=0)
        span = min(s["max_seq_len"], w - 1 + n)
        pos = torch.cat([torch.arange(sinks, device=DEV)[None].expand(len(lens), -1),
                         first + torch.arange(span, device=DEV)[None]], 1)
        live = torch.cat([torch.arange(sinks, device=DEV)[None] < first, torch.ones_like(pos[:, sinks:], dtype=torch.bool)],
                         1) & (pos < lens[:, None])
    else:
        pos = torch.arange(s["max_seq_len"], device=DEV)[None].expand(len(lens), -1)
        live = pos < lens[:, None]
    at = torch.where(live, pos, 0).long()
    blk, off = table.gather(1, at // bs).long(), at % bs
    q = torch.zeros((len(lens), n) + s["q"].shape[1:], device=DEV)
    q[req, row] = s["q"].float()
    if op == "mla":
        e = s["cache"][blk, off]
        nope = _decode(e[..., :256], e[..., 320:352])
        k = torch.cat([nope, e[..., 256:320].contiguous().view(torch.float8_e4m3fn).float()], -1)[:, None]
        v = nope[:, None]
        groups = case["heads"]
    else:
        h, hs = case["kv_heads"], case["hs"]
        side = s["cache"].view(s["blocks"], 2, -1)
        data = side[..., :bs * h * hs // 2].unflatten(-1, (bs, h, hs // 2))
        scale = side[..., bs * h * hs // 2:].unflatten(-1, (bs, h, hs // 16))
        k = _decode(data[blk, 0, off], scale[blk, 0, off].contiguous()).transpose(1, 2) * s["k_scale"]
        v = _decode(data[blk, 1, off], scale[blk, 1, off].contiguous()).transpose(1, 2) * s["v_scale"]
        groups = case["heads"] // h
    hk = k.shape[1]
    q = q.unflatten(2, (hk, groups)).transpose(1, 2).flatten(2, 3)                 # [batch, kv heads, n * groups, hs]
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["softmax_scale"]
    i = torch.arange(n, device=DEV)[None, :, None]
    here = ctx[:, :, None] + i                                                     # each query's position
    j = pos[:, None]
    if op == "window":
        see = (j <= here) & ((j < sinks) | (here - j < w))
    else:
        mask = torch.zeros((len(lens), n, case["qmax"]), dtype=torch.bool, device=DEV)
        mask[req, row] = s["tree_mask"]
        draft = (pos - ctx)[:, None].expand(-1, n, -1)
        see = (draft < 0) | mask.gather(2, draft.clamp(0, case["qmax"] - 1).long())
    see = (see & live[:, None]).repeat_interleave(groups, 1)[:, None]
    score = score.masked_fill(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + torch.where(top > -math.inf, top, 0.0)
    o = o.unflatten(2, (n, groups)).transpose(1, 2).flatten(2, 3)                  # [batch, n, heads, values]
    lse = lse.unflatten(2, (n, groups)).transpose(1, 2).flatten(2, 4)
    return dict(out=o[req, row].to(torch.bfloat16), lse=lse[req, row])


# --------------------------------------------------------------------------
# 64-bit values from the definitions
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None                                     # whole numbers and copied bytes
    s = prepare(case, seed)
    if case["op"] == "qk":
        return dict(q=_exact_rows(case, s, s["q"], s["q_weight"]), k=_exact_rows(case, s, s["k"], s["k_weight"]))
    starts, lens = s["query_starts"].tolist(), s["seq_lens"].tolist()
    outs, lses = [], []
    for b, length in enumerate(lens):
        positions = torch.arange(length, device=DEV)
        pages = s["block_table"][b].long()[positions // case["block"]]
        slots = positions % case["block"]
        q = s["q"][starts[b]:starts[b + 1]].double()
        n = q.shape[0]
        where = torch.arange(length - n, length, device=DEV)
        if case["op"] == "window":
            gap = where[:, None] - positions[None]
            hidden = (gap < 0) | ((gap >= case["window"]) & (positions >= case["sinks"])[None])
        else:
            hidden = torch.zeros(n, length, dtype=torch.bool, device=DEV)
            hidden[:, length - n:] = ~s["tree_mask"][starts[b]:starts[b + 1], :n]
        out = torch.empty(n, case["heads"], 512 if case["op"] == "mla" else case["hs"], dtype=torch.float64, device=DEV)
        lse = torch.empty(n, case["heads"], dtype=torch.float64, device=DEV)
        for head in range(case["heads"]):
            if case["op"] == "mla":
                if head == 0:
                    entry = s["cache"][pages, slots]
                    values = _exact_values(entry[:, :256], entry[:, 320:])
                    keys = torch.cat([values, entry[:, 256:320].contiguous().view(torch.float8_e4m3fn).double()], 1)
            else:
                kv, each = divmod(head, case["heads"] // case["kv_heads"])
                if each == 0:
                    keys = _exact_side(case, s, pages, slots, kv, 0)
                    values = _exact_side(case, s, pages, slots, kv, 1)
            logit = (q[:, head] @ keys.T) * s["softmax_scale"]
            logit[hidden] = -math.inf
            lse[:, head] = torch.logsumexp(logit, 1)
            out[:, head] = torch.exp(logit - lse[:, head, None]) @ values
        outs.append(out)
        lses.append(lse)
    return dict(out=torch.cat(outs), lse=torch.cat(lses))


def _exact_values(data, scale):
    code = torch.stack([data & 15, data >> 4], -1).flatten(1).long()
    size = code % 8
    value = torch.where(size < 2, size * 0.5, (1 + (size % 2) * 0.5) * 2.0 ** (size // 2 - 1).double())
    value = torch.where(code >= 8, -value, value).double()
    return value * scale.contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)


def _exact_side(case, s, pages, slots, head, side):
    h, hs, bs = case["kv_heads"], case["hs"], case["block"]
    flat = s["cache"].view(s["blocks"], 2, bs * h * hs * 9 // 16)[:, side]
    one = (slots * h + head)[:, None]
    data = flat[pages[:, None], one * (hs // 2) + torch.arange(hs // 2, device=DEV)]
    scale = flat[pages[:, None], bs * h * hs // 2 + one * (hs // 16) + torch.arange(hs // 16, device=DEV)]
    return _exact_values(data, scale) * (s["v_scale"] if side else s["k_scale"]).double()


def _exact_rows(case, s, x, w):
    x = x.double()
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["hs"] + 1e-6) * w.double()
    half = case["rot"] // 2
    turn = s["cos_sin"][s["positions"]].double()[:, None]
    turn = torch.complex(turn[..., :half].contiguous(), turn[..., half:].contiguous())
    if case["interleaved"]:
        first, second = slice(0, case["rot"], 2), slice(1, case["rot"], 2)
    else:
        first, second = slice(0, half), slice(half, case["rot"])
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
    y = y.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y
