"""Cases and plain forms of the operators of an 8-bit paged K/V cache and of
whole prompts: append with the position rotation, attention over the cache,
attention of packed prompts.

A case names an operator (`op`) and its sizes; lengths of a batch are drawn
from the case's own `lens` number, contents from the seed.  With `own` False,
`run` computes the operator with elementary torch operations in 32 bits,
rounded once at the end; with `own` True it calls this repository's package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TOP = 448.0                                             # largest e4m3 value
LEAST = 2.0 ** -100                                     # smallest scale of a page


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decoded token: launch latency is what counts
        dict(name="append_one_token", op="append", batch=1, qmin=1, qmax=1, cmin=1037, cmax=1037, heads=32, kv_heads=8,
             hs=128, rot=128, block=16, interleaved=False, keys=False, lens=1),
        # a decode batch: every request's token joins a page that is partly full
        dict(name="append_decode", op="append", batch=256, qmin=1, qmax=1, cmin=100, cmax=4000, heads=32, kv_heads=8,
             hs=128, rot=128, block=16, interleaved=False, keys=False, lens=2),
        # prompts of a prefill step; the rotated keys go on to the prompt's attention
        dict(name="append_prefill", op="append", batch=6, qmin=1000, qmax=4096, cmin=0, cmax=300, heads=32, kv_heads=8,
             hs=128, rot=128, block=16, interleaved=False, keys=True, lens=3),
        # one user decoding
        dict(name="cache_one_token", op="cache", batch=1, qmin=1, qmax=1, cmin=1037, cmax=1037, heads=32, kv_heads=8,
             hs=128, block=16, window=0, sinks=0, lens=4),
        # a decode batch with contexts of 1 Ki to 32 Ki tokens
        dict(name="cache_decode", op="cache", batch=64, qmin=1, qmax=1, cmin=1024, cmax=32768, heads=32, kv_heads=8,
             hs=128, block=16, window=0, sinks=0, lens=5),
        # a few drafted tokens of each request behind a 4 Ki window with sinks
        dict(name="cache_window", op="cache", batch=32, qmin=2, qmax=8, cmin=1024, cmax=16384, heads=32, kv_heads=8,
             hs=128, block=64, window=4096, sinks=4, lens=6),
        # ragged prefill chunks over cached contexts
        dict(name="cache_chunk", op="cache", batch=3, qmin=1024, qmax=2048, cmin=2048, cmax=6144, heads=32, kv_heads=8,
             hs=128, block=16, window=0, sinks=0, lens=7),
        # one short question
        dict(name="prompt_one", op="prompt", batch=1, qmin=37, qmax=37, cmin=0, cmax=0, heads=32, kv_heads=8, dk=128,
             dv=128, causal=True, lens=8),
        # many short prompts packed into one step
        dict(name="prompt_packed", op="prompt", batch=64, qmin=20, qmax=500, cmin=0, cmax=0, heads=32, kv_heads=8, dk=128,
             dv=128, causal=True, lens=9),
        # long prompts
        dict(name="prompt_long", op="prompt", batch=2, qmin=6000, qmax=8192, cmin=0, cmax=0, heads=32, kv_heads=8, dk=128,
             dv=128, causal=True, lens=10),
        # prompts of a latent-cache model after the up-projection: keys of 192, values of 128
        dict(name="prompt_latent", op="prompt", batch=4, qmin=1000, qmax=4096, cmin=0, cmax=0, heads=16, kv_heads=16,
             dk=192, dv=128, causal=True, lens=11),
        # the same model's chunk of queries over gathered chunks of context
        dict(name="prompt_context", op="prompt", batch=3, qmin=500, qmax=1024, cmin=4096, cmax=8192, heads=16,
             kv_heads=16, dk=192, dv=128, causal=False, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "cache", "cache", "prompt", "prompt"])
    kv = rng.choice([1, 2, 4, 8])
    case = dict(op=op, kv_heads=kv, heads=kv * rng.choice([1, 2, 3, 4, 8]), lens=rng.randrange(1 << 30))
    if op == "append":
        hs = rng.choice([64, 80, 96, 128, 128, 192, 256])
        case.update(hs=hs, rot=rng.choice([hs, hs // 2 // 16 * 16]), block=rng.choice([16, 16, 24, 64, 128]),
                    interleaved=rng.random() < 0.4, keys=rng.random() < 0.5)
        if rng.random() < 0.5:                          # decoding, with a few drafted tokens
            case.update(batch=_log(rng, 1, 256), qmin=1, qmax=rng.choice([1, 1, 1, 5]), cmin=0, cmax=_log(rng, 10, 2000))
        else:
            case.update(batch=_log(rng, 1, 16), qmin=1, qmax=_log(rng, 10, 600), cmin=0, cmax=_log(rng, 1, 500))
        return case
    if op == "cache":
        cmax = _log(rng, 10, 8000)
        case.update(hs=rng.choice([64, 80, 96, 128, 128, 256]), block=rng.choice([16, 16, 24, 64, 128]),
                    batch=_log(rng, 1, 32), qmin=1, qmax=_log(rng, 1, 64), cmin=cmax // rng.randint(1, 8), cmax=cmax,
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]), sinks=rng.choice([0, 1, 4, 40]))
        if rng.random() < 0.4:                          # a prefill chunk
            case.update(batch=rng.randint(1, 3), qmax=_log(rng, 100, 2000))
    else:
        dk, dv = rng.choice([(64, 64), (80, 80), (96, 96), (128, 128), (128, 128), (192, 128), (192, 128), (256, 256)])
        qmax = _log(rng, 1, 4000)
        case.update(dk=dk, dv=dv, batch=_log(rng, 1, 24), qmin=max(1, qmax // rng.randint(1, 20)), qmax=qmax,
                    causal=rng.random() < 0.7, cmin=0, cmax=0)
        if not case["causal"] or rng.random() < 0.3:    # queries over a gathered context
            case.update(cmax=_log(rng, 1, 8000))
    while work(case)["flops"] > 3e11 or _padded(case) > 3e9:       # no dearer than the listed ones
        case["batch"] = (case["batch"] + 1) // 2
        case["qmax"] = (case["qmax"] + 1) // 2
        case["qmin"] = min(case["qmin"], case["qmax"])
    return case


def _lengths(case):
    """(query lengths, key lengths) of a batch: the first request has the
    longest query, the others any."""
    r = random.Random(case["lens"])
    q = [case["qmax"]] + [r.randint(case["qmin"], case["qmax"]) for _ in range(case["batch"] - 1)]
    c = [r.randint(case["cmin"], case["cmax"]) for _ in q]
    if not case.get("causal", True):                    # keys of their own; a request may have none
        return q, [max(c[0], 1)] + c[1:]
    return q, [n + m for n, m in zip(q, c)]


def _padded(case):
    """Logits of the batch when every request is as long as the longest."""
    q, l = _lengths(case)
    return len(q) * max(q) * max(l) * case["heads"]


def _sum_min(lo, hi, w):
    """Sum of min(x, w) over lo <= x < hi."""
    m = min(max(w, lo), hi)
    return (m - lo) * (lo + m - 1) // 2 + (hi - m) * w


def work(case):
    q, l = _lengths(case)
    h, hk, t = case["heads"], case["kv_heads"], sum(q)
    if case["op"] == "append":
        hs, bs = case["hs"], case["block"]
        pages = sum((n - 1) // bs - (n - m) // bs + 1 for n, m in zip(l, q))
        values = t * hk * hs
        return dict(bytes=4 * t * h * hs + (6 + 2 * case["keys"]) * values + 4 * t * case["rot"] + 16 * pages * hk,
                    flops=t * (3 * (h + hk) * case["rot"] + 2 * hk * hs))
    if case["op"] == "cache":
        hs = case["hs"]
        w = case["window"] + case["sinks"] if case["window"] else max(l)
        pairs = sum(_sum_min(m - n + 1, m + 1, w) for n, m in zip(q, l))
        keys = sum(min(m, w + n - 1) for n, m in zip(q, l))
        return dict(bytes=keys * hk * (2 * hs + 8 / case["block"]) + 4 * t * h * hs, flops=4 * hs * pairs * h)
    dk, dv = case["dk"], case["dv"]
    pairs = sum(n * (m - n) + n * (n + 1) // 2 if case["causal"] else n * m for n, m in zip(q, l))
    return dict(bytes=2 * t * h * (dk + dv) + 2 * sum(l) * hk * (dk + dv), flops=2 * (dk + dv) * pairs * h)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _starts(lens):
    return torch.tensor([0] + lens).cumsum(0).int().to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    q, l = _lengths(case)
    t, h, hk = sum(q), case["heads"], case["kv_heads"]
    s = dict(op=op, case=case, tokens=t, max_query_len=max(q), max_key_len=max(l), query_starts=_starts(q))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)

    if op == "prompt":
        s["softmax_scale"] = case["dk"] ** -0.5
        s["key_starts"] = _starts(l)
        if case["dk"] == case["dv"] and q == l:                     # one fused projection's output
            qkv = normal(t, h + 2 * hk, case["dk"])
            s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        else:
            s["q"], s["k"], s["v"] = normal(t, h, case["dk"]), normal(sum(l), hk, case["dk"]), normal(sum(l), hk, case["dv"])
        return s
    hs, bs = case["hs"], case["block"]
    pages = torch.tensor([-(-n // bs) for n in l])
    nb = int(pages.sum()) + 3
    order = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).int()
    owned = torch.arange(int(pages.max()) + 1)[None] < pages[:, None]
    table = torch.full(owned.shape, -1, dtype=torch.int32)
    table[owned] = order[:int(pages.sum())]
    # codes as a write makes them of normally distributed values, and each page's largest value over 448
    pool = (128 * torch.randn(1 << 16, generator=g, device=DEV)).clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)
    pick = torch.randint(0, pool.numel(), (nb, 2, bs, hk, hs), generator=g, device=DEV, dtype=torch.int32)
    s.update(blocks=nb, block_table=table.to(DEV), seq_lens=_i32(l), cache=pool[pick],
             scales=(1.5 + 3 * torch.rand(nb, 2, hk, generator=g, device=DEV)) / TOP)
    if op == "append":
        qkv = normal(t, h + 2 * hk, hs)
        s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        rot = case["rot"]
        inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        ang = torch.arange(max(l), dtype=torch.float64, device=DEV)[:, None] * inv
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        return s
    s["q"] = (1.5 * normal(t, h, hs).float()).to(torch.bfloat16)
    s["softmax_scale"] = hs ** -0.5
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    if own:
        return _own(state)
    return dict(append=_plain_append, cache=_plain_cache, prompt=_plain_prompt)[state["op"]](state)


def _own(s):
    import gather_concat_cache_amd as gc
    op, case = s["op"], s["case"]
    if op == "append":
        q, k = gc.rope_append_fp8_kv(s["q"], s["k"], s["v"], s["cache"], s["scales"], s["block_table"], s["query_starts"],
                                     s["seq_lens"], s["cos_sin"], interleaved=case["interleaved"], return_k=case["keys"])
        return _appended(s, q, k)
    if op == "cache":
        out, lse = gc.attention_fp8_kv(s["q"], s["cache"], s["scales"], s["block_table"], s["query_starts"], s["seq_lens"],
                                       s["max_key_len"], s["softmax_scale"], window=case["window"] or None,
                                       num_sinks=case["sinks"], return_lse=True)
    else:
        out, lse = gc.prompt_attention(s["q"], s["k"], s["v"], s["query_starts"], s["key_starts"], s["max_key_len"],
                                       s["softmax_scale"], causal=case["causal"], return_lse=True)
    return dict(out=out, lse=lse)


def _appended(s, q, k):
    """The operator's outputs; the cache as the e4m3 values that it holds."""
    out = dict(q=q, cache=s["cache"].view(torch.float8_e4m3fn), scales=s["scales"])
    if s["case"]["keys"]:
        out["k"] = k
    return out


def _rows(s):
    """Each packed query's request, its number in it, and the requests' tokens
    before the queries."""
    qs = s["query_starts"]
    t = torch.arange(s["tokens"], device=DEV, dtype=torch.int32)
    req = torch.searchsorted(qs, t, right=True) - 1
    return req, (t - qs[req]).long(), qs[1:] - qs[:-1]


def _plain_append(s):
    case, bs = s["case"], s["case"]["block"]
    req, row, qlen = _rows(s)
    ctx = s["seq_lens"] - qlen
    pos = ctx[req] + row
    rot = case["rot"]
    cs = s["cos_sin"][pos][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]

    def turn(x):
        x = x.float()
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, x[..., rot:]], -1)

    k = turn(s["k"])
    kv = torch.stack([k, s["v"].float()], 1)                                       # [tokens, 2, heads, hs]
    blk, off = s["block_table"][req, pos // bs].long(), pos % bs
    scales = s["scales"]
    # pages that hold tokens from before: the first of each request, unless it begins there
    page = s["block_table"].gather(1, (ctx // bs).long()[:, None])[:, 0].long()
    kept = torch.zeros(s["blocks"], dtype=torch.int32, device=DEV)
    kept[page] = ctx % bs
    need = torch.zeros_like(scales).index_reduce_(0, blk, kv.abs().amax(-1), "amax")
    need = (need / TOP).clamp(min=LEAST)
    touched = torch.zeros(s["blocks"], dtype=torch.bool, device=DEV)
    touched[blk] = True
    (mn, en), (mo, eo) = torch.frexp(need), torch.frexp(scales)
    grow = (en - eo + (mn > mo).int()).clamp(min=0)                                # least k with scale 2^k >= need
    grow = torch.where((kept > 0)[:, None, None], grow, 0)
    new = torch.where((kept > 0)[:, None, None], torch.ldexp(scales, grow), need)
    was = s["cache"][page]
    less = was.view(torch.float8_e4m3fn).float() * torch.ldexp(torch.ones_like(scales), -grow)[page][:, :, None, :, None]
    held = (torch.arange(bs, device=DEV) < kept[page][:, None])[:, None, :, None, None]
    s["cache"][page] = torch.where(held, less.to(torch.float8_e4m3fn).view(torch.uint8), was)
    code = (kv * (1 / new)[blk][..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    s["cache"][blk, :, off] = code.view(torch.uint8)
    scales.copy_(torch.where(touched[:, None, None], new, scales))
    return _appended(s, turn(s["q"]).to(torch.bfloat16), k.to(torch.bfloat16))


def _softmax(score, see, v):
    """(rows' weighted values, lse) of float logits."""
    score = score.masked_fill_(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, 1.0), torch.log(total) + top


def _plain_cache(s):
    case, bs, lens, n = s["case"], s["case"]["block"], s["seq_lens"], s["max_query_len"]
    req, row, qlen = _rows(s)
    ctx = (lens - qlen)[:, None]
    w, sinks = case["window"], case["sinks"]
    every = torch.arange(s["max_key_len"], device=DEV)[None]
    if w:                                               # the positions that any query of a request can see
        first = (ctx - (w - 1)).clamp(min=0)
        head = every[:, :sinks].expand(len(lens), -1)
        pos = torch.cat([head, first + every[:, :w - 1 + n]], 1)
        live = torch.cat([head < first, torch.ones_like(pos[:, head.shape[1]:], dtype=torch.bool)], 1) & (pos < lens[:, None])
    else:
        pos = every.expand(len(lens), -1)
        live = pos < lens[:, None]
    at = torch.where(live, pos, 0).long()
    blk, off = s["block_table"].gather(1, at // bs).long(), at % bs
    h, hk = case["heads"], case["kv_heads"]
    k, v = ((s["cache"][blk, side, off].view(torch.float8_e4m3fn).float() * s["scales"][blk, side][..., None]).transpose(1, 2).contiguous() for side in (0, 1))
    q = torch.zeros((len(lens), n) + s["q"].shape[1:], device=DEV)
    q[req, row] = s["q"].float()
    q = q.unflatten(2, (hk, h // hk)).transpose(1, 2).flatten(2, 3)                # [batch, kv heads, n * group, hs]
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["softmax_scale"]
    here = (ctx + torch.arange(n, device=DEV))[:, :, None]                         # each query's position
    j = pos[:, None]
    see = (j <= here) & live[:, None]
    if w:
        see &= (j < sinks) | (here - j < w)
    o, lse = _softmax(score, see.repeat_interleave(h // hk, 1)[:, None], v)
    return _packed(o, lse, n, h // hk, req, row)


def _packed(o, lse, n, group, req, row):
    o = o.unflatten(2, (n, group)).transpose(1, 2).flatten(2, 3)                   # [batch, n, heads, values]
    lse = lse.unflatten(2, (n, group)).transpose(1, 2).flatten(2, 4)
    return dict(out=o[req, row].to(torch.bfloat16), lse=lse[req, row])


def _plain_prompt(s):
    case, n, m = s["case"], s["max_query_len"], s["max_key_len"]
    req, row, qlen = _rows(s)
    ks = s["key_starts"]
    klen = ks[1:] - ks[:-1]
    h, hk, b = case["heads"], case["kv_heads"], len(klen)
    t = torch.arange(s["k"].shape[0], device=DEV, dtype=torch.int32)
    kreq = torch.searchsorted(ks, t, right=True) - 1
    krow = (t - ks[kreq]).long()
    q = torch.zeros((b, n, h, case["dk"]), device=DEV)
    q[req, row] = s["q"].float()
    q = q.unflatten(2, (hk, h // hk)).transpose(1, 2).flatten(2, 3)
    k = torch.zeros((b, hk, case["dk"], m), device=DEV)
    k[kreq, :, :, krow] = s["k"].float()
    v = torch.zeros((b, hk, m, case["dv"]), device=DEV)
    v[kreq, :, krow] = s["v"].float()
    score = torch.matmul(q, k).mul_(s["softmax_scale"])
    j = torch.arange(m, device=DEV)[None, None]
    see = (j < klen[:, None, None]).expand(b, n, m)
    if case["causal"]:
        see = see & (j <= (klen - qlen)[:, None, None] + torch.arange(n, device=DEV)[None, :, None])
    o, lse = _softmax(score, see.repeat_interleave(h // hk, 1)[:, None], v)
    return _packed(o, lse, n, h // hk, req, row)


# --------------------------------------------------------------------------
# 64-bit values from the definitions
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    starts, outs, lses = s["query_starts"].tolist(), [], []
    lens = _lengths(case)[1]
    offset = 0
    for b, length in enumerate(lens):
        q = s["q"][starts[b]:starts[b + 1]].double()
        n = q.shape[0]
        at = torch.arange(length, device=DEV)
        gap = torch.arange(length - n, length, device=DEV)[:, None] - at[None]
        if case["op"] == "cache":
            pages = s["block_table"][b].long()[at // case["block"]]
            hidden = gap < 0
            if case["window"]:
                hidden |= (gap >= case["window"]) & (at >= case["sinks"])
        else:
            hidden = (gap < 0) & case["causal"]
        out = torch.empty(n, case["heads"], case.get("dv") or case["hs"], dtype=torch.float64, device=DEV)
        lse = torch.empty(n, case["heads"], dtype=torch.float64, device=DEV)
        for head in range(case["heads"]):
            kv, each = divmod(head, case["heads"] // case["kv_heads"])
            if each == 0 and case["op"] == "cache":
                keys, values = (s["cache"][pages, side, at % case["block"], kv].view(torch.float8_e4m3fn).double()
                                * s["scales"][pages, side, kv].double()[:, None] for side in (0, 1))
            elif each == 0:
                keys, values = s["k"][offset:offset + length, kv].double(), s["v"][offset:offset + length, kv].double()
            logit = (q[:, head] @ keys.T) * s["softmax_scale"]
            logit[hidden] = -math.inf
            lse[:, head] = torch.logsumexp(logit, 1)
            out[:, head] = torch.exp(logit - torch.nan_to_num(lse[:, head, None], neginf=0.0)) @ values
        offset += length
        outs.append(out)
        lses.append(lse)
    return dict(out=torch.cat(outs), lse=torch.cat(lses))


def _exact_turn(case, x, where, cos_sin):
    y = x.double().clone()
    half = case["rot"] // 2
    table = cos_sin[where].double()[:, None]
    turn = torch.complex(table[..., :half].contiguous(), table[..., half:].contiguous())
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (slice(0, half),
                                                                                               slice(half, 2 * half))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_e4m3(x):
    """The nearest e4m3 value, ties to even, of float64 values."""
    x = x.clamp(-TOP, TOP)
    step = torch.ldexp(torch.ones_like(x), (torch.frexp(x)[1] - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_append(case, s):
    q, l = _lengths(case)
    bs = case["block"]
    where = torch.cat([torch.arange(m - n, m, device=DEV) for n, m in zip(q, l)])
    qt, kt = (_exact_turn(case, s[x], where, s["cos_sin"]) for x in "qk")
    cache, scales = s["cache"].view(torch.float8_e4m3fn).double(), s["scales"].double()
    table, at = s["block_table"].tolist(), 0
    for b, (n, m) in enumerate(zip(q, l)):
        pos = m - n
        while pos < m:
            page, off = table[b][pos // bs], pos % bs
            cnt = min(bs - off, m - pos)
            x = torch.stack([kt[at:at + cnt], s["v"][at:at + cnt].double()])       # [2, tokens, heads, hs]
            need = (x.abs().amax((1, 3)) / TOP).clamp(min=LEAST)
            if off:
                times = torch.exp2(torch.ceil(torch.log2(need / scales[page])).clamp(min=0))
                cache[page, :, :off] = _exact_e4m3(cache[page, :, :off] / times[:, None, :, None])
                need = scales[page] * times
            scales[page] = need
            cache[page, :, off:off + cnt] = _exact_e4m3(x / need[:, None, :, None])
            pos, at = pos + cnt, at + cnt
    out = dict(q=qt, cache=cache, scales=scales)
    if case["keys"]:
        out["k"] = kt
    return out
