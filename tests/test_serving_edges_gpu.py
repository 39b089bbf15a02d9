"""GPU tests of the 8-bit paged cache and of the prompts' attention at the edges
of what their headers allow: value scales over the whole range, values that are
not finite in every form of the prompt kernel, and every form that a call's
sizes select."""
import numpy as np
import pytest
import torch

import operator_refs as pages_ref
import serving_refs as ref
from gpu_util import dev, host
from test_operators_gpu import Batch, check_pages, close, random_state
from test_serving_gpu import cache_view, check_cache, g, random_codes  # noqa: F401

pytestmark = pytest.mark.gpu


def rows_kernel(total_q, batch, group, hs):
    """Rows a workgroup that the sizes of a cache attention call select: 16 or 32
    (the kernel of few rows) or 128."""
    mean = -(-total_q * group // batch)
    return 16 if mean <= 16 or (hs > 128 and mean <= 32) else 32 if mean <= 32 else 128


# ---------------------------------------------------------------------------
# value scales over their whole range
# ---------------------------------------------------------------------------
def check_scaled(g, batch, hk, group, hs, codes, scales, q, scale, window=None, sinks=0, mask=None, workspace=None):  # noqa: F811
    """attention_fp8_kv over codes uint8 [nb, 2, bs, hk, hs] and scales fp32 [nb,
    2, hk] against 64 bits, each row with the largest value scale that it sees."""
    bs = batch.bs
    flat, view = cache_view(batch.nb, bs, hk, hs, "nhd")
    view.copy_(dev(codes))
    qt, q64 = ref.bf16(q)
    bt, starts, lens = batch.metadata()
    out, lse = g.attention_fp8_kv(qt.cuda(), view, dev(scales), bt, starts, lens, max(batch.lens), scale, window=window,
                                  num_sinks=sinks, tree_mask=None if mask is None else dev(mask), return_lse=True,
                                  workspace=workspace)
    torch.cuda.synchronize()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, (n, m) in enumerate(zip(batch.qlens, batch.lens)):
        r0 = int(batch.starts[b])
        see = ref.causal(n, m, window, sinks) if mask is None else ref.tree(n, m, mask[r0:r0 + n])
        at = np.arange(m)
        blk = batch.table[b][at // bs]
        for h in range(hk):
            k, v = (ref.e4m3(codes[blk, side, at % bs, h]) * scales[blk, side, h].astype(np.float64)[:, None] for side in (0, 1))
            for i in range(n):
                if not see[i].any():
                    continue
                heads = slice(h * group, (h + 1) * group)
                floor = 2.0 ** -31 * 448 * scales[blk, 1, h][see[i]].max()
                o, l, ot, lt = ref.attend(q64[r0 + i, heads], k, v, np.repeat(see[i:i + 1], group, 0), float(np.float32(scale)),
                                          2.0 ** -11, floor)
                close(lse[r0 + i, heads], l, lt, f"request {b} query {i} head {h} lse")
                close(out[r0 + i, heads], o, ot, f"request {b} query {i} head {h} out")


@pytest.mark.parametrize("qlen,group,hs,bs", [(1, 4, 64, 16), (1, 2, 64, 24), (5, 4, 64, 16), (5, 4, 128, 24), (12, 4, 64, 16),
                                              (12, 4, 128, 40), (1, 1, 256, 16)])
def test_cache_long_runs_of_zero_values(g, qlen, group, hs, bs):  # noqa: F811
    """65536 keys whose values are zero, as an append of zeros leaves them (scale
    2^-100): the sum of weights over scales is beyond binary32 once the logits
    rise behind the first keys; the lse is an ordinary number."""
    rng = np.random.default_rng(hs + bs)
    n = 65536
    batch = Batch(rng, [qlen], [n], bs)
    codes = np.zeros((batch.nb, 2, bs, 1, hs), np.uint8)
    scales = np.full((batch.nb, 2, 1), 2.0 ** -100, np.float32)
    at = np.arange(n)
    codes[batch.table[0][at // bs], 0, at % bs, 0, 0] = np.where(at < 128, 0, 0x38)     # 0, then 1: logits 0, then 7.5 in log2 units
    scales[:, 0] = 1.0
    q = rng.standard_normal((qlen, group, hs))
    q[:, :, 0] = 1.0
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    check_scaled(g, batch, 1, group, hs, codes, scales, q, 5.2, workspace=none)


RANGE = [2.0 ** -100, 2.0 ** -97, 2.0 ** -9, 2.0 ** 60, 2.0 ** 110]


@pytest.mark.parametrize("kind", ["causal", "window", "tree"])
@pytest.mark.parametrize("qlens,group,hs,bs", [([1, 2, 1], 2, 64, 16), ([1, 2, 1], 2, 128, 24), ([4, 3, 5], 4, 128, 16),
                                               ([4, 3, 5], 4, 64, 40), ([3, 70, 20], 2, 64, 16), ([3, 70, 20], 2, 128, 24),
                                               ([3, 40, 20], 2, 256, 16)])
def test_cache_scales_over_their_range(g, qlens, group, hs, bs, kind):  # noqa: F811
    """Pages of zero, tiny, ordinary, large and huge values in one sequence, in
    any order: every weight counts in the lse and in the output."""
    rng = np.random.default_rng(hs + bs + len(kind))
    lens = [310, 290, 2100]
    batch = Batch(rng, qlens, lens, bs)
    codes = random_codes(rng, (batch.nb, 2, bs, 2, hs))
    scales = np.empty((batch.nb, 2, 2), np.float32)
    scales[:, 0] = 2.0 ** rng.uniform(-11, -9, (batch.nb, 2))
    pick = rng.integers(0, len(RANGE), (batch.nb, 2))
    scales[:, 1] = np.array(RANGE, np.float32)[pick]
    for h in range(2):
        codes[pick[:, h] == 0, 1, :, h] = 0                  # an append of zeros
    for b, n in enumerate(lens):                             # nothing was written behind a sequence's last token
        codes[batch.table[b, (n - 1) // bs], :, (n - 1) % bs + 1:] = 0xFF
    q = rng.standard_normal((batch.T, 2 * group, hs))
    mask = rng.random((batch.T, max(qlens))) < 0.5 if kind == "tree" else None
    if mask is not None:
        mask |= np.eye(max(qlens), dtype=bool)[np.concatenate([np.arange(n) for n in qlens])]
    w, s = (150, 20) if kind == "window" else (None, 0)
    for ws in (None, torch.empty(0, dtype=torch.uint8, device="cuda")):
        check_scaled(g, batch, 2, group, hs, codes, scales, q, hs ** -0.5, w, s, mask, ws)


@pytest.mark.parametrize("order", ["rising", "falling"])
@pytest.mark.parametrize("qlen,bs", [(1, 16), (1, 24), (4, 64), (8, 16), (8, 24), (40, 16), (40, 24)])
def test_cache_scales_in_order(g, qlen, bs, order):  # noqa: F811
    """Value scales that rise or fall page by page from one end of their range to
    the other: no jump loses the sum of the pages before it."""
    rng = np.random.default_rng(bs + qlen)
    batch = Batch(rng, [qlen], [700], bs)
    codes = random_codes(rng, (batch.nb, 2, bs, 1, 64))
    scales = np.full((batch.nb, 2, 1), 2.0 ** -9, np.float32)
    pages = -(-700 // bs)
    for ends in ((-100, 110), (-39, 110), (-39, 20)):
        steps = np.array([ends[0], ends[1]])[(np.arange(pages) >= pages // 2).astype(int)], np.linspace(*ends, pages)
        for step in steps:
            scales[batch.table[0, :pages], 1, 0] = 2.0 ** (step if order == "rising" else step[::-1])
            check_scaled(g, batch, 1, 4, 64, codes, scales, rng.standard_normal((qlen, 4, 64)), 0.125,
                         workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("qlens", [[1, 2], [5, 6], [40, 30]])
def test_cache_least_scales_alone(g, qlens):  # noqa: F811
    rng = np.random.default_rng(1)
    batch = Batch(rng, qlens, [300, 200], 16)
    codes = random_codes(rng, (batch.nb, 2, 16, 1, 64))
    scales = np.full((batch.nb, 2, 1), 2.0 ** -9, np.float32)
    scales[:, 1] = (2.0 ** -rng.integers(96, 101, (batch.nb, 1))).astype(np.float32)
    check_scaled(g, batch, 1, 4, 64, codes, scales, rng.standard_normal((batch.T, 4, 64)), 0.125)


# ---------------------------------------------------------------------------
# pages of codes and scales
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("sizes", [[(96, np.uint8), (24, np.float32)], [(40, np.uint8), (7, np.uint8), (16, np.uint8)], [(3, np.float32)] * 2])
@pytest.mark.parametrize("rows,nb,bs,stride", [(5, 20, 4, 6), (40, 200, 16, 9), (300, 3000, 1, 30)])
def test_pages_of_several_geometries(g, sizes, rows, nb, bs, stride):  # noqa: F811
    """Copies, forks and compactions of pages whose bytes lie in arrays of
    different sizes and types, several of each, against the plain model."""
    rng = np.random.default_rng(rows + len(sizes))
    state = random_state(rng, rows, nb, bs, stride)
    caches = [rng.integers(0, 100, (nb, n)).astype(t) for n, t in sizes + sizes[::-1]]
    n = rows + 5
    parents, children = (rng.integers(-2, rows + 2, n).astype(np.int32) for _ in range(2))
    gpu = [dev(c) for c in caches]
    src, dst = np.arange(nb, dtype=np.int32)[:nb // 2], np.arange(nb, dtype=np.int32)[nb // 2:][:nb // 2]
    g.copy_pages(gpu, dev(src), dev(dst))
    for c, x in zip(gpu, caches):
        x[dst] = x[src]
        assert np.array_equal(host(c), x)
    state = check_pages(lambda t, l, r, c: g.fork_requests(c, bs, t, l, r, dev(parents), dev(children)),
                        lambda t, l, r, c: pages_ref.fork(t, l, r, parents, children, bs, c), state, caches)
    gone = rng.integers(-1, rows + 1, rows // 2).astype(np.int32)
    state = check_pages(lambda t, l, r, c: g.free_requests(bs, t, l, r, dev(gone)),
                        lambda t, l, r, c: pages_ref.free(t, l, r, gone, bs), state, caches)
    check_pages(lambda t, l, r, c: g.compact_pages(c, bs, t, l, r), lambda t, l, r, c: pages_ref.compact(t, l, r, bs, c), state, caches)


def test_pages_of_several_geometries_refusals(g):  # noqa: F811
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = torch.zeros(4, 8, device="cuda"), torch.zeros(5, 16, device="cuda")
    for bad in ([a, b], [a, torch.zeros(4, 16)], [a, torch.zeros(4, 16, device="cuda").expand(2, 4, 16)[0], b[:4].t().contiguous().t()], []):
        with pytest.raises(ValueError):
            g.copy_pages(bad, i, i)


@pytest.mark.parametrize("inside", [False, True])
def test_cache_pages_fork_and_compact(g, inside):  # noqa: F811
    """Forked and compacted pages of the 8-bit cache keep their values, with the
    scales as a second array or inside the pages; the fork's appends leave its
    parent alone; all of it in a captured graph too."""
    rng = np.random.default_rng(41)
    hq, hk, hs, bs, nb = 4, 2, 64, 16, 24
    codes = 2 * bs * hk * hs
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if inside:
        pool = torch.full((nb, codes + 16 * hk), 0xFF, dtype=torch.uint8, device="cuda")
        cache = pool[:, :codes].unflatten(1, (2, bs, hk, hs))
        scales = pool[:, codes:codes + 8 * hk].view(torch.float32).unflatten(1, (2, hk))
        moved = pool
    else:
        cache = torch.full((nb, 2, bs, hk, hs), 0xFF, dtype=torch.uint8, device="cuda")
        scales = torch.full((nb, 2, hk), float("nan"), device="cuda")
        moved = [cache, scales]
    table = torch.full((4, 6), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(nb, dtype=torch.int32, device="cuda")
    state = (bs, table, lens, refs)

    def append(row, n, size):
        old = int(lens[row])
        assert int(g.extend_requests(*state, i32(row), i32(old + n))) == 1
        k, v = (ref.bf16(size * rng.standard_normal((n, hk, hs)))[0].cuda() for _ in range(2))
        g.rope_append_fp8_kv(None, k, v, cache, scales, table[row:row + 1], i32(0, n), lens[row:row + 1], None)

    q = ref.bf16(rng.standard_normal((1, hq, hs)))[0].cuda()

    def attend(row):
        return g.attention_fp8_kv(q, cache, scales, table[row:row + 1], i32(0, 1), lens[row:row + 1], 96, 0.125, return_lse=True)

    append(3, 40, 1.0)                                       # to be freed: a hole
    append(0, 37, 5.0)
    want = attend(0)
    assert g.fork_requests(moved, *state, i32(0, 0), i32(1, 2)).tolist() == [1, 1]
    for row in (1, 2):
        assert all(torch.equal(a, b) for a, b in zip(attend(row), want))
    append(1, 3, 100.0)                                      # the fork's partial page gets scales of its own
    forked = attend(1)
    assert not torch.equal(forked[0], want[0])
    for row in (0, 2):
        assert all(torch.equal(a, b) for a, b in zip(attend(row), want))
    g.free_requests(*state, i32(3))
    before = [x.clone() for x in (cache, scales, table, lens, refs)]
    g.compact_pages(moved, *state)
    for row, w in ((0, want), (1, forked), (2, want)):
        assert all(torch.equal(a, b) for a, b in zip(attend(row), w))
    after = [x.clone() for x in (cache, scales, table, lens, refs)]
    assert int(table.max()) < int(before[2].max())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.compact_pages(moved, *state)
    for _ in range(3):
        for x, y in zip((cache, scales, table, lens, refs), before):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(table, after[2]) and torch.equal(refs, after[4])
        live = refs > 0
        assert torch.equal(cache[live], after[0][live]) and torch.equal(scales[live], after[1][live])


# ---------------------------------------------------------------------------
# values that are not finite, in every form of the prompt kernel
# ---------------------------------------------------------------------------
def seen_specials(see, v):
    """What the weighted sum of each row and dim is where it sees values that are
    not finite (positive weights): +-infinity, or NaN of a NaN or of both."""
    up, down, nan = ((see.astype(float) @ x.astype(float)) > 0 for x in (v == np.inf, v == -np.inf, np.isnan(v)))
    some = up | down | nan
    return some, np.where(nan | (up & down), np.nan, np.where(up, np.inf, -np.inf))


FORMS = [(128, 128), (64, 64), (192, 128), (256, 256), (80, 80), (200, 136), (40, 64)]


@pytest.mark.parametrize("dk,dv", FORMS)
@pytest.mark.parametrize("qlens,klens,kw", [
    ([64, 40, 30], [64, 40, 30], {}), ([64, 40, 30], [64, 40, 30], dict(window=7, num_sinks=1)), ([90, 9], [70, 130], dict(causal=False)),
    ([3, 40], [2100, 900], {}), ([3, 40], [2100, 900], dict(causal=False)), ([33, 20], [64, 50], dict(accumulate=True)),
    ([3, 40], [2100, 900], dict(accumulate=True)),
])
def test_prompt_values_that_are_not_finite(g, dk, dv, qlens, klens, kw):  # noqa: F811
    """Rows that see an infinity get it with its sign, those that see a NaN or
    both signs a NaN, and no other row or dim changes; lse counts them as any
    key.  Keys split, joined with an earlier part, and behind a window."""
    rng = np.random.default_rng(dk + dv + sum(klens))
    hk, group, hq = 2, 2, 4
    qs, ks = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (qlens, klens))
    q, k = (ref.bf16(0.5 * rng.standard_normal((n, h, dk)))[0].cuda() for n, h in ((qs[-1], hq), (ks[-1], hk)))
    v, v64 = ref.bf16(rng.standard_normal((ks[-1], hk, dv)))
    kw = dict(kw)
    accumulate = kw.pop("accumulate", False)
    if accumulate:
        kw["causal"] = False
        old = ref.bf16(rng.standard_normal((qs[-1], hq, dv)))[0].cuda(), torch.zeros(int(qs[-1]), hq, device="cuda")

    def call(v):
        more = dict(out=old[0].clone(), lse=old[1].clone(), accumulate=True) if accumulate else {}
        return g.prompt_attention(q, k, v, dev(qs), dev(ks), max(klens), dk ** -0.5, return_lse=True, **kw, **more)

    want, want_lse = (x.double().cpu().numpy() for x in call(v.cuda()))
    for values in ((-np.inf,), (np.inf,), (np.nan,), (np.inf, -np.inf, np.nan)):
        x = v.clone()
        for at in rng.integers(0, ks[-1], 6):
            x[int(at), int(rng.integers(hk)), int(rng.integers(dv))] = float(rng.choice(values))
        for b in range(len(klens)):                          # where some rows see it, others not
            x[int(ks[b]) + klens[b] - qlens[b] // 2 - 1, b % hk, 3 + b] = float(values[-1])
            x[int(ks[b]) + klens[b] - qlens[b] // 2, b % hk, 3 + b] = float(values[0])
        x64 = x.double().numpy()
        out, lse = (y.double().cpu().numpy() for y in call(x.cuda()))
        for b, (n, m) in enumerate(zip(qlens, klens)):
            see = ref.causal(n, m, kw.get("window"), kw.get("num_sinks", 0)) if kw.get("causal", True) else np.ones((n, m), bool)
            rows, keys = slice(qs[b], qs[b + 1]), slice(ks[b], ks[b + 1])
            for h in range(hq):
                some, what = seen_specials(see, x64[keys, h // group])
                got = out[rows, h]
                assert np.array_equal(got[some], what[some], equal_nan=True), (values, b, h)
                # a finite sum elsewhere: two calls differ by their roundings of weights (2^-8, where the tile is computed
                # another way) and of the output
                near = 2.0 ** -6 * (np.abs(want[rows, h]) + 1)
                close(got[~some], want[rows, h][~some], near[~some], f"{values} request {b} head {h}")
        close(lse, want_lse, 1e-5 * (np.abs(np.where(np.isfinite(want_lse), want_lse, 0)) + 1), f"{values} lse")


def test_prompt_rows_that_see_a_nan(g):  # noqa: F811
    """A NaN row of keys or values reaches every dim of every row that sees it."""
    rng = np.random.default_rng(9)
    for dk, dv in FORMS:
        q, k, v = (ref.bf16(rng.standard_normal((70, 2, d)))[0].cuda() for d in (dk, dk, dv))
        starts = dev(np.array([0, 40, 70], np.int32))
        want, lse = g.prompt_attention(q, k, v, starts, starts, 40, dk ** -0.5, return_lse=True)
        see = torch.zeros(70, dtype=torch.bool, device="cuda")
        see[30:40] = True
        for x in (k, v):
            y = x.clone()
            y[30] = float("nan")
            got, got_lse = g.prompt_attention(q, y if x is k else k, y if x is v else v, starts, starts, 40, dk ** -0.5, return_lse=True)
            assert torch.isnan(got[see]).all() and torch.equal(got[~see], want[~see]), (dk, dv)
            assert torch.isnan(got_lse[see]).all() if x is k else torch.equal(got_lse, lse), (dk, dv)
            assert torch.equal(got_lse[~see], lse[~see])


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_append_refuses_a_cache_without_heads(g):  # noqa: F811
    """No kernel would write the queries that the call returns."""
    x = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    cache, scales = x(3, 2, 16, 0, 64, t=torch.uint8), x(3, 2, 0, t=torch.float32)
    with pytest.raises(ValueError):
        g.rope_append_fp8_kv(x(5, 4, 64), x(5, 0, 64), x(5, 0, 64), cache, scales, x(1, 4, t=torch.int32), x(2, t=torch.int32),
                             x(1, t=torch.int32), None)


# ---------------------------------------------------------------------------
# every form that a call's sizes select
# ---------------------------------------------------------------------------
FORM_CASES = [  # rows of a tile, query lengths, lengths, group, head size
    (16, [1, 2, 1], [60, 45, 300], 4, 64), (16, [1, 2, 1], [60, 45, 300], 4, 128), (16, [5, 9, 2], [60, 45, 300], 2, 256),
    (32, [4, 7, 3], [60, 45, 300], 4, 64), (32, [4, 7, 3], [60, 45, 300], 4, 128), (32, [4, 7, 3], [60, 45, 300], 4, 96),
    (128, [33, 9, 70], [60, 9, 200], 2, 64), (128, [33, 9, 70], [60, 9, 200], 4, 256), (128, [33, 9, 70], [60, 9, 200], 2, 176),
    (128, [33, 9, 140], [60, 9, 900], 2, 256), (128, [33, 9, 70], [60, 9, 200], 4, 128), (128, [33, 9, 70], [60, 9, 200], 4, 80),
]


@pytest.mark.parametrize("kind", ["causal", "window", "tree"])
@pytest.mark.parametrize("bs", [16, 24])
@pytest.mark.parametrize("rows,qlens,lens,group,hs", FORM_CASES)
def test_cache_every_form(g, rows, qlens, lens, group, hs, bs, kind):  # noqa: F811
    """Both kernels at all their head sizes, over whole pages and others, causal,
    behind a window and with a tree mask."""
    rng = np.random.default_rng(rows + hs + bs)
    batch = Batch(rng, qlens, lens, bs)
    assert rows_kernel(batch.T + 2, len(qlens), group, hs) == rows
    mask = None
    if kind == "tree":
        mask = rng.random((batch.T, max(qlens))) < 0.4
        mask[int(batch.starts[1]) + 1] = False               # a row that sees its context alone, if there is any
    w, s = (40, 6) if kind == "window" else (None, 0)
    check_cache(g, rng, batch, 2, group, hs, "nhd", w, s, mask=mask)


def test_cache_every_form_is_there():
    """All head sizes of both kernels are among the cases above."""
    padded = lambda hs: 64 if hs <= 64 else 128 if hs <= 128 else 256  # noqa: E731
    assert {(r, padded(hs)) for r, _, _, _, hs in FORM_CASES} == {(16, 64), (16, 128), (16, 256), (32, 64), (32, 128), (128, 64), (128, 128),
                                                                  (128, 256)}


# ---------------------------------------------------------------------------
# other calls that the headers allow
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_without_any_keys(g, causal):  # noqa: F811
    """No key in the whole batch: zeros with lse -infinity, or what an earlier
    part left."""
    rng = np.random.default_rng(2)
    q = ref.bf16(rng.standard_normal((40, 4, 128)))[0].cuda()
    k = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    qs, ks = dev(np.array([0, 7, 40], np.int32)), torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = g.prompt_attention(q, k, k, qs, ks, 0, 0.1, causal=causal, return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    part, part_lse = ref.bf16(rng.standard_normal((40, 4, 128)))[0].cuda(), dev(rng.standard_normal((40, 4)).astype(np.float32))
    out, lse = part.clone(), part_lse.clone()
    g.prompt_attention(q, k, k, qs, ks, 0, 0.1, causal=causal, out=out, lse=lse, accumulate=True)
    assert torch.equal(out, part) and torch.equal(lse, part_lse)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bs", [16, 128, 1024])
def test_append_in_place_whatever_the_page(g, bs, inter):  # noqa: F811
    """k_out=k where a page's rows stay in registers and where they are read
    twice: the bits of a call with outputs of its own."""
    rng = np.random.default_rng(bs)
    hq, hk, hs, rot, lens = 4, 3, 64, 48, [1100, 40, 300]
    T, pages = sum(lens), [-(-n // bs) for n in lens]
    table = np.full((3, max(pages)), -1, np.int32)
    order = rng.permutation(sum(pages))
    for b, n in enumerate(pages):
        table[b, :n] = order[sum(pages[:b]):sum(pages[:b + 1])]
    qkv = ref.bf16(rng.standard_normal((T, hq + 2 * hk, hs)))[0].cuda()
    cs = dev(rng.standard_normal((1200, rot)).astype(np.float32))
    got = []
    for own in (True, False):
        x = qkv.clone()
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        cache = torch.zeros(sum(pages), 2, bs, hk, hs, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(sum(pages), 2, hk, device="cuda")
        starts = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
        out = g.rope_append_fp8_kv(q, k, v, cache, scales, dev(table), starts, dev(np.array(lens, np.int32)), cs, interleaved=inter,
                                   return_k=True, **({} if own else dict(q_out=q, k_out=k)))
        got.append((*out, cache, scales, v.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert torch.equal(got[0][4], qkv[:, hq + hk:])
