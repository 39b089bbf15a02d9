"""GPU tests of the 8-bit paged cache (append with rotation, attention) and of
the prompts' attention against plain 64-bit references (serving_refs.py), at
the sizes, layouts and masks where they can go wrong."""
import numpy as np
import pytest
import torch

import serving_refs as ref
from gpu_util import dev
from test_operators_gpu import Batch, close, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gather_concat_cache_amd as gc
    return gc


def cache_view(nb, bs, hk, hs, layout, fill=0xFF):
    """(flat bytes on the GPU, uint8 view [nb, 2, bs, hk, hs]) of one layout."""
    order = {"nhd": (nb, 2, bs, hk, hs), "hnd": (nb, 2, hk, bs, hs), "planes": (2, nb, bs, hk, hs),
             "wide": (nb, 2, bs, hk + 1, hs + 16)}[layout]
    flat = torch.full((int(np.prod(order)),), fill, dtype=torch.uint8, device="cuda")
    x = flat.view(order)
    if layout == "hnd":
        x = x.transpose(2, 3)
    if layout == "planes":
        x = x.transpose(0, 1)
    if layout == "wide":
        x = x[..., :hk, :hs]
    return flat, x


def random_codes(rng, shape):
    """e4m3 bytes of mixed sizes, no NaN code."""
    c = rng.integers(0, 0x7F, shape, dtype=np.uint8) | rng.integers(0, 2, shape, dtype=np.uint8) << 7
    return c


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
APPEND = [  # q heads, kv heads, head size, rot, interleaved, bf16 table, block, layout, qlens, lens
    (4, 2, 128, 128, False, False, 16, "nhd", [1, 0, 3, 17, 40, 1], [1, 5, 18, 33, 40, 116]),
    (8, 8, 64, 32, True, False, 16, "hnd", [5, 33, 1, 1], [37, 33, 16, 17]),
    (3, 1, 80, 48, False, True, 24, "wide", [70, 2, 1, 25], [70, 50, 25, 73]),
    (0, 3, 96, 96, True, True, 7, "planes", [9, 1, 1, 20], [9, 7, 8, 30]),
    (5, 5, 256, 256, False, False, 64, "nhd", [130, 1, 64], [140, 65, 64]),
    (12, 12, 16, 0, False, False, 1, "nhd", [3, 1, 4], [5, 1, 4]),
    (2, 1, 192, 64, True, False, 128, "hnd", [200, 100, 1], [333, 100, 129]),
    (16, 16, 128, 64, False, False, 48, "nhd", [60, 1, 47, 2], [70, 48, 47, 50]),
    (1, 1, 48, 16, False, False, 16, "nhd", [1] * 70, list(range(1, 71))),
    (64, 2, 128, 128, False, False, 16, "nhd", [1], [1000]),
    (2, 8, 128, 128, False, False, 128, "nhd", [150, 1, 129, 0, 3], [160, 129, 129, 4, 131]),
    (1, 2, 64, 0, False, False, 1024, "nhd", [1100, 1, 30], [1300, 1025, 31]),
]


def run_append(g, seed, hq, hk, hs, rot, inter, tab16, bs, layout, qlens, lens, keys=True, positions=None, edit=None,
               magnitude=None, cache=None):
    rng = np.random.default_rng(seed)
    batch = Batch(rng, qlens, lens, bs)
    if edit:
        edit(batch)
    nb, T = batch.nb, batch.T
    flat, view = cache_view(nb, bs, hk, hs, layout) if cache is None else cache
    was = random_codes(rng, (nb, 2, bs, hk, hs))
    view.copy_(dev(was))
    scales0 = (rng.uniform(0.5, 6.0, (nb, 2, hk)) / 448).astype(np.float32)
    scales = dev(scales0)
    before_flat = flat.clone()
    mags = 1.0 if magnitude is None else magnitude
    qkv, x64 = ref.bf16(rng.standard_normal((T + 2, hq + 2 * hk + 1, hs)) * mags)
    qkv = qkv.cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:hq + 2 * hk]
    ang = np.arange(200)[:, None] * 3.0 ** -np.arange(rot // 2)
    table = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))
    table = table.to(torch.bfloat16) if tab16 else table
    tab = table.to(torch.float64).numpy()
    bt, starts, dlens = batch.metadata()
    q_out = torch.full((T + 2, hq, hs), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((T + 2, hk, hs), 7.0, dtype=torch.bfloat16, device="cuda")
    args = (bt, starts, dlens, None if rot == 0 else table.cuda())
    kw = dict(positions=None if positions is None else dev(positions), interleaved=inter)
    qo, ko = g.rope_append_fp8_kv(q if hq else None, k, v, view, scales, *args, q_out=q_out if hq else None,
                                  k_out=k_out if keys else None, **kw)
    torch.cuda.synchronize()
    assert (qo is q_out) == (hq > 0) and (ko is k_out) == keys
    # rotated rows
    r = np.zeros(T + 2, np.int64)
    for b, (n, m) in enumerate(zip(qlens, lens)):
        s = int(batch.starts[b])
        r[s:s + n] = max(m, 0) - n + np.arange(n)
    if positions is not None:
        r = positions
    for out, x, what in ((q_out, x64[:, :hq], "q"), (k_out, x64[:, hq:hq + hk], "k")):
        assert (out[T:] == 7).all(), f"{what}: rows behind the last request were written"
        if (what == "q" and hq) or (what == "k" and keys):
            want, mag = ref.rotate(x, r, tab, rot, inter)
            close(out[:T], want[:T], (2.0 ** -8 * np.abs(want) + 2.0 ** -22 * mag + 1e-37)[:T], what)
    # the cache against 64-bit values.  A code is off by half an e4m3 step (2^-4 of the value, 2^-10 of the scale below the
    # normal range), a scale by 2^-22, a rotated value by 2^-22 of what meets in it
    kt, kmag = ref.rotate(x64[:, hq:hq + hk], r, tab, rot, inter)
    v64 = x64[:, hq + hk:hq + 2 * hk]
    want_c, want_s = ref.e4m3(was), scales0.astype(np.float64)
    wrote, scaled, shrunk = ref.append(want_c, want_s, kt, v64, batch.table, batch.starts, batch.lens, bs)
    got_s = scales.cpu().numpy().astype(np.float64)
    assert (got_s == scales0)[~scaled].all(), "a scale without a new token changed"
    close(got_s[scaled], want_s[scaled], 2.0 ** -21 * want_s[scaled], "scales")
    got = view.cpu().numpy()
    same = ~wrote & ~shrunk
    assert (got == was)[same].all(), "an older entry changed without its scale"
    got_c = ref.e4m3(got)
    close(got_c[shrunk], want_c[shrunk], 0, "older codes")
    value = (got_c * got_s[:, :, None, :, None])[wrote]
    true = np.zeros(got_c.shape)
    mag = np.zeros(got_c.shape)
    for b, (n, m) in enumerate(zip(qlens, lens)):
        for i in range(n):
            pos, t = max(m, 0) - n + i, int(batch.starts[b]) + i
            if pos >= 0 and pos // bs < batch.table.shape[1] and 0 <= batch.table[b, pos // bs] < nb:
                true[batch.table[b, pos // bs], :, pos % bs] = np.stack([kt[t], v64[t]])
                mag[batch.table[b, pos // bs], :, pos % bs] = np.stack([kmag[t], np.abs(v64[t])])
    step = np.broadcast_to((got_s * 2.0 ** -10)[:, :, None, :, None], got_c.shape)[wrote]
    close(value, true[wrote], 1.001 * (2.0 ** -4 * np.abs(true[wrote]) + step) + 2.0 ** -20 * mag[wrote], "entries")
    # and against the definition's own binary32 operations, bit for bit
    x32 = x64.astype(np.float32)
    k32 = ref.rotate(x32[:, hq:hq + hk], r, tab.astype(np.float32), rot, inter)[0]
    want_c, want_s = ref.e4m3(was), scales0.copy()
    ref.append(want_c, want_s, k32, x32[:, hq + hk:hq + 2 * hk], batch.table, batch.starts, batch.lens, bs)
    close(got_c, want_c, 0, "codes")
    assert (got_s == want_s).all(), "scales"
    # bytes outside the pages' rows
    now = flat.clone()
    view.copy_(dev(was))
    assert torch.equal(flat, before_flat), "bytes outside the entries changed"
    flat.copy_(now)
    return dict(q=qo, k=ko, scales=scales, view=view, batch=batch, inputs=(q, k, v), args=args, kw=kw, was=was, scales0=scales0)


@pytest.mark.parametrize("case", APPEND)
def test_append(g, case):
    run_append(g, 1, *case)


def test_append_in_place_and_without_keys(g):
    """q_out=q and k_out=k give the same bits; without k_out the cache is the same."""
    case = (8, 2, 128, 64, False, False, 16, "nhd", [40, 1, 3], [50, 17, 3])
    a = run_append(g, 5, *case)
    b = run_append(g, 5, *case, keys=False)
    assert torch.equal(a["view"], b["view"]) and torch.equal(a["scales"], b["scales"]) and torch.equal(a["q"], b["q"])
    q, k, v = b["inputs"]
    b["view"].copy_(dev(b["was"]))
    b["scales"].copy_(dev(b["scales0"]))
    g.rope_append_fp8_kv(q, k, v, b["view"], b["scales"], *b["args"], q_out=q, k_out=k, **b["kw"])
    T = b["batch"].T
    assert torch.equal(a["view"], b["view"]) and torch.equal(q[:T], a["q"][:T]) and torch.equal(k[:T], a["k"][:T])


@pytest.mark.parametrize("bs", [16, 64, 160])
def test_append_positions_of_their_own(g, bs):
    """Rotation rows from `positions`, some outside the table, whatever the
    cache positions are."""
    rng = np.random.default_rng(2)
    pos = rng.integers(-2, 203, 47)
    run_append(g, 2, 4, 2, 64, 64, False, False, bs, "nhd", [30, 15], [200, 15], positions=pos)


def test_append_missing_pages(g):
    """Ids outside the cache, table rows that are too short and positions below
    zero: the cache keeps its bytes, the rotated rows are written."""
    def edit(batch):
        batch.table[0, 1] = -1
        batch.table[0, 3] = batch.nb
        batch.table[1, :] = 1 << 30
    run_append(g, 3, 4, 2, 64, 32, False, False, 16, "nhd", [60, 5, 9, 3], [70, 33, 4, -2], edit=edit)


def test_append_magnitudes(g):
    """Zeros, tiny and huge tokens; a page's scale that has to grow far."""
    mags = np.ones((47, 1, 1))
    mags[0:8] = 0.0
    mags[8:16] = 1e-38
    mags[20] = 1e37
    mags[33:36] = 1e-20
    run_append(g, 4, 2, 2, 32, 0, False, False, 16, "nhd", [30, 15], [35, 15], magnitude=mags)


def test_append_token_by_token(g):
    """A page filled one token a call: every older code is divided by powers of
    two only, so each entry is within half a step of its own first scale and of
    the subnormal steps since."""
    rng = np.random.default_rng(9)
    T, hk, hs, bs = 33, 2, 64, 16
    k, k64 = ref.bf16(rng.standard_normal((T, hk, hs)) * 2.0 ** rng.uniform(-3, 6, (T, 1, 1)))
    v, v64 = ref.bf16(rng.standard_normal((T, hk, hs)) * 2.0 ** rng.uniform(-3, 6, (T, 1, 1)))
    k, v = k.cuda(), v.cuda()
    table = dev(np.array([[2, 0, 1]], np.int32))
    cache = torch.full((3, 2, bs, hk, hs), 0xFF, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.full((3, 2, hk), float("nan"), device="cuda")
    starts = dev(np.array([0, 1], np.int32))
    for t in range(T):
        g.rope_append_fp8_kv(None, k[t:t + 1], v[t:t + 1], cache, scales, table, starts, dev(np.array([t + 1], np.int32)), None)
    s = scales.double().cpu().numpy()
    c = ref.e4m3(cache.view(torch.uint8).cpu().numpy())
    for t in range(T):
        blk = [2, 0, 1][t // bs]
        for side, x in enumerate((k64[t], v64[t])):
            sc = s[blk, side][:, None]
            assert (np.abs(x).max(1) <= 448 * sc[:, 0] * (1 + 2.0 ** -20)).all()
            # subnormal roundings: each at most half of the smallest step at the scale of its time, a geometric sum
            close(c[blk, side, t % bs] * sc, x, 1.001 * (2.0 ** -4 * np.abs(x) + 2 * 2.0 ** -10 * sc), f"token {t}")


def test_append_on_a_stream_and_captured(g):
    """The same bits from another stream and from a replayed graph."""
    case = (8, 2, 128, 128, False, False, 16, "nhd", [20, 1, 5], [50, 17, 5])
    a = run_append(g, 6, *case)
    q, k, v = a["inputs"]
    view, scales = torch.empty_like(a["view"]), torch.empty_like(a["scales"])
    was, s0 = dev(a["was"]), dev(a["scales0"])
    T = a["batch"].T

    def call(stream=None):
        view.copy_(was)
        scales.copy_(s0)
        return g.rope_append_fp8_kv(q, k, v, view, scales, *a["args"], **a["kw"], return_k=True, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        view.copy_(was)
        scales.copy_(s0)
    qo, ko = g.rope_append_fp8_kv(q, k, v, view, scales, *a["args"], **a["kw"], return_k=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = a["view"].clone()
    assert torch.equal(view, want) and torch.equal(qo[:T], a["q"][:T]) and torch.equal(ko[:T], a["k"][:T])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qo, ko = call()
    for _ in range(3):
        view.zero_()
        qo.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(view, want) and torch.equal(scales, a["scales"]) and torch.equal(qo[:T], a["q"][:T])


# ---------------------------------------------------------------------------
# attention over the cache
# ---------------------------------------------------------------------------
def check_cache(g, rng, batch, hk, group, hs, layout="nhd", window=None, sinks=0, mask=None, max_seq_len=None, workspace=None,
                pad=0, scale=None, spread=1.0, stream=None):
    nb, bs = batch.nb, batch.bs
    flat, view = cache_view(nb, bs, hk, hs, layout)
    bytes_ = np.full((nb, 2, bs, hk, hs), 0xFF, np.uint8)      # the NaN code where nothing was written
    scales = np.full((nb, 2, hk), np.nan, np.float32)
    for b, n in enumerate(batch.lens):
        for p in range(max(n, 0)):
            blk = int(batch.table[b, p // bs]) if p // bs < batch.table.shape[1] else -1
            if 0 <= blk < nb:
                bytes_[blk, :, p % bs] = random_codes(rng, (2, hk, hs))
                if p % bs == 0:
                    scales[blk] = 2.0 ** rng.uniform(-9 - spread, -9 + spread, (2, hk))
    view.copy_(dev(bytes_))
    q, q64 = queries(rng, batch.T + 2, hk * group, hs, pad)
    bt, starts, lens = batch.metadata()
    scale = hs ** -0.5 if scale is None else scale
    out = torch.full((batch.T + 2, hk * group, hs), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((batch.T + 2, hk * group), 7.0, device="cuda")
    longest = max(list(batch.lens) + [1]) if max_seq_len is None else max_seq_len
    full_mask = None
    if mask is not None:
        full_mask = np.zeros((batch.T + 2, mask.shape[1]), bool)
        full_mask[:batch.T] = mask
    dsc = dev(scales)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    g.attention_fp8_kv(q, view, dsc, bt, starts, lens, longest, scale, window=window, num_sinks=sinks,
                       tree_mask=None if mask is None else dev(full_mask), out=out, lse=lse, return_lse=True,
                       workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    assert (out[batch.T:] == 7).all() and (lse[batch.T:] == 7).all(), "rows behind the last sequence were written"
    scale32 = float(np.float32(scale))
    value = ref.e4m3(bytes_) * scales.astype(np.float64)[:, :, None, :, None]
    for b, (n, length) in enumerate(zip(batch.qlens, batch.lens)):
        r0, m = int(batch.starts[b]), max(length, 0)
        see = ref.causal(n, m, window, sinks) if mask is None else ref.tree(n, m, mask[r0:r0 + n])
        at = np.arange(m)
        blk = batch.table[b][np.minimum(at // bs, batch.table.shape[1] - 1)]
        ok = (at // bs < batch.table.shape[1]) & (blk >= 0) & (blk < nb)
        blk = np.where(ok, blk, 0)
        vis = np.repeat(see & ok[None], group, 0)
        for h in range(hk):
            k, v = (np.nan_to_num(value[blk, side, at % bs, h], nan=0.0) for side in (0, 1))
            vs = np.nan_to_num(scales[blk, 1, h].astype(np.float64), nan=0.0)
            rows = q64[r0:r0 + n, h * group:(h + 1) * group].reshape(-1, hs)
            # weights in binary16: half a step is 2^-11; below its normal range they are off by 2^-25 where the row's largest
            # is at least 2^6, and meet codes up to 448 of the largest scale
            o, l, ot, lt = ref.attend(rows, k, v, vis, scale32, 2.0 ** -11, 2.0 ** -31 * 448 * (vs * ok).max(initial=0.0))
            close(out[r0:r0 + n, h * group:(h + 1) * group].reshape(-1, hs), o, ot, f"request {b} head {h} out")
            close(lse[r0:r0 + n, h * group:(h + 1) * group].reshape(-1), l, lt, f"request {b} head {h} lse")
    return out, lse


CACHE = [  # kv heads, group, head size, block, layout, window, sinks
    (1, 1, 16, 16, "nhd", None, 0), (2, 4, 64, 16, "nhd", 8, 2), (1, 3, 80, 24, "wide", 33, 5),
    (2, 2, 128, 16, "hnd", 40, 4), (1, 8, 128, 64, "planes", 1, 0), (2, 1, 176, 16, "wide", 64, 40),
    (1, 4, 256, 32, "nhd", 17, 1), (3, 2, 96, 1, "nhd", 50, 3), (1, 16, 128, 7, "hnd", 1000, 4),
    (1, 20, 64, 16, "planes", 5, 100), (2, 5, 48, 40, "hnd", None, 0), (1, 2, 240, 5, "nhd", 9, 2),
    (4, 8, 128, 16, "nhd", 31, 33), (1, 1, 112, 48, "nhd", 32, 32), (8, 1, 256, 128, "nhd", None, 0),
]


@pytest.mark.parametrize("hk,group,hs,bs,layout,window,sinks", CACHE)
def test_cache_attention(g, hk, group, hs, bs, layout, window, sinks):
    """Decode, short chunks and long ones in one batch; lengths of zero, one,
    around the tile and page borders; a query longer than its sequence."""
    rng = np.random.default_rng(hs + bs)
    batch = Batch(rng, [1, 0, 3, 1, 40, 1, 5, 2], [1, 9, 3, 33, 75, 130, 2, 0], bs)
    check_cache(g, rng, batch, hk, group, hs, layout, window, sinks)


@pytest.mark.parametrize("qlens,lens", [([1] * 9, [1, 15, 16, 17, 31, 32, 33, 64, 200]), ([130], [130]), ([70, 1, 64], [300, 5, 64]),
                                        ([2] * 20, list(range(2, 42, 2))), ([1], [700]), ([5, 3], [400, 90]), ([9], [150])])
@pytest.mark.parametrize("window,sinks", [(None, 0), (20, 4), (64, 0)])
def test_cache_attention_lengths(g, qlens, lens, window, sinks):
    rng = np.random.default_rng(len(lens))
    batch = Batch(rng, qlens, lens, 16)
    check_cache(g, rng, batch, 2, 4, 128, "nhd", window, sinks, pad=24)


@pytest.mark.parametrize("hs,bs", [(128, 16), (64, 24), (256, 16), (64, 16)])
def test_cache_key_split_and_workspace(g, hs, bs):
    """Keys split over many workgroups, over few (a small or no workspace), and
    sequences longer than max_seq_len says: all within the bounds."""
    for ws, longest in ((None, 2100), (None, 300), (None, 5), (0, 2100), (200000, 2100)):
        rng = np.random.default_rng(5)
        batch = Batch(rng, [1, 4, 2], [2100, 900, 40], bs)
        workspace = None if ws is None else torch.empty(ws, dtype=torch.uint8, device="cuda")
        check_cache(g, rng, batch, 1, 2, hs, max_seq_len=longest, workspace=workspace)


@pytest.mark.parametrize("bs", [16, 24])
def test_cache_scales_far_apart(g, bs):
    """Pages whose scales differ by 2^40 and more, K and V: weights keep their
    precision at every scale."""
    rng = np.random.default_rng(17)
    batch = Batch(rng, [1, 20, 3], [300, 130, 90], bs)
    check_cache(g, rng, batch, 2, 2, 64, spread=20.0)


def test_cache_hidden_pages_and_holes(g):
    rng = np.random.default_rng(3)
    batch = Batch(rng, [2, 1, 3, 40], [90, 50, 64, 90], 16)
    for b in (0, 3):
        batch.table[b, 2] = -1
        batch.table[b, 4] = batch.nb
    batch.table[1, :] = -1
    out, lse = check_cache(g, rng, batch, 2, 2, 64, window=60, sinks=3)
    assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()


@pytest.mark.parametrize("hk,group,hs,bs", [(2, 4, 128, 16), (1, 1, 64, 24), (1, 7, 80, 16), (1, 2, 256, 8)])
def test_cache_tree(g, hk, group, hs, bs):
    """Trees, an arbitrary mask, rows whose mask leaves nothing but the
    context, and (no context) nothing at all."""
    rng = np.random.default_rng(hs)
    qlens, lens = [8, 1, 33, 5, 12, 3], [60, 1, 33, 5, 140, 2]
    batch = Batch(rng, qlens, lens, bs)
    mask = rng.random((batch.T, 33)) < 0.4
    r0 = int(batch.starts[3])
    mask[r0 + 1] = False
    out, lse = check_cache(g, rng, batch, hk, group, hs, mask=mask)
    assert (out[r0 + 1] == 0).all() and torch.isneginf(lse[r0 + 1]).all()
    check_cache(g, rng, batch, hk, group, hs, mask=mask[:, :9])
    check_cache(g, rng, batch, hk, group, hs, mask=mask[:, :0])


def test_cache_large_batch(g):
    """More requests than are counted and split."""
    rng = np.random.default_rng(21)
    lens = rng.integers(1, 40, 530)
    batch = Batch(rng, rng.integers(1, 3, 530), lens + 2, 16)
    check_cache(g, rng, batch, 1, 2, 64)


def test_cache_on_a_stream_negative_and_zero_scale(g):
    rng = np.random.default_rng(13)
    batch = Batch(rng, [3, 1, 40], [50, 20, 60], 16)
    check_cache(g, rng, batch, 1, 2, 64, scale=-0.2, stream=torch.cuda.Stream())
    check_cache(g, rng, batch, 1, 2, 64, scale=0.0, window=9, sinks=1)


@pytest.mark.parametrize("window,sinks", [(None, 0), (900, 40)])
@pytest.mark.parametrize("bs", [16, 40])
def test_cache_long_chunks(g, bs, window, sinks):
    """Chunks of several row tiles over lengths that differ."""
    rng = np.random.default_rng(23)
    batch = Batch(rng, [300, 0, 700, 129], [1100, 5, 1900, 129], bs)
    check_cache(g, rng, batch, 1, 2, 64, window=window, sinks=sinks)


def small_cache(rng, nb, bs, hk, hs):
    codes = dev(random_codes(rng, (nb, 2, bs, hk, hs)))
    return codes, dev((2.0 ** rng.uniform(-10, -8, (nb, 2, hk))).astype(np.float32))


@pytest.mark.parametrize("bs", [16, 24])
def test_cache_captured(g, bs):
    """Append and attention (keys split, so the join is in it) in one graph:
    every replay gives the eager bits for the inputs of its time."""
    rng = np.random.default_rng(24)
    hk, hq, hs, nb = 2, 8, 128, 300
    cache, scales = small_cache(rng, nb, bs, hk, hs)
    view = cache.view(torch.float8_e4m3fn)
    was, was_scales = cache.clone(), scales.clone()
    table = dev(rng.permutation(nb).astype(np.int32)[:2 * 140].reshape(2, 140))
    starts, lens = dev(np.array([0, 1, 4], np.int32)), dev(np.array([1800, 2203], np.int32))
    q, k, v = (ref.bf16(rng.standard_normal((4, h, hs)))[0].cuda() for h in (hq, hk, hk))

    def call():
        qr, _ = g.rope_append_fp8_kv(q, k, v, view, scales, table, starts, lens, None)
        return g.attention_fp8_kv(qr, view, scales, table, starts, lens, 2203, 0.09, return_lse=True)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = call()
    for i in range(3):
        for x in (q, k, v):
            x.mul_(0.5 + i)
        lens.sub_(dev(np.array([i, 40 * i], np.int32)))
        cache.copy_(was)
        scales.copy_(was_scales)
        want, want_lse = call()
        state = cache.clone(), scales.clone()
        cache.copy_(was)
        scales.copy_(was_scales)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert torch.equal(cache, state[0]) and torch.equal(scales, state[1])


@pytest.mark.parametrize("bs", [16, 24])
def test_cache_behind_4_gib(g, bs):
    """Pages whose bytes lie behind 2^32 give the bits of pages at the start,
    in append and in both kinds of attention."""
    rng = np.random.default_rng(25)
    hk, hq, hs, nb = 8, 16, 128, 12
    cache, scales = small_cache(rng, nb, bs, hk, hs)
    far = (5 << 30) // (2 * bs * hk * hs)
    big = torch.empty((far + nb, 2, bs, hk, hs), dtype=torch.uint8, device="cuda")
    big_scales = torch.empty((far + nb, 2, hk), device="cuda")
    big[far:], big_scales[far:] = cache, scales
    near = dev(rng.permutation(nb).astype(np.int32).reshape(2, 6))
    lens = dev(np.array([90, 95], np.int32))
    for starts in ([0, 1, 3], [0, 70, 101]):
        T = starts[-1]
        starts = dev(np.array(starts, np.int32))
        q, k, v = (ref.bf16(rng.standard_normal((T, h, hs)))[0].cuda() for h in (hq, hk, hk))
        got = []
        for c, s, t in ((cache, scales, near), (big, big_scales, near + far)):
            g.rope_append_fp8_kv(None, k, v, c, s, t, starts, lens, None)
            got.append(g.attention_fp8_kv(q, c, s, t, starts, lens, 95, 0.09, return_lse=True))
        assert torch.equal(big[far:], cache) and torch.equal(big_scales[far:], scales)
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_cache_lengths_behind_the_table(g):
    """seq_lens that claim up to 2^31 - 1 keys, of which the table has 64: the
    bits of a sequence that ends there, with many heads a key head."""
    rng = np.random.default_rng(27)
    cache, scales = small_cache(rng, 8, 16, 1, 64)
    table = dev(rng.permutation(8).astype(np.int32).reshape(2, 4))
    starts = dev(np.array([0, 1, 3], np.int32))
    q = ref.bf16(rng.standard_normal((3, 256, 64)))[0].cuda()
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    got = [g.attention_fp8_kv(q, cache, scales, table, starts, dev(np.array([n, 40], np.int32)), 4096, 0.1, return_lse=True, workspace=none)
           for n in (64, 2 ** 31 - 1)]
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_calls_on_two_streams_at_once(g):
    """Two calls of each attention in flight together, each with its own
    workspace (allocated by the call), give the bits of one alone."""
    rng = np.random.default_rng(26)
    hk, hq, hs, bs, nb = 2, 8, 128, 16, 512
    cache, scales = small_cache(rng, nb, bs, hk, hs)
    one, lens = dev(np.array([0, 2], np.int32)), dev(np.array([4000], np.int32))
    tables = [dev(rng.permutation(nb).astype(np.int32)[None, :256].copy()) for _ in range(2)]
    qs = [ref.bf16(rng.standard_normal((2, hq, hs)))[0].cuda() for _ in range(2)]
    k, v = (ref.bf16(rng.standard_normal((4000, hk, hs)))[0].cuda() for _ in range(2))

    def calls(i, stream=None):
        return [g.attention_fp8_kv(qs[i], cache, scales, tables[i], one, lens, 4000, 0.09, stream=stream),
                g.prompt_attention(qs[i], k, v, one, dev_keys, 4000, 0.09, stream=stream)]

    dev_keys = dev(np.array([0, 4000], np.int32))
    want = [calls(i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[calls(i, streams[i]) for i in range(2)] for _ in range(10)]
    torch.cuda.synchronize()
    for both in got:
        for a, b in zip(both, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_argument_refusals(g):
    """What the binding refuses, with the tensors on the GPU."""
    x = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    cache, scales = x(3, 2, 16, 2, 64, t=torch.uint8), x(3, 2, 2, t=torch.float32)
    table, starts, lens = x(1, 4, t=torch.int32), x(2, t=torch.int32), x(1, t=torch.int32)
    q, k = x(5, 4, 64), x(5, 2, 64)
    paged = (cache, scales, table, starts, lens)
    bad = [
        lambda: g.attention_fp8_kv(q, *paged, 4, 1.0, window=3, tree_mask=x(5, 2, t=torch.bool)),
        lambda: g.attention_fp8_kv(q, *paged, 4, 1.0, window=0),
        lambda: g.attention_fp8_kv(x(5, 3, 64), *paged, 4, 1.0),
        lambda: g.attention_fp8_kv(q, cache, scales[:2], table, starts, lens, 4, 1.0),
        lambda: g.attention_fp8_kv(q, cache, scales, table, lens, lens, 4, 1.0),
        lambda: g.attention_fp8_kv(q, *paged, 4, float("nan")),
        lambda: g.attention_fp8_kv(q, *paged, 4, 1.0, out=x(5, 4, 32)),
        lambda: g.rope_append_fp8_kv(None, k, k, *paged, None, q_out=q),
        lambda: g.rope_append_fp8_kv(q, k, k[:4], *paged, None),
        lambda: g.rope_append_fp8_kv(q, k[..., ::2], k[..., ::2], *paged, None),
        lambda: g.rope_append_fp8_kv(q, k, k, *paged, x(9, 80, t=torch.float32)),
        lambda: g.rope_append_fp8_kv(q, k, k, *paged, x(9, 24, t=torch.float32)),
        lambda: g.rope_append_fp8_kv(q, k, k, *paged, None, positions=x(4, t=torch.int64)),
        lambda: g.rope_append_fp8_kv(q, k, k, cache[:1].expand(3, -1, -1, -1, -1), *paged[1:], None),
        lambda: g.prompt_attention(q, k, k, starts, starts, 5, 1.0, accumulate=True),
        lambda: g.prompt_attention(q, k, k, starts, starts, 5, 1.0, causal=False, window=4),
        lambda: g.prompt_attention(q, k, k, starts, lens, 5, 1.0),
        lambda: g.prompt_attention(q, k, k[:4], starts, starts, 5, 1.0),
        lambda: g.prompt_attention(q, k, k, starts, starts, -1, 1.0),
        lambda: g.prompt_attention(q, x(5, 3, 64), x(5, 3, 64), starts, starts, 5, 1.0),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, RuntimeError)):
            call()
            pytest.fail(f"call {i} was taken")


# ---------------------------------------------------------------------------
# prompts
# ---------------------------------------------------------------------------
def check_prompt(g, rng, qlens, klens, hk, group, dk, dv, causal=True, window=None, sinks=0, max_key_len=None, workspace=None,
                 fused=False, scale=None, accumulate=False, edit=None, stream=None):
    qs, ks = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (qlens, klens))
    T, Tk, hq = int(qs[-1]), int(ks[-1]), hk * group
    def rows(n, h, d):
        return rng.standard_normal((n, h, d)) * 10.0 ** rng.uniform(-1, 0.3, (n, h, 1))
    if fused:                                                # one projection's output, queries, keys and values side by side
        t, x = ref.bf16(rows(T + 2, hq + 2 * hk, dk))
        t = t.cuda()
        q, k, v = t[:, :hq], t[:T, hq:hq + hk], t[:T, hq + hk:]
        q64, k64, v64 = x[:, :hq], x[:T, hq:hq + hk], x[:T, hq + hk:]
    else:
        (q, q64), (k, k64), (v, v64) = (ref.bf16(rows(n, h, d)) for n, h, d in ((T + 2, hq, dk), (Tk, hk, dk), (Tk, hk, dv)))
        if edit:
            edit(k, v)
            k64, v64 = k.double().numpy(), v.double().numpy()
        q, k, v = q.cuda(), k.cuda(), v.cuda()
    scale = dk ** -0.5 if scale is None else scale
    out = torch.full((T + 2, hq, dv), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 2, hq), 7.0, device="cuda")
    if accumulate:
        o0, o064 = ref.bf16(rng.standard_normal((T, hq, dv)))
        l0 = rng.uniform(-6, 6, (T, hq)).astype(np.float32)
        l0[::3] = -np.inf
        o0[::3] = float("nan")                               # a part that saw nothing may hold anything
        out[:T], lse[:T] = o0.cuda(), dev(l0)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    g.prompt_attention(q, k, v, dev(qs), dev(ks), max(klens + [0]) if max_key_len is None else max_key_len, scale, causal=causal,
                       window=window, num_sinks=sinks, out=out, lse=lse, return_lse=True, accumulate=accumulate,
                       workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    assert (out[T:] == 7).all() and (lse[T:] == 7).all(), "rows behind the last sequence were written"
    scale32 = float(np.float32(scale))
    for b, (n, m) in enumerate(zip(qlens, klens)):
        see = ref.causal(n, m, window, sinks) if causal else np.ones((n, m), bool)
        see = np.repeat(see, group, 0)
        a, c = slice(int(qs[b]), int(qs[b + 1])), slice(int(ks[b]), int(ks[b + 1]))
        for h in range(hk):
            heads = slice(h * group, (h + 1) * group)
            kk, vv = k64[c, h], v64[c, h]
            odd = ~np.isfinite(vv)
            rows64 = q64[a, heads].reshape(-1, dk)
            # weights in bf16: half a step is 2^-8, and its range is binary32's
            o, l, ot, lt = ref.attend(rows64, np.nan_to_num(kk, nan=0, posinf=0, neginf=0), np.where(odd, 0, vv), see, scale32, 2.0 ** -8, 0.0)
            got, got_l = out[a, heads].reshape(-1, dv).double().cpu().numpy(), lse[a, heads].reshape(-1).double().cpu().numpy()
            if accumulate:
                l_0, o_0 = l0[a, heads].reshape(-1).astype(np.float64), o064[a, heads].reshape(-1, dv)
                top = np.maximum(l, l_0)
                with np.errstate(invalid="ignore"):
                    wa, wb = (np.where(x == -np.inf, 0, np.exp(x - np.where(top == -np.inf, 0, top)))[:, None] for x in (l, l_0))
                    tot = np.where(wa + wb > 0, wa + wb, 1)
                    near = (lt + 2.0 ** -20 * (np.abs(np.where(top == -np.inf, 0, top)) + 20))[:, None]     # of the two parts' weights
                    oo = np.where(wb > 0, o_0, 0)
                    o, ot = (wa * o + wb * oo) / tot, (wa * ot + 2.0 ** -8 * np.abs(wa * o + wb * oo) + near * (wa * np.abs(o) + wb * np.abs(oo))) / tot + 1e-30
                    l = np.where(top == -np.inf, -np.inf, top + np.log(tot[:, 0]))
                    lt = near[:, 0] + 2.0 ** -20 * (np.abs(np.where(np.isinf(l), 0, l)) + 20)
            if odd.any():
                poison = (see.astype(float) @ odd.astype(float)) > 0
                assert not np.isfinite(got[poison]).any() and np.isfinite(got[~poison]).all()
                got = np.where(poison, o, got)
            close(got, o, ot, f"request {b} head {h} out")
            close(got_l, l, lt, f"request {b} head {h} lse")
    return out, lse


PROMPT = [  # kv heads, group, dk, dv, window, sinks
    (2, 4, 128, 128, None, 0), (1, 1, 64, 64, None, 0), (2, 1, 192, 128, None, 0), (1, 3, 256, 256, None, 0),
    (1, 8, 80, 80, 33, 5), (3, 2, 96, 64, 8, 2), (1, 5, 8, 8, None, 0), (2, 2, 128, 64, 40, 70), (1, 16, 64, 128, 1, 0),
    (8, 1, 128, 128, 64, 0), (1, 2, 200, 40, 17, 1), (1, 1, 136, 248, None, 0), (16, 1, 64, 64, None, 0),
]


@pytest.mark.parametrize("hk,group,dk,dv,window,sinks", PROMPT)
def test_prompts(g, hk, group, dk, dv, window, sinks):
    """Sequences of zero and one token, around the tiles' borders, with and
    without context before the queries, and queries at negative positions."""
    rng = np.random.default_rng(dk + dv)
    check_prompt(g, rng, [1, 0, 33, 64, 7, 130, 1, 3, 5], [1, 0, 33, 64, 70, 130, 200, 2, 0], hk, group, dk, dv, True, window, sinks)


@pytest.mark.parametrize("hk,group,dk,dv", [(2, 4, 128, 128), (1, 1, 192, 128), (1, 2, 72, 136), (2, 3, 64, 64), (1, 1, 256, 256)])
def test_prompts_over_context(g, hk, group, dk, dv):
    """Without the causal order: every query sees its request's keys, of which
    there may be none."""
    rng = np.random.default_rng(dk)
    check_prompt(g, rng, [1, 40, 3, 0, 130, 2], [65, 7, 0, 9, 128, 1], hk, group, dk, dv, causal=False)


@pytest.mark.parametrize("lens", [[1] * 20, [127, 128, 129], [31, 32, 33, 63, 65], [300], [2] * 70, [0, 0, 5, 0]])
def test_prompt_lengths(g, lens):
    check_prompt(g, np.random.default_rng(3), lens, lens, 2, 4, 128, 128, fused=True)


@pytest.mark.parametrize("dk,dv", [(128, 128), (192, 128), (80, 96)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (900, 40)])
def test_prompt_long_batches(g, dk, dv, window, sinks):
    """Many row tiles, which start with the longest, of lengths that differ."""
    check_prompt(g, np.random.default_rng(4), [1100, 1, 1900, 700], [1100, 900, 1900, 1030], 1, 2, dk, dv, window=window, sinks=sinks)


def test_prompt_rows_behind_4_gib(g):
    """Rows 2^24 bytes apart give the bits of rows that lie together."""
    rng = np.random.default_rng(10)
    n, d = 300, 128
    q, k, v = (ref.bf16(rng.standard_normal((n, 1, d)))[0].cuda() for _ in range(3))
    wide = torch.zeros((n, 1 << 23), dtype=torch.bfloat16, device="cuda")
    far = [wide[:, None, i * d:(i + 1) * d] for i in range(4)]
    for x, y in zip(far, (q, k, v)):
        x.copy_(y)
    starts = dev(np.array([0, 30, n], np.int32))
    want, lse = g.prompt_attention(q, k, v, starts, starts, n, 0.1, return_lse=True)
    got, got_lse = g.prompt_attention(*far[:3], starts, starts, n, 0.1, out=far[3], return_lse=True)
    assert torch.equal(got, want) and torch.equal(got_lse, lse)


@pytest.mark.parametrize("dk,dv", [(128, 128), (192, 128), (256, 256)])
def test_prompt_key_split_and_workspace(g, dk, dv):
    for ws, longest in ((None, 2100), (None, 300), (None, 5), (0, 2100), (200000, 2100)):
        workspace = None if ws is None else torch.empty(ws, dtype=torch.uint8, device="cuda")
        check_prompt(g, np.random.default_rng(5), [1, 40, 2], [2100, 900, 40], 1, 2, dk, dv, max_key_len=longest, workspace=workspace)


@pytest.mark.parametrize("klens", [[70, 5, 0, 130], [1500, 900, 0, 3]])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_accumulate(g, klens, causal):
    """Joined with an earlier part; parts that saw nothing do not count."""
    check_prompt(g, np.random.default_rng(6), [4, 5, 3, 9], klens, 2, 2, 128, 128, causal=causal, accumulate=True)


def test_prompt_chunks_of_context(g):
    """A prompt's tail over its context in two chunks and itself: the same as
    in one go, within the bounds of three roundings to bf16."""
    rng = np.random.default_rng(7)
    hq, hk, d, n, m = 4, 2, 128, 50, 300
    q, k, v = (ref.bf16(rng.standard_normal(s))[0].cuda() for s in ((n, hq, d), (m, hk, d), (m, hk, d)))
    start = lambda x: dev(np.array([0, x], np.int32))  # noqa: E731
    whole, lse = g.prompt_attention(q, k, v, start(n), start(m), m, d ** -0.5, return_lse=True)
    out, part = g.prompt_attention(q, k[m - n:], v[m - n:], start(n), start(n), n, d ** -0.5, return_lse=True)
    for a, b in ((0, 128), (128, m - n)):
        g.prompt_attention(q, k[a:b], v[a:b], start(n), start(b - a), b - a, d ** -0.5, causal=False, out=out, lse=part, accumulate=True)
    close(part, lse.double().cpu().numpy(), 1e-4, "lse")
    # every part's weights and output are rounded to bf16 (2 * 2^-8), as are the whole's
    bound = 8 * 2.0 ** -8 * float(v.abs().max()) * 0.5
    assert float((out.float() - whole.float()).abs().max()) < bound


@pytest.mark.parametrize("tokens", [1, 8, 9])
def test_prompt_many_splits(g, tokens):
    """Dozens of key splits a row, for the joins of few rows and of more than
    2048: against the call that does not split.  Values are positive and grow
    along the keys, so that outputs (1 .. 3) are off by less than four roundings
    of 2^-8 to bf16 (weights and outputs, both calls); an lse of about 10 by the
    rounding of sums, 2^-24 a step of 512 and of the parts."""
    rng = np.random.default_rng(11)
    n, hq = 32768, 256
    q, k = (ref.bf16(rng.standard_normal((m, h, 64)))[0].cuda() for m, h in ((tokens, hq), (n, 1)))
    v = (1 + torch.arange(n, device="cuda") / n)[:, None, None].expand(n, 1, 64) + torch.rand(n, 1, 64, device="cuda")
    v = v.to(torch.bfloat16)
    qs, ks = dev(np.array([0, tokens], np.int32)), dev(np.array([0, n], np.int32))
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    one, one_lse = g.prompt_attention(q, k, v, qs, ks, n, 0.125, return_lse=True, workspace=none)
    out, lse = g.prompt_attention(q, k, v, qs, ks, n, 0.125, return_lse=True)
    assert float((lse - one_lse).abs().max()) < 1e-3
    assert float(((out.float() - one.float()) / one.float()).abs().max()) < 4 * 2.0 ** -8


def test_prompt_values_that_are_hidden(g):
    """Infinities and NaN in keys and values reach the rows that see them and
    no other, not those of the same tile or of the next sequence."""
    def edit(k, v):
        v[20, 0, 3] = float("inf")
        v[61, 1, 5] = float("nan")
        v[100, 0, 127] = float("-inf")
    check_prompt(g, np.random.default_rng(8), [64, 40, 30], [64, 40, 30], 2, 2, 128, 128, edit=edit)
    check_prompt(g, np.random.default_rng(8), [64, 40, 30], [64, 40, 30], 2, 2, 128, 128, window=7, sinks=1, edit=edit)

    rng = np.random.default_rng(9)
    q, k, v = (ref.bf16(rng.standard_normal((70, 2, 64)))[0].cuda() for _ in range(3))
    starts = dev(np.array([0, 40, 70], np.int32))
    want, lse = g.prompt_attention(q, k, v, starts, starts, 40, 0.125, return_lse=True)
    for x in (k, v):
        y = x.clone()
        y[30] = float("nan")
        got, l = g.prompt_attention(q, y if x is k else k, y if x is v else v, starts, starts, 40, 0.125, return_lse=True)
        same = torch.ones(70, dtype=torch.bool, device="cuda")
        same[30:40] = False
        assert torch.equal(got[same], want[same]) and torch.equal(l[same], lse[same])
        assert torch.isnan(got[30:40]).any() or torch.isinf(got[30:40]).any()


def test_prompt_scales_streams_and_batches(g):
    rng = np.random.default_rng(13)
    check_prompt(g, rng, [33, 1], [33, 20], 1, 2, 64, 64, scale=-0.2, stream=torch.cuda.Stream())
    check_prompt(g, rng, [33, 1], [33, 20], 1, 2, 64, 64, scale=0.0)
    n = rng.integers(1, 6, 530).tolist()
    check_prompt(g, rng, n, n, 1, 2, 64, 64)


def test_prompt_captured(g):
    """A replayed graph (keys split, so the join is in it) gives the eager bits
    for the inputs of its time."""
    rng = np.random.default_rng(14)
    q, k, v = (ref.bf16(rng.standard_normal((n, h, 128)))[0].cuda() for n, h in ((3, 8), (3000, 2), (3000, 2)))
    qs, ks = dev(np.array([0, 1, 3], np.int32)), dev(np.array([0, 1000, 3000], np.int32))
    call = lambda: g.prompt_attention(q, k, v, qs, ks, 2000, 0.1, return_lse=True)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = call()
    for i in range(3):
        q.mul_(0.5 + i)
        want = call()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------
def test_prompt_then_decode(g):
    """Two prompts through append and prompt attention, then tokens through
    append and cache attention, on pages that the pool grants; against 64-bit
    attention over the dequantized cache (decode) and the inputs (prompt)."""
    rng = np.random.default_rng(31)
    hq, hk, hs, bs, nb, steps = 4, 2, 64, 16, 24, 20
    lens = [37, 50]
    B = len(lens)
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    seq = torch.zeros(B, dtype=torch.int32, device="cuda")
    refs = torch.zeros(nb, dtype=torch.int32, device="cuda")
    rows = torch.arange(B, dtype=torch.int32, device="cuda")
    cache = torch.full((nb, 2, bs, hk, hs), 0xFF, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.full((nb, 2, hk), float("nan"), device="cuda")
    ang = np.arange(128)[:, None] * 10000.0 ** -(np.arange(0, hs, 2) / hs)
    cs = dev(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))
    tab = cs.double().cpu().numpy()

    def grow(n):
        st = g.extend_requests(bs, table, seq, refs, rows, torch.tensor(n, dtype=torch.int32, device="cuda"))
        assert (st == 1).all()

    def inputs(n):
        t, x = ref.bf16(rng.standard_normal((n, hq + 2 * hk, hs)))
        t = t.cuda()
        return (t[:, :hq], t[:, hq:hq + hk], t[:, hq + hk:]), x

    grow(lens)
    (q, k, v), x = inputs(sum(lens))
    starts = dev(np.array([0, lens[0], sum(lens)], np.int32))
    qr, kr = g.rope_append_fp8_kv(q, k, v, cache, scales, table, starts, seq, cs, return_k=True)
    out = g.prompt_attention(qr, kr, v, starts, starts, max(lens), hs ** -0.5)
    pos = np.concatenate([np.arange(n) for n in lens])
    q64, k64 = qr.double().cpu().numpy(), kr.double().cpu().numpy()
    assert np.abs(q64 - ref.rotate(x[:, :hq], pos, tab, hs, False)[0]).max() < 0.05
    for b, n in enumerate(lens):
        s = slice(int(starts[b]), int(starts[b + 1]))
        for h in range(hq):
            o, _, ot, _ = ref.attend(q64[s, h], k64[s, h // 2], x[s, hq + hk + h // 2], ref.causal(n, n), hs ** -0.5, 2.0 ** -8, 0.0)
            close(out[s, h], o, ot, f"prompt {b} head {h}")
    one = dev(np.arange(B + 1).astype(np.int32))
    for step in range(1, steps + 1):
        now = [n + step for n in lens]
        grow(now)
        (q, k, v), x = inputs(B)
        qr, _ = g.rope_append_fp8_kv(q, k, v, cache, scales, table, one, seq, cs)
        out = g.attention_fp8_kv(qr, cache, scales, table, one, seq, max(now), hs ** -0.5)
    value = ref.e4m3(cache.view(torch.uint8).cpu().numpy()) * scales.double().cpu().numpy()[:, :, None, :, None]
    t, q64 = table.cpu().numpy(), qr.double().cpu().numpy()
    for b, n in enumerate(now):
        blk, off = t[b][np.arange(n) // bs], np.arange(n) % bs
        for h in range(hq):
            k, v = value[blk, 0, off, h // 2], value[blk, 1, off, h // 2]
            o, _, ot, _ = ref.attend(q64[b:b + 1, h], k, v, np.ones((1, n), bool), hs ** -0.5, 2.0 ** -11,
                                     2.0 ** -31 * 448 * float(scales.nan_to_num(0).max()))
            close(out[b:b + 1, h], o, ot, f"decode {b} head {h}")
