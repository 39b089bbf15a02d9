"""GPU tests of the operators around the cache against plain 64-bit
references (operator_refs.py), at the sizes, layouts and masks where they can
go wrong."""
import itertools

import numpy as np
import pytest
import torch

import operator_refs as ref
from gpu_util import dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gather_concat_cache_amd as gc
    return gc


def close(got, want, tol, what):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    bad = ~same & ~(np.abs(got - want) <= tol)
    if bad.any():
        i = np.unravel_index(int(np.argmax(bad)), bad.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; first at {i}: got {got[i]!r}, want {want[i]!r}, "
                             f"bound {np.broadcast_to(tol, bad.shape)[i]:.3g}")


# ---------------------------------------------------------------------------
# norms and rotation
# ---------------------------------------------------------------------------
QK = [  # tokens, q heads, k heads, head size, rot, interleaved, bf16 table
    (1, 32, 8, 128, 128, False, False), (1, 1, 1, 16, 16, False, False), (7, 5, 3, 80, 32, False, False),
    (7, 5, 3, 80, 32, True, True), (33, 12, 4, 64, 64, True, False), (19, 3, 1, 96, 48, False, True),
    (5, 17, 2, 192, 96, True, False), (9, 4, 4, 256, 256, False, False), (3, 2, 1, 512, 64, False, False),
    (4, 3, 2, 48, 0, False, False), (300, 8, 2, 128, 64, False, True), (2, 6, 0, 112, 112, True, False),
]


@pytest.mark.parametrize("T,hq,hk,hs,rot,inter,tab16", QK)
def test_qk_norm_rope(g, T, hq, hk, hs, rot, inter, tab16):
    rng = np.random.default_rng(hs + T)
    qkv, qkv64 = ref.bf16(rng.standard_normal((T, hq + 2 * hk + 1, hs)) * 10.0 ** rng.integers(-3, 3, (T, 1, 1)))
    qkv = qkv.cuda()
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    w = [ref.bf16(1 + 0.3 * rng.standard_normal(hs)) for _ in range(2)]
    pos = rng.integers(0, 50, T)
    if T > 4:
        pos[1], pos[3] = -1, 50                              # outside the table: zero rows
    ang = np.arange(50)[:, None] * 3.0 ** -np.arange(rot // 2)
    table = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))
    table = table.to(torch.bfloat16) if tab16 else table
    cs = None if rot == 0 else table.cuda()
    args = (q, k if hk else None, w[0][0].cuda(), w[1][0].cuda() if hk else None, dev(pos), cs)
    qo, ko = g.qk_norm_rope(*args, eps=1e-5, interleaved=inter)
    eps = float(np.float32(1e-5))
    tab = table.to(torch.float64).numpy()
    for out, x, wt, n in ((qo, qkv64[:, :hq], w[0][1], "q"), (ko, qkv64[:, hq:hq + hk], w[1][1], "k")):
        if out is not None:
            want, tol = ref.norm_rope(x, wt, pos, tab, rot, eps, inter)
            close(out, want, tol, n)
    # in place inside the fused projection: the same bits, nothing else touched
    rest = qkv[:, hq + hk:].clone()
    g.qk_norm_rope(*args, eps=1e-5, interleaved=inter, q_out=q, k_out=k if hk else None)
    assert torch.equal(q, qo) and (ko is None or torch.equal(k, ko)) and torch.equal(qkv[:, hq + hk:], rest)


def test_qk_norm_rope_zero_rows(g):
    """A zero head stays zero with eps > 0; no tokens is a no-op."""
    q = torch.zeros(2, 2, 32, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(32, dtype=torch.bfloat16, device="cuda")
    cs = torch.ones(4, 32, device="cuda")
    qo, ko = g.qk_norm_rope(q, None, w, None, torch.zeros(2, dtype=torch.int64, device="cuda"), cs)
    assert ko is None and torch.equal(qo, q)
    qo, _ = g.qk_norm_rope(q[:0], None, w, None, torch.zeros(0, dtype=torch.int64, device="cuda"), cs)
    assert qo.shape == (0, 2, 32)


# ---------------------------------------------------------------------------
# attention: batches
# ---------------------------------------------------------------------------
def fp4_bytes(rng, shape):
    return rng.integers(0, 256, shape, dtype=np.uint8)


def scale_bytes(rng, shape):
    """e4m3 codes of 2^-5 .. 1.75, now and then the largest, the smallest, or 0."""
    s = rng.integers(0x10, 0x3E, shape, dtype=np.uint8)
    odd = rng.random(shape)
    return np.where(odd < 0.01, 0x7E, np.where(odd < 0.02, 0x01, np.where(odd < 0.03, 0, s))).astype(np.uint8)


class Batch:
    """Ragged requests over shuffled pages, with unused pages full of 0xFF
    (NaN scales), ids outside the cache behind each row's end."""

    def __init__(self, rng, qlens, lens, bs, spare=2):
        self.bs, self.qlens, self.lens = bs, list(qlens), list(lens)
        n = [ref.pages(x, bs) for x in lens]
        self.nb = sum(n) + spare
        order = rng.permutation(self.nb)
        self.used = order[:sum(n)]
        self.table = rng.choice(np.array([-1, -7, self.nb, 1 << 30], np.int32), (len(lens), max(n + [1]) + 1))
        at = 0
        for b, k in enumerate(n):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.starts = np.concatenate([[0], np.cumsum(self.qlens)]).astype(np.int32)
        self.T = int(self.starts[-1])

    def metadata(self):
        return dev(self.table.astype(np.int32)), dev(self.starts), dev(np.array(self.lens, np.int32))


def kv_cache(g, rng, batch, hk, hs, layout):
    """Flat bytes with written entries at the batch's positions only."""
    nb, bs = batch.nb, batch.bs
    full = hs // 2 + hs // 16
    if layout == "split":
        L = g.nvfp4_kv_split_layout(bs, hk, hs)
    elif layout == "hnd":
        L = g.nvfp4_kv_split_layout(bs, hk, hs, hnd=True)
    else:                                                    # [data | scale] rows of a head, padded to 8 bytes
        row = (full + 7) // 8 * 8
        L = g.NvFp4KvLayout(data_offset=0, data_token_stride=hk * row, data_head_stride=row, scale_offset=hs // 2,
                            scale_token_stride=hk * row, scale_head_stride=row, side_stride=bs * hk * row + 8,
                            block_stride=2 * bs * hk * row + 16)
    flat = np.full(nb * L.block_stride + 64, 0xFF, np.uint8)
    for b, n in enumerate(batch.lens):
        for p in range(n):
            blk, off = int(batch.table[b, p // bs]), p % bs
            if not 0 <= blk < nb:
                continue
            for side in (0, 1):
                base = blk * L.block_stride + side * L.side_stride
                for h in range(hk):
                    d = base + L.data_offset + off * L.data_token_stride + h * L.data_head_stride
                    s = base + L.scale_offset + off * L.scale_token_stride + h * L.scale_head_stride
                    flat[d:d + hs // 2] = fp4_bytes(rng, hs // 2)
                    flat[s:s + hs // 16] = scale_bytes(rng, hs // 16)
    d = dev(flat)
    view = torch.as_strided(d, (nb, 2, bs, hk, full), (L.block_stride, L.side_stride, hk * full, full, 1))
    return flat, view, L


def queries(rng, T, heads, dk, pad=0):
    """bf16 queries of mixed magnitudes, in a wider buffer when pad."""
    t, x = ref.bf16(rng.standard_normal((T, heads, dk)) * 10.0 ** rng.uniform(-2, 0.5, (T, heads, 1)))
    if not pad:
        return t.cuda(), x
    wide = torch.zeros(T, heads + 1, dk + pad, dtype=torch.bfloat16, device="cuda")
    wide[:, :heads, :dk] = t.cuda()
    return wide[:, :heads, :dk], x


def check_kv(g, rng, batch, hk, group, hs, layout="split", window=None, sinks=0, mask=None, max_seq_len=None,
             workspace=None, pad=0, scale=None, edit=None, see_of=None):
    flat, cache, L = kv_cache(g, rng, batch, hk, hs, layout)
    q, q64 = queries(rng, batch.T + 2, hk * group, hs, pad)   # two rows behind the last sequence
    gk, gv = np.float32(0.7), np.float32(1.9)
    bt, starts, lens = batch.metadata()
    scale = hs ** -0.5 if scale is None else scale
    out = torch.full((batch.T + 2, hk * group, hs), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((batch.T + 2, hk * group), 7.0, device="cuda")
    longest = max(batch.lens + [1]) if max_seq_len is None else max_seq_len
    kw = dict(layout=L, out=out, lse=lse, return_lse=True, workspace=workspace)
    head = (q, cache, dev(np.array([gk])), dev(np.array([gv])), bt, starts, lens)
    if mask is None:
        g.attention_nvfp4_kv(*head, longest, scale, window=window, num_sinks=sinks, **kw)
    else:
        full_mask = np.zeros((batch.T + 2, mask.shape[1]), bool)
        full_mask[:batch.T] = mask
        g.tree_attention_nvfp4_kv(*head, dev(full_mask), longest, scale, **kw)
    torch.cuda.synchronize()
    assert (out[batch.T:] == 7).all() and (lse[batch.T:] == 7).all(), "rows behind the last sequence were written"
    scale32 = float(np.float32(scale))
    for b, (n, length) in enumerate(zip(batch.qlens, batch.lens)):
        r0 = int(batch.starts[b])
        m = max(length, 0)
        see = ref.causal(n, length, window, sinks) if mask is None else ref.tree(n, length, mask[r0:r0 + n])
        see = see[:, :m] if m else np.zeros((n, 0), bool)
        for h in range(hk):
            k, v, ok = ref.kv_positions(flat, L, batch.table[b], m, batch.bs, batch.nb, h, hs)
            vis = np.repeat(see & ok[None], group, 0)
            rows = q64[r0:r0 + n, h * group:(h + 1) * group].reshape(-1, hs)
            o, l, ot, lt = ref.attend(rows, k, v, vis, scale32, float(gk), float(gv))
            what = f"request {b} head {h}"
            close(out[r0:r0 + n, h * group:(h + 1) * group].reshape(-1, hs), o, ot, what + " out")
            close(lse[r0:r0 + n, h * group:(h + 1) * group].reshape(-1), l, lt, what + " lse")
    return out, lse


KV = [  # kv heads, group, head size, block, layout, window, sinks
    (1, 1, 16, 16, "split", None, 0), (2, 4, 64, 16, "split", 8, 2), (1, 3, 80, 24, "split", 33, 5),
    (2, 2, 128, 16, "hnd", 40, 4), (1, 8, 128, 64, "row", 1, 0), (2, 1, 176, 16, "row", 64, 40),
    (1, 4, 256, 32, "split", 17, 1), (3, 2, 96, 1, "row", 50, 3), (1, 16, 128, 7, "hnd", 1000, 4),
    (1, 20, 64, 16, "split", 5, 100), (2, 5, 48, 40, "hnd", None, 0), (1, 2, 240, 5, "row", 9, 2),
    (4, 8, 128, 16, "split", 31, 33), (1, 1, 112, 48, "split", 32, 32),
]


@pytest.mark.parametrize("hk,group,hs,bs,layout,window,sinks", KV)
def test_window_attention(g, hk, group, hs, bs, layout, window, sinks):
    """Decode, short chunks and long ones in one batch; lengths of zero, one,
    around the tile and page borders; a query longer than its sequence."""
    rng = np.random.default_rng(hs + bs)
    batch = Batch(rng, [1, 0, 3, 1, 40, 1, 5, 2], [1, 9, 3, 33, 75, 130, 2, 0], bs)
    check_kv(g, rng, batch, hk, group, hs, layout, window, sinks)


@pytest.mark.parametrize("qlens,lens", [([1] * 9, [1, 15, 16, 17, 31, 32, 33, 64, 200]), ([130], [130]), ([70, 1, 64], [300, 5, 64]),
                                        ([2] * 20, list(range(2, 42, 2))), ([1], [700])])
@pytest.mark.parametrize("window,sinks", [(None, 0), (20, 4), (64, 0)])
def test_window_attention_lengths(g, qlens, lens, window, sinks):
    rng = np.random.default_rng(len(lens))
    batch = Batch(rng, qlens, lens, 16)
    check_kv(g, rng, batch, 2, 4, 128, "split", window, sinks, pad=24)


@pytest.mark.parametrize("hs,bs", [(128, 16), (64, 24), (256, 16)])
def test_key_split_and_workspace(g, hs, bs):
    """Keys split over many workgroups, over few (a small or no workspace), and
    sequences longer than max_seq_len says: all within the bounds."""
    for ws, longest in ((None, 2100), (None, 300), (None, 5), (0, 2100), (200000, 2100)):
        rng = np.random.default_rng(5)
        batch = Batch(rng, [1, 4, 2], [2100, 900, 40], bs)
        workspace = None if ws is None else torch.empty(ws, dtype=torch.uint8, device="cuda")
        check_kv(g, rng, batch, 1, 2, hs, max_seq_len=longest, workspace=workspace)


def test_hidden_pages_and_holes(g):
    """Ids outside the cache in the middle of a row hide their positions; a
    row whose every page is missing is zeros with lse -inf."""
    rng = np.random.default_rng(3)
    batch = Batch(rng, [2, 1, 3], [90, 50, 64], 16)
    batch.table[0, 2] = -1
    batch.table[0, 4] = batch.nb
    batch.table[1, :] = -1
    out, lse = check_kv(g, rng, batch, 2, 2, 64, window=60, sinks=3)
    assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()


def test_nan_bytes_in_hidden_positions(g):
    """Entries that only some rows of a tile see, with every byte of the ones
    hidden from all set to the NaN code: outputs stay finite and right."""
    rng = np.random.default_rng(8)
    batch = Batch(rng, [4, 1], [100, 70], 16)
    out, lse = check_kv(g, rng, batch, 1, 4, 128, window=10, sinks=2)
    assert torch.isfinite(out[:5]).all() and torch.isfinite(lse[:5]).all()


def test_extreme_queries(g):
    """Rows of zeros, of the smallest and of large magnitudes, and logits that
    put all weight on one key."""
    rng = np.random.default_rng(12)
    batch = Batch(rng, [6], [80], 16)
    flat, cache, L = kv_cache(g, rng, batch, 1, 64, "split")
    x = rng.standard_normal((6, 2, 64)) * np.array([0.0, 1e-38, 1e-20, 300.0, 1e4, 1.0])[:, None, None]
    q, q64 = ref.bf16(x)
    bt, starts, lens = batch.metadata()
    one = torch.ones(1, device="cuda")
    out, lse = g.attention_nvfp4_kv(q.cuda(), cache, one, one, bt, starts, lens, 80, 0.125, return_lse=True)
    k, v, ok = ref.kv_positions(flat, L, batch.table[0], 80, 16, batch.nb, 0, 64)
    see = np.repeat(ref.causal(6, 80), 2, 0)
    o, l, ot, lt = ref.attend(q64.reshape(-1, 64), k, v, see, 0.125)
    close(out.reshape(-1, 64), o, ot, "out")
    close(lse.reshape(-1), l, lt, "lse")


def test_negative_and_zero_scales(g):
    rng = np.random.default_rng(13)
    batch = Batch(rng, [3, 1], [50, 20], 16)
    check_kv(g, rng, batch, 1, 2, 64, scale=-0.2)
    check_kv(g, rng, batch, 1, 2, 64, scale=0.0, window=9, sinks=1)


@pytest.mark.parametrize("hk,group,hs,bs", [(2, 4, 128, 16), (1, 1, 64, 24), (1, 7, 80, 16), (1, 2, 256, 8)])
def test_tree_attention_kv(g, hk, group, hs, bs):
    """Trees, an arbitrary mask, rows whose mask leaves nothing but the
    context, and (no context) nothing at all."""
    rng = np.random.default_rng(hs)
    qlens, lens = [8, 1, 33, 5, 12, 3], [60, 1, 33, 5, 140, 2]
    batch = Batch(rng, qlens, lens, bs)
    mask = rng.random((batch.T, 33)) < 0.4
    for b, n in enumerate(qlens[:3]):
        r0 = batch.starts[b]
        for i in range(n):                                   # a real tree
            parent = rng.integers(-1, i) if i else -1
            mask[r0 + i] = mask[r0 + parent] if parent >= 0 else False
            mask[r0 + i, i] = True
    r0 = batch.starts[3]
    mask[r0 + 1] = False                                     # no context either: an empty row
    out, lse = check_kv(g, rng, batch, hk, group, hs, mask=mask)
    assert (out[int(r0) + 1] == 0).all() and torch.isneginf(lse[int(r0) + 1]).all()
    check_kv(g, rng, batch, hk, group, hs, mask=mask[:, :9])  # columns behind the mask are hidden


def test_tree_mask_of_a_chain_is_causal(g):
    """A lower-triangular tree mask gives the causal operator's bits."""
    rng = np.random.default_rng(4)
    batch = Batch(rng, [9, 4], [300, 77], 16)
    mask = np.zeros((batch.T, 9), bool)
    for b, n in enumerate(batch.qlens):
        mask[batch.starts[b]:batch.starts[b] + n, :n] = np.tril(np.ones((n, n), bool))
    _, cache, L = kv_cache(g, rng, batch, 2, 64, "split")
    q, _ = queries(rng, batch.T, 8, 64)
    bt, starts, lens = batch.metadata()
    one = torch.ones(1, device="cuda")
    a = g.attention_nvfp4_kv(q, cache, one, one, bt, starts, lens, 300, 0.125, return_lse=True)
    b = g.tree_attention_nvfp4_kv(q, cache, one, one, bt, starts, lens, dev(mask), 300, 0.125, return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def check_mla(g, rng, batch, heads, estr=352, mask=None, max_seq_len=None, pad=0):
    nb, bs = batch.nb, batch.bs
    flat = np.full((nb, bs, estr), 0xFF, np.uint8)
    for b, n in enumerate(batch.lens):
        for p in range(n):
            blk = int(batch.table[b, p // bs])
            if 0 <= blk < nb:
                e = flat[blk, p % bs]
                e[:256] = fp4_bytes(rng, 256)
                e[256:320] = rng.integers(0, 0x48, 64, dtype=np.uint8) | rng.integers(0, 2, 64, dtype=np.uint8) << 7
                e[320:352] = scale_bytes(rng, 32)
    q, q64 = queries(rng, batch.T + 1, heads, 576, pad)
    bt, starts, lens = batch.metadata()
    out = torch.full((batch.T + 1, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((batch.T + 1, heads), 7.0, device="cuda")
    m = None
    if mask is not None:
        m = torch.zeros(batch.T + 1, mask.shape[1] + 3, dtype=torch.uint8, device="cuda")[:, :mask.shape[1]]
        m[:batch.T] = dev(mask.astype(np.uint8))
    longest = max(batch.lens + [1]) if max_seq_len is None else max_seq_len
    g.tree_attention_nvfp4_ds_mla(q, dev(flat), bt, starts, lens, m, longest, 192 ** -0.5, out=out, lse=lse,
                                  return_lse=True)
    torch.cuda.synchronize()
    assert (out[batch.T:] == 7).all() and (lse[batch.T:] == 7).all(), "rows behind the last sequence were written"
    for b, (n, length) in enumerate(zip(batch.qlens, batch.lens)):
        r0 = int(batch.starts[b])
        see = ref.causal(n, length) if mask is None else ref.tree(n, length, mask[r0:r0 + n])
        k, v, ok = ref.mla_positions(flat.reshape(-1), batch.table[b], length, bs, nb, bs * estr, estr)
        vis = np.repeat(see & ok[None], heads, 0)
        o, l, ot, lt = ref.attend(q64[r0:r0 + n].reshape(-1, 576), k, v, vis, float(np.float32(192 ** -0.5)))
        close(out[r0:r0 + n].reshape(-1, 512), o, ot, f"request {b} out")
        close(lse[r0:r0 + n].reshape(-1), l, lt, f"request {b} lse")


@pytest.mark.parametrize("heads,bs,estr", [(16, 64, 352), (1, 16, 352), (5, 24, 368), (20, 1, 352), (32, 48, 352),
                                           (128, 64, 384)])
def test_mla_chain(g, heads, bs, estr):
    rng = np.random.default_rng(heads)
    batch = Batch(rng, [1, 0, 1, 4, 2, 1], [1, 3, 33, 40, 1, 150], bs)
    check_mla(g, rng, batch, heads, estr, pad=8)


@pytest.mark.parametrize("heads,bs", [(16, 64), (3, 40), (20, 16)])
def test_mla_tree(g, heads, bs):
    rng = np.random.default_rng(heads + 1)
    batch = Batch(rng, [7, 1, 20, 3], [90, 1, 20, 70], bs)
    mask = rng.random((batch.T, 20)) < 0.5
    mask[8] = False                                          # no context: an empty row
    check_mla(g, rng, batch, heads, mask=mask)


@pytest.mark.parametrize("longest", [1300, 64])
def test_mla_key_split(g, longest):
    rng = np.random.default_rng(2)
    batch = Batch(rng, [1, 2], [1300, 500], 64)
    check_mla(g, rng, batch, 16, max_seq_len=longest)


def test_tree_mask_without_columns(g):
    """A mask of no columns hides every drafted token: rows see the context
    alone, and nothing at all without one."""
    rng = np.random.default_rng(14)
    batch = Batch(rng, [3, 2, 40], [50, 2, 100], 16)
    none = np.zeros((batch.T, 0), bool)
    out, lse = check_kv(g, rng, batch, 1, 2, 64, mask=none)
    assert (out[3:5] == 0).all() and torch.isneginf(lse[3:5]).all()
    check_mla(g, rng, batch, 4, mask=none)


# The kernels count the requests of a batch over 64 lanes: one a lane, several a
# lane, and, in large batches, by the packed rows alone.
@pytest.mark.parametrize("requests", [64, 65, 200, 256, 257, 512, 513, 1025, 4097])
def test_many_requests(g, requests):
    """Ragged batches with requests without queries, and keys, in between."""
    rng = np.random.default_rng(requests)
    qlens = rng.choice([0, 1, 1, 2, 9], requests)
    lens = qlens + rng.choice([0, 0, 1, 5], requests) - (rng.random(requests) < 0.1)
    batch = Batch(rng, qlens.tolist(), np.maximum(lens, 0).tolist(), 16)
    check_kv(g, rng, batch, 1 + (requests == 257), 3, 16, window=4, sinks=1)
    if requests < 1000:
        check_mla(g, rng, batch, 5)


@pytest.mark.parametrize("requests,qlen", [(3, 2), (70, 1), (130, 1), (5, 20), (4, 40)])
@pytest.mark.parametrize("hs", [64, 576])
def test_key_split_of_uneven_batches(g, requests, qlen, hs):
    """One long request among short ones: splits are sized by the batch's work,
    so it is split further than a batch of its length would be."""
    rng = np.random.default_rng(requests)
    lens = rng.integers(qlen, 60, requests)
    lens[requests // 2] = 1900
    batch = Batch(rng, [qlen] * requests, lens.tolist(), 16)
    if hs == 576:
        check_mla(g, rng, batch, 3)
    else:
        check_kv(g, rng, batch, 1, 2, hs)


@pytest.mark.parametrize("qlen,window,sinks", [(1, 500, 70), (40, 300, 70), (70, 333, 33), (129, 64, 100)])
def test_sinks_and_window_split(g, qlen, window, sinks):
    """Odd numbers of sink tiles before a window that is split over workgroups."""
    rng = np.random.default_rng(qlen)
    batch = Batch(rng, [qlen, 1], [900, 700], 16)
    check_kv(g, rng, batch, 1, 2, 128, window=window, sinks=sinks)


@pytest.mark.parametrize("qlen,window,sinks,hs", [(1, 1500, 70, 128), (9, 1601, 33, 64), (70, 1500, 70, 128), (40, 1777, 1, 256)])
def test_long_window_split(g, qlen, window, sinks, hs):
    """Windows long enough to be split, with sinks before them, in each kernel."""
    rng = np.random.default_rng(qlen + 7)
    batch = Batch(rng, [qlen, 1, qlen], [2600, 700, 1300], 16)
    lib = g._operators._load()
    assert lib.gcache_attention_workspace_bytes(batch.T + 2, 3, 2, 1, hs, 2600, window, sinks) > 0
    check_kv(g, rng, batch, 1, 2, hs, window=window, sinks=sinks)


@pytest.mark.parametrize("hs", [64, 80, 128, 256, 576])
def test_many_splits_of_few_rows(g, hs):
    """So many splits that a workgroup joins each row; short requests beside."""
    rng = np.random.default_rng(hs + 1)
    batch = Batch(rng, [1, 2, 1, 1], [4400, 3900, 90, 1], 16)
    if hs == 576:
        check_mla(g, rng, batch, 5)
        check_mla(g, rng, batch, 1, mask=rng.random((batch.T, 2)) < 0.5)
    else:
        check_kv(g, rng, batch, 1, 3, hs)


def test_rows_of_infinities_and_nan(g):
    """A query row that holds NaN or an infinity spoils its own output only."""
    rng = np.random.default_rng(15)
    batch = Batch(rng, [12], [300], 16)
    _, cache, L = kv_cache(g, rng, batch, 1, 64, "split")
    q, _ = queries(rng, batch.T, 4, 64)
    bt, starts, lens = batch.metadata()
    one = torch.ones(1, device="cuda")
    call = lambda x: g.attention_nvfp4_kv(x, cache, one, one, bt, starts, lens, 300, 0.1)        # noqa: E731
    want, bad = call(q), q.clone()
    bad[3, 1, 5], bad[7, 0, 0], bad[8, 2, 63] = float("nan"), float("inf"), -float("inf")
    got = call(bad)
    keep = torch.ones(12, 4, dtype=torch.bool, device="cuda")
    keep[3, 1] = keep[7, 0] = keep[8, 2] = False
    assert torch.equal(got[keep], want[keep])


def test_lengths_that_grow_under_a_graph(g):
    """A captured call follows the lengths and block tables of each replay, up
    to its max_seq_len, and two captured calls keep their own scratch."""
    rng = np.random.default_rng(16)
    batch = Batch(rng, [1, 1, 2], [2000, 1500, 700], 16)
    _, cache, L = kv_cache(g, rng, batch, 1, 128, "split")
    flat = torch.randint(0, 0x38, (batch.nb, 16, 352), dtype=torch.uint8, device="cuda")
    q, _ = queries(rng, batch.T, 8, 128)
    ql, _ = queries(rng, batch.T, 16, 576)
    bt, starts, full = batch.metadata()
    one = torch.ones(1, device="cuda")
    lens = full.clone()

    def both():
        return (g.attention_nvfp4_kv(q, cache, one, one, bt, starts, lens, 2000, 0.09),
                g.tree_attention_nvfp4_ds_mla(ql, flat, bt, starts, lens, None, 2000, 0.07))

    both()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(both())
        graphs.append(graph)
    for now in ([2000, 1500, 700], [3, 1, 2], [1, 900, 2], [0, 0, 0], [1999, 33, 700]):
        lens.copy_(dev(np.array(now, np.int32)))
        want = both()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), now


def test_offsets_past_32_bits(g):
    """Pages that start beyond 4 GiB of the cache."""
    rng = np.random.default_rng(21)
    bs, hk, hs = 16, 2, 128
    L = g.nvfp4_kv_split_layout(bs, hk, hs)
    nb = (1 << 32) // L.block_stride + 70
    cache = torch.zeros((nb, 2, bs, hk, 72), dtype=torch.uint8, device="cuda")
    small = rng.integers(0, 0x38, (8, 2, bs, hk, 72), dtype=np.uint8)
    q, _ = queries(rng, 1, 8, hs)
    one = torch.ones(1, device="cuda")
    starts, lens = dev(np.array([0, 1], np.int32)), dev(np.array([115], np.int32))
    got = []
    for first in (3, nb - 8):
        cache[first:first + 8] = dev(small)
        bt = dev(np.arange(first, first + 8, dtype=np.int32)[None])
        got.append(g.attention_nvfp4_kv(q, cache, one, one, bt, starts, lens, 115, 0.1, window=50, num_sinks=4))
    assert torch.equal(got[0], got[1]) and (got[0] != 0).any()
    flat = cache.reshape(-1)[:nb * bs * hk * 144 // (64 * 352) * 64 * 352].view(-1, 64, 352)
    last = flat.shape[0] - 2
    entries = rng.integers(0, 0x38, (2, 64, 352), dtype=np.uint8)
    q, _ = queries(rng, 1, 16, 576)
    got = []
    for first in (0, last):
        flat[first:first + 2] = dev(entries)
        bt = dev(np.arange(first, first + 2, dtype=np.int32)[None])
        got.append(g.tree_attention_nvfp4_ds_mla(q, flat, bt, starts, lens, None, 115, 0.1))
    assert torch.equal(got[0], got[1]) and (got[0] != 0).any()


def test_empty_calls(g):
    one = torch.ones(1, device="cuda")
    cache = torch.zeros((0, 2, 16, 1, 72), dtype=torch.uint8, device="cuda")
    q = torch.ones(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    bt = torch.zeros((1, 3), dtype=torch.int32, device="cuda")
    st, ln = dev(np.array([0, 2], np.int32)), dev(np.array([9], np.int32))
    out, lse = g.attention_nvfp4_kv(q, cache, one, one, bt, st, ln, 9, 1.0, return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()    # a cache without blocks: nothing to see
    out = g.attention_nvfp4_kv(q[:0], cache, one, one, bt, dev(np.zeros(2, np.int32)), ln, 9, 1.0)
    assert out.shape == (0, 2, 128)


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def random_state(rng, rows, nb, bs, stride, share=0.2):
    lens, table = np.zeros(rows, np.int32), np.full((rows, stride), -1, np.int32)
    refs = np.zeros(nb, np.int32)
    free = list(rng.permutation(nb))
    for r in range(rows):
        if rng.random() < 0.3:
            continue
        n = int(rng.integers(0, stride * bs + 1))
        k = ref.pages(n, bs)
        if k > len(free):
            continue
        own = [free.pop() for _ in range(k)]
        for j in range(k - 1):                               # full pages may be shared
            if rng.random() < share and (refs > 0).any():
                free.append(own[j])
                own[j] = int(rng.choice(np.nonzero(refs > 0)[0]))
        table[r, :k], lens[r] = own, n
        for page in own:
            refs[page] += 1
    return table, lens, refs


def check_pages(call, model, state, caches):
    """Run `call` on the GPU copies and `model` on the CPU state; compare all."""
    table, lens, refs = (a.copy() for a in state)
    d = [dev(a) for a in state]
    gpu = [dev(c) for c in caches]
    got = call(*d, gpu)
    torch.cuda.synchronize()
    mine = [c.copy() for c in caches]
    want = model(table, lens, refs, mine)
    for n, a, b in (("table", d[0], table), ("lens", d[1], lens), ("refs", d[2], refs)):
        assert np.array_equal(host(a), b), n
    if want is not None:
        assert np.array_equal(host(got), want)
    for i, (a, b) in enumerate(zip(gpu, mine)):
        assert np.array_equal(host(a), b), f"cache {i}"
    return table, lens, refs


PAGES = [(5, 20, 4, 6, 1, 96), (40, 200, 16, 9, 3, 352), (300, 3000, 1, 30, 2, 40), (17, 64, 5, 8, 2, 7), (64, 5000, 64, 90, 1, 1024),
         (9, 30, 3, 5, 70, 12)]


@pytest.mark.parametrize("rows,nb,bs,stride,layers,page", PAGES)
def test_fork_extend_free_compact(g, rows, nb, bs, stride, layers, page):
    rng = np.random.default_rng(rows)
    state = random_state(rng, rows, nb, bs, stride)
    caches = [rng.integers(0, 256, (nb, page), dtype=np.uint8) for _ in range(layers)]
    i32 = np.int32
    n = rows + 5
    parents = rng.integers(-2, rows + 2, n).astype(i32)      # bad rows, duplicates, occupied children among them
    children = rng.integers(-2, rows + 2, n).astype(i32)
    state = check_pages(lambda t, l, r, c: g.fork_requests(c, bs, t, l, r, dev(parents), dev(children)),
                        lambda t, l, r, c: ref.fork(t, l, r, parents, children, bs, c), state, caches)
    which = rng.integers(-1, rows + 1, n).astype(i32)
    new = (state[1][np.clip(which, 0, rows - 1)] + rng.integers(-1, 3 * bs, n)).astype(i32)
    state = check_pages(lambda t, l, r, c: g.extend_requests(bs, t, l, r, dev(which), dev(new)),
                        lambda t, l, r, c: ref.extend(t, l, r, which, new, bs), state, caches)
    gone = rng.integers(-1, rows + 1, max(1, rows // 3)).astype(i32)
    state = check_pages(lambda t, l, r, c: g.free_requests(bs, t, l, r, dev(gone)),
                        lambda t, l, r, c: ref.free(t, l, r, gone, bs), state, caches)
    check_pages(lambda t, l, r, c: g.compact_pages(c, bs, t, l, r),
                lambda t, l, r, c: ref.compact(t, l, r, bs, c), state, caches)


@pytest.mark.parametrize("n", [1024, 1025, 5000])
def test_many_grants(g, n):
    """Calls of more requests than one workgroup's: duplicates and rows that are
    taken among them, free pages for some."""
    rng = np.random.default_rng(n)
    rows, nb, bs, stride = 3 * n // 2, 2 * n, 8, 3
    state = random_state(rng, rows, nb, bs, stride)
    caches = [rng.integers(0, 256, (nb, 24), dtype=np.uint8)]
    parents, children = (rng.integers(-1, rows + 1, n).astype(np.int32) for _ in range(2))
    state = check_pages(lambda t, l, r, c: g.fork_requests(c, bs, t, l, r, dev(parents), dev(children)),
                        lambda t, l, r, c: ref.fork(t, l, r, parents, children, bs, c), state, caches)
    which = rng.integers(-1, rows + 1, n).astype(np.int32)
    new = (state[1][np.clip(which, 0, rows - 1)] + rng.integers(0, 2 * bs, n)).astype(np.int32)
    check_pages(lambda t, l, r, c: g.extend_requests(bs, t, l, r, dev(which), dev(new)),
                lambda t, l, r, c: ref.extend(t, l, r, which, new, bs), state, caches)


@pytest.mark.parametrize("live", ["none", "all", "low", "high"])
def test_compact_borders(g, live):
    nb, bs = 9000, 4
    rng = np.random.default_rng(1)
    refs = np.zeros(nb, np.int32)
    at = {"none": [], "all": np.arange(nb), "low": np.arange(5000), "high": np.arange(nb - 4100, nb)}[live]
    refs[at] = rng.integers(1, 4, len(at))
    table = np.full((2, 40), -1, np.int32)
    lens = np.zeros(2, np.int32)
    if len(at):
        table[1, :37] = rng.choice(at, 37)
        lens[1] = 37 * bs - 3
    table[1, 5] = nb + 3                                     # an id outside: carried along
    caches = [rng.integers(0, 256, (nb, 48), dtype=np.uint8)]
    check_pages(lambda t, l, r, c: g.compact_pages(c, bs, t, l, r),
                lambda t, l, r, c: ref.compact(t, l, r, bs, c), (table, lens, refs), caches)


def test_page_supply_runs_out(g):
    """Requests in order until the free pages do not suffice; the rest are
    refused and left as they were."""
    nb, bs = 12, 4
    refs = np.ones(nb, np.int32)
    refs[[2, 3, 7, 9, 11]] = 0
    table = np.full((6, 8), -1, np.int32)
    table[0, :2] = [0, 1]
    lens = np.array([7, 0, 0, 0, 0, 0], np.int32)
    i = lambda *v: np.array(v, np.int32)                     # noqa: E731
    caches = [np.arange(nb * 16, dtype=np.uint8).reshape(nb, 16)]
    for rows, new in ((i(1, 2, 3, 4), i(8, 5, 4, 1)), (i(1, 2, 3), i(8, 16, 1)), (i(5), i(20)), (i(5), i(21)),
                      (i(0, 1), i(2 ** 31 - 1, 4))):
        check_pages(lambda t, l, r, c: g.extend_requests(bs, t, l, r, dev(rows), dev(new)),
                    lambda t, l, r, c: ref.extend(t, l, r, rows, new, bs), (table, lens, refs), caches)
    par, chi = i(0, 0, 0, 0, 0, 0), i(1, 2, 2, 3, 4, 5)
    refs[[7, 9]] = 1
    check_pages(lambda t, l, r, c: g.fork_requests(c, bs, t, l, r, dev(par), dev(chi)),
                lambda t, l, r, c: ref.fork(t, l, r, par, chi, bs, c), (table, lens, refs), caches)


@pytest.mark.parametrize("page,pad", [(22528, 0), (40, 0), (41, 3), (6, 2), (20000, 16)])
def test_copy_pages(g, page, pad):
    """Alignments from bytes to 16-byte pieces; padding between pages and
    pairs outside the cache are left alone."""
    rng = np.random.default_rng(page)
    nb = 40
    flat = [rng.integers(0, 256, (nb, page + pad), dtype=np.uint8) for _ in range(3)]
    order = rng.permutation(nb).astype(np.int32)
    src, dst = order[:15].copy(), order[15:30].copy()
    src[3], dst[5] = -1, nb
    src[8] = src[9]
    gpu = [dev(f) for f in flat]
    g.copy_pages([f[:, :page] for f in gpu], dev(src), dev(dst))
    for f, d in zip(flat, gpu):
        for a, b in zip(src, dst):
            if 0 <= a < nb and 0 <= b < nb:
                f[b, :page] = f[a, :page]
        assert np.array_equal(host(d), f)


# ---------------------------------------------------------------------------
# together, streams, graphs
# ---------------------------------------------------------------------------
class Serving:
    """Two layers of a small model's cache, requests on rows, everything on the
    device: prompt, fork, drafts, attention, free, compact."""

    def __init__(self, g, seed=0):
        self.g, self.bs, self.hk, self.hq, self.hs = g, 16, 2, 8, 64
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.nb, self.rows = 64, 6
        full = self.hs // 2 + self.hs // 16
        self.caches = [torch.full((self.nb, 2, self.bs, self.hk, full), 0xFF, dtype=torch.uint8, device="cuda")
                       for _ in range(2)]
        self.table = torch.full((self.rows, 12), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(self.rows, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(self.nb, dtype=torch.int32, device="cuda")
        self.state = (self.bs, self.table, self.lens, self.refs)
        self.one = torch.ones(1, device="cuda")
        self.w = torch.ones(self.hs, dtype=torch.bfloat16, device="cuda")
        ang = torch.arange(256, device="cuda")[:, None] * 0.5 ** torch.arange(self.hs // 2, device="cuda")
        self.cs = torch.cat([ang.cos(), ang.sin()], 1).float()

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda").to(torch.bfloat16)

    def step(self, row, n):
        """n new tokens of a row: extend, norm and rotate, write both layers.
        Returns the rotated queries."""
        i32 = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")      # noqa: E731
        old = int(self.lens[row])
        assert int(self.g.extend_requests(*self.state, i32(row), i32(old + n))) == 1
        pos = torch.arange(old, old + n, device="cuda")
        q, k, v = self.normal(n, self.hq, self.hs), self.normal(n, self.hk, self.hs), self.normal(n, self.hk, self.hs)
        q, k = self.g.qk_norm_rope(q, k, self.w, self.w, pos, self.cs)
        slots = self.table[row, pos // self.bs].long() * self.bs + pos % self.bs
        for c in self.caches:
            self.g.reshape_and_cache_nvfp4(k, v, c, slots, self.one, self.one)
        return q

    def attend(self, q, row, n, mask=None, layer=0):
        st = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        head = (q, self.caches[layer], self.one, self.one, self.table[row:row + 1], st, self.lens[row:row + 1])
        if mask is None:
            return self.g.attention_nvfp4_kv(*head, 192, self.hs ** -0.5, window=40, num_sinks=4)
        return self.g.tree_attention_nvfp4_kv(*head, mask, 192, self.hs ** -0.5)


def test_serving_steps_together(g):
    """Norm and rotation -> cache write -> fork -> tree attention -> free ->
    compact: attention over a fork equals attention over its parent bit for
    bit, writes to the fork leave the parent alone, compaction changes no
    output, and an output agrees with the 64-bit reference of what the
    existing gather reads back from the cache."""
    s = Serving(g)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")           # noqa: E731
    s.step(4, 30)                                            # a request in between, to make holes
    q = s.step(0, 75)
    s.step(5, 50)
    before = s.attend(q, 0, 75)
    assert g.fork_requests(s.caches, *s.state, i32(0, 0), i32(1, 2)).tolist() == [1, 1]
    assert torch.equal(s.attend(q, 1, 75), before) and torch.equal(s.attend(q, 2, 75, layer=1), before)
    qd = s.step(1, 7)                                        # seven drafted tokens on the fork
    assert torch.equal(s.attend(q, 0, 75), before)
    mask = torch.eye(7, dtype=torch.bool, device="cuda")
    mask[3:, 0] = True
    mask[5:, 3] = True
    drafts = s.attend(qd, 1, 7, mask)
    # the same attention from the gather's bf16 copy of the cache, in 64 bits
    k = torch.empty(82, s.hk, s.hs, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    g.gather_upconvert_nvfp4_kv(s.caches[0], k, v, s.table[1:2].contiguous(), i32(0), s.one, s.one)
    see = np.repeat(ref.tree(7, 82, host(mask)), 4, 0)
    for h in range(s.hk):
        o, _, ot, _ = ref.attend(qd.double().cpu().numpy()[:, 4 * h:4 * h + 4].reshape(-1, s.hs),
                                 k[:, h].double().cpu().numpy(), v[:, h].double().cpu().numpy(), see, s.hs ** -0.5)
        close(drafts[:, 4 * h:4 * h + 4].reshape(-1, s.hs), o, ot, f"drafts head {h}")
    g.free_requests(*s.state, i32(4, 2))
    page_map = g.compact_pages(s.caches, *s.state)
    live = int((s.refs > 0).sum())
    assert (s.refs[:live] > 0).all() and int(page_map.max()) == live - 1
    assert torch.equal(s.attend(q, 0, 75), before) and torch.equal(s.attend(qd, 1, 7, mask), drafts)
    assert torch.equal(s.attend(qd, 1, 7, mask, layer=1), drafts)
    g.free_requests(*s.state, i32(0, 1, 5))
    assert int(s.refs.abs().sum()) == 0 and (s.table == -1).all() and int(s.lens.abs().sum()) == 0


def test_other_streams_and_two_calls_at_once(g):
    """Calls on two other streams at the same time, each with its own scratch,
    give the bits of the same calls one after the other."""
    rng = np.random.default_rng(6)
    batch = Batch(rng, [1, 2], [1500, 700], 16)
    _, cache, L = kv_cache(g, rng, batch, 1, 128, "split")
    q, _ = queries(rng, batch.T, 8, 128)
    bt, starts, lens = batch.metadata()
    one = torch.ones(1, device="cuda")
    call = lambda w, **kw: g.attention_nvfp4_kv(q, cache, one, one, bt, starts, lens, 1500, 0.09, window=w,      # noqa: E731
                                                num_sinks=4, **kw)
    want = [call(None), call(900)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [call(w, stream=s) for w, s in zip((None, 900), streams)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_graph_replay(g):
    """One decoding step (extend, norm, write, split attention, fork, free,
    compact) captured once and replayed with new contents: every replay has
    the eager results."""
    def inputs(seed):
        s = Serving(g, seed)
        s.step(0, 140)
        s.step(3, 20)
        return s, s.normal(1, s.hq, s.hs), s.normal(1, s.hk, s.hs), s.normal(1, s.hk, s.hs)

    def step(s, q, k, v, out):
        ids = step.ids
        g.extend_requests(*s.state, ids["row"], s.lens[:1] + 1)
        pos = s.lens[:1].long() - 1
        qr, kr = g.qk_norm_rope(q, k, s.w, s.w, pos, s.cs)
        slots = s.table[0].gather(0, pos // s.bs).long() * s.bs + pos % s.bs
        g.reshape_and_cache_nvfp4(kr, v, s.caches[0], slots, s.one, s.one)
        a = g.attention_nvfp4_kv(qr, s.caches[0], s.one, s.one, s.table[:1], ids["starts"], s.lens[:1], 4096, 0.1)
        g.fork_requests(s.caches, *s.state, ids["row"], ids["child"])
        g.free_requests(*s.state, ids["gone"])
        m = g.compact_pages(s.caches, *s.state)
        out[:-s.nb].copy_(a.reshape(-1))
        out[-s.nb:].copy_(m)

    step.ids = {k: torch.tensor(v, dtype=torch.int32, device="cuda")
                for k, v in (("row", [0]), ("child", [2]), ("gone", [3]), ("starts", [0, 1]))}
    live = inputs(1)
    out = torch.zeros(8 * 64 + 64, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(*live, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*live, out)
    state = (*live[0].caches, live[0].table, live[0].lens, live[0].refs)
    for seed in (1, 2, 3):
        fresh = inputs(seed)
        want = torch.zeros_like(out)
        for dst, src in zip((*state, *live[1:]),
                            (*fresh[0].caches, fresh[0].table, fresh[0].lens, fresh[0].refs, *fresh[1:])):
            dst.copy_(src)
        step(*fresh, want)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), seed
        for a, b in zip(state, (*fresh[0].caches, fresh[0].table, fresh[0].lens, fresh[0].refs)):
            assert torch.equal(a, b), seed


@pytest.mark.parametrize("n", [1, 3, 1024, 1025])
@pytest.mark.parametrize("beyond", [0, 1, 4])
def test_extend_of_an_unused_pool(g, n, beyond):
    """All pages free and tables wider than the pool: a request for every page
    is granted, one for more is refused and leaves the state as it was, and so
    do the requests behind it.  Both planning kernels."""
    nb, bs = 6, 16
    rows = np.arange(n, dtype=np.int32)
    new = np.full(n, bs, np.int32)
    new[0] = (nb + beyond) * bs - 3
    state = (np.full((n, nb + 5), -9, np.int32), np.zeros(n, np.int32), np.zeros(nb, np.int32))
    table, lens, refs = check_pages(lambda t, l, r, c: g.extend_requests(bs, t, l, r, dev(rows), dev(new)),
                                    lambda t, l, r, c: ref.extend(t, l, r, rows, new, bs), state, [])
    if beyond:
        assert (table == -9).all() and not lens.any() and not refs.any()
    else:
        assert table[0, :nb].tolist() == list(range(nb)) and lens[0] == new[0]


def far_cache(g, flat, L, nb, bs, hk, hs, far):
    """The entries of `flat` (layout L) in an allocation of over 4 GiB: K and V
    planes apart ("planes"), or the heads' data and scales ("heads")."""
    full = hs // 2 + hs // 16
    apart = (1 << 32) + 4096
    d, s = bs * hs // 2, bs * hs // 16                       # a page's data and scales of one head
    if far == "planes":
        F = g.NvFp4KvLayout(data_offset=0, data_token_stride=hk * hs // 2, data_head_stride=hs // 2, scale_offset=hk * d,
                     scale_token_stride=hk * hs // 16, scale_head_stride=hs // 16, side_stride=apart,
                     block_stride=(hk * (d + s) + 7) // 8 * 8)
    else:
        page = (d + s + 7) // 8 * 8
        F = g.NvFp4KvLayout(data_offset=0, data_token_stride=hs // 2, data_head_stride=apart, scale_offset=d,
                     scale_token_stride=hs // 16, scale_head_stride=apart, side_stride=page, block_stride=2 * page)
    big = torch.full(((hk - 1) * F.data_head_stride + F.side_stride + nb * F.block_stride + 64,), 0xFF, dtype=torch.uint8,
                     device="cuda")
    for side, h, (what, n) in itertools.product((0, 1), range(hk), (("data", hs // 2), ("scale", hs // 16))):
        at = lambda X, base: torch.as_strided(               # noqa: E731
            base, (nb, bs, n), (X.block_stride, getattr(X, what + "_token_stride"), 1),
            getattr(X, what + "_offset") + side * X.side_stride + h * getattr(X, what + "_head_stride"))
        at(F, big).copy_(at(L, torch.from_numpy(flat)))
    return torch.as_strided(big, (nb, 2, bs, hk, full), (F.block_stride, F.side_stride, hk * full, full, 1)), F


@pytest.mark.parametrize("far", ["planes", "heads"])
@pytest.mark.parametrize("hs,bs,qlens", [(128, 16, [1, 2]), (80, 24, [1, 3]), (256, 16, [1, 1]), (64, 16, [40, 1]),
                                         (128, 16, [70, 3]), (176, 8, [33, 1])])
def test_strides_past_32_bits(g, hs, bs, qlens, far):
    """Sides and heads more than 4 GiB apart, few rows and many."""
    rng = np.random.default_rng(hs + bs)
    hk, group, lens = 2, 4, [150, 71]
    batch = Batch(rng, qlens, lens, bs)
    flat, _, L = kv_cache(g, rng, batch, hk, hs, "split")
    cache, F = far_cache(g, flat, L, batch.nb, bs, hk, hs, far)
    q, q64 = queries(rng, batch.T, hk * group, hs)
    bt, starts, sl = batch.metadata()
    one = torch.ones(1, device="cuda")
    scale = 0.0625
    out, lse = g.attention_nvfp4_kv(q, cache, one, one, bt, starts, sl, 150, scale, layout=F, return_lse=True)
    for b, (n, length) in enumerate(zip(qlens, lens)):
        r0 = int(batch.starts[b])
        see = np.repeat(ref.causal(n, length), group, 0)
        for h in range(hk):
            k, v, _ = ref.kv_positions(flat, L, batch.table[b], length, bs, batch.nb, h, hs)
            o, l, ot, lt = ref.attend(q64[r0:r0 + n, h * group:(h + 1) * group].reshape(-1, hs), k, v, see, scale)
            close(out[r0:r0 + n, h * group:(h + 1) * group].reshape(-1, hs), o, ot, f"request {b} head {h} out")
            close(lse[r0:r0 + n, h * group:(h + 1) * group].reshape(-1), l, lt, f"request {b} head {h} lse")


def test_windows_and_sinks_past_32_bits(g):
    """A window or a number of sinks of 2^31 and more covers every position:
    the answers are those without it.  Sizes of pages that no int32 holds
    are refused."""
    rng = np.random.default_rng(31)
    batch = Batch(rng, [1, 40], [200, 90], 16)
    _, cache, L = kv_cache(g, rng, batch, 1, 64, "split")
    q, _ = queries(rng, batch.T, 2, 64)
    bt, starts, lens = batch.metadata()
    one = torch.ones(1, device="cuda")
    call = lambda **kw: g.attention_nvfp4_kv(q, cache, one, one, bt, starts, lens, 200, 0.125, **kw)      # noqa: E731
    wide = 1 << 30                                           # beyond any position, within int32
    for kw, same in ((dict(window=(1 << 32) + 8), {}), (dict(window=1 << 31), {}), (dict(window=(1 << 63) - 1, num_sinks=3), {}),
                     (dict(window=7, num_sinks=1 << 32), dict(window=7, num_sinks=wide)),
                     (dict(window=1, num_sinks=(1 << 40) + 1), dict(window=1, num_sinks=wide))):
        assert torch.equal(call(**kw), call(**same)), kw
    for kw in (dict(window=0), dict(window=-(1 << 32) + 5), dict(window=4, num_sinks=-(1 << 32))):
        with pytest.raises((ValueError, RuntimeError)):
            call(**kw)
    refs = torch.zeros(batch.nb, dtype=torch.int32, device="cuda")
    for bs in ((1 << 32) + 16, 1 << 31, 0, -16):
        with pytest.raises((ValueError, RuntimeError)):
            g.free_requests(bs, bt, lens, refs, lens[:1])
        with pytest.raises((ValueError, RuntimeError)):
            g.extend_requests(bs, bt, lens, refs, lens[:1], lens[:1])


@pytest.mark.parametrize("hs,rot,inter", [(128, 128, False), (64, 32, True), (256, 96, False), (16, 16, True), (80, 0, False),
                                          (512, 64, False)])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-6])
def test_qk_norm_rope_magnitudes(g, hs, rot, inter, eps):
    """Heads of every magnitude bf16 has, whose mean square leaves binary32 at
    either end, beside ordinary ones in the same token; eps may be 0."""
    rng = np.random.default_rng(hs)
    T, hq, hk = 6, 7, 2
    x = rng.standard_normal((T, hq + hk, hs))
    power = rng.choice([-130, -124, -110, -80, -63, -62, -50, -30, 0, 30, 59, 61, 64, 100, 124], (T, hq + hk, 1))
    qk, qk64 = ref.bf16(x * 2.0 ** power)
    qk = qk.cuda()
    w = [ref.bf16(1 + 0.3 * rng.standard_normal(hs)) for _ in range(2)]
    pos = rng.integers(0, 30, T)
    ang = np.arange(30)[:, None] * 3.0 ** -np.arange(rot // 2)
    table = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))
    cs = table.cuda() if rot else None
    q, k = g.qk_norm_rope(qk[:, :hq], qk[:, hq:], w[0][0].cuda(), w[1][0].cuda(), dev(pos), cs, eps=eps, interleaved=inter)
    for out, at, wt, n in ((q, slice(0, hq), w[0][1], "q"), (k, slice(hq, None), w[1][1], "k")):
        want, tol = ref.norm_rope(qk64[:, at], wt, pos, table.double().numpy(), rot, float(np.float32(eps)), inter)
        close(out, want, tol, n)


def kv_bytes(flat, L, blk, off, hk, hs):
    """Views of every data and scale byte of one position, all heads, K and V."""
    for side in (0, 1):
        for h in range(hk):
            base = blk * L.block_stride + side * L.side_stride
            d = base + L.data_offset + off * L.data_token_stride + h * L.data_head_stride
            s = base + L.scale_offset + off * L.scale_token_stride + h * L.scale_head_stride
            yield flat[d:d + hs // 2]
            yield flat[s:s + hs // 16]


@pytest.mark.parametrize("hs,bs,qlens", [(128, 16, [1, 3]), (80, 24, [2, 1]), (256, 16, [1, 2]), (64, 16, [45, 2]),
                                         (128, 16, [130, 40]), (176, 8, [50, 1])])
def test_nan_bytes_before_a_window(g, hs, bs, qlens):
    """Positions of the sequence that the window hides from every row, in tiles
    that other positions share, hold NaN codes in all bytes: the outputs are
    those with ordinary bytes there."""
    rng = np.random.default_rng(hs + bs + 1)
    window, sinks, lens, hk = 21, 5, [233, 150], 2
    batch = Batch(rng, qlens, lens, bs)
    flat, cache, L = kv_cache(g, rng, batch, hk, hs, "split")
    q, _ = queries(rng, batch.T, 4 * hk, hs)
    bt, starts, sl = batch.metadata()
    one = torch.ones(1, device="cuda")
    call = lambda c: g.attention_nvfp4_kv(q, c, one, one, bt, starts, sl, 233, 0.1, window=window, num_sinks=sinks,     # noqa: E731
                                          layout=L, return_lse=True)
    want = call(cache)
    hidden = 0
    for b, (n, length) in enumerate(zip(qlens, lens)):
        for p in np.nonzero(~ref.causal(n, length, window, sinks).any(0))[0]:
            hidden += 1
            for x in kv_bytes(flat, L, int(batch.table[b, p // bs]), int(p) % bs, hk, hs):
                x[:] = 0xFF
    assert hidden > 150
    got = call(torch.as_strided(dev(flat), cache.shape, cache.stride()))
    assert torch.isfinite(got[0]).all() and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("hs,bs", [(128, 16), (80, 24), (256, 16)])
@pytest.mark.parametrize("n", [5, 40])
def test_nan_bytes_of_hidden_drafts(g, hs, bs, n):
    """Drafted tokens that no row's mask names, per-head cache."""
    rng = np.random.default_rng(hs + n)
    batch = Batch(rng, [n], [70 + n], bs)
    flat, cache, L = kv_cache(g, rng, batch, 1, hs, "split")
    q, _ = queries(rng, n, 4, hs)
    bt, starts, sl = batch.metadata()
    one = torch.ones(1, device="cuda")
    mask = rng.random((n, n)) < 0.6
    mask[:, 1::3] = False
    call = lambda c: g.tree_attention_nvfp4_kv(q, c, one, one, bt, starts, sl, dev(mask), 110, 0.1, layout=L,      # noqa: E731
                                               return_lse=True)
    want = call(cache)
    for p in range(71, 70 + n, 3):
        for x in kv_bytes(flat, L, int(batch.table[0, p // bs]), p % bs, 1, hs):
            x[:] = 0xFF
    got = call(torch.as_strided(dev(flat), cache.shape, cache.stride()))
    assert torch.isfinite(got[0]).all() and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("bs", [64, 40])
@pytest.mark.parametrize("n,heads", [(4, 4), (9, 2), (20, 8)])
def test_nan_bytes_of_hidden_latent_drafts(g, bs, n, heads):
    """The same over the latent cache, RoPE bytes too, in the kernel for few rows and the one for many."""
    rng = np.random.default_rng(bs + n)
    batch = Batch(rng, [n], [75 + n], bs)
    flat = np.full((batch.nb, bs, 352), 0xFF, np.uint8)
    for p in range(75 + n):
        e = flat[batch.table[0, p // bs], p % bs]
        e[:256], e[320:352] = fp4_bytes(rng, 256), scale_bytes(rng, 32)
        e[256:320] = rng.integers(0, 0x48, 64, dtype=np.uint8)
    q, _ = queries(rng, n, heads, 576)
    bt, starts, sl = batch.metadata()
    mask = rng.random((n, n)) < 0.6
    mask[:, 1::3] = False
    call = lambda: g.tree_attention_nvfp4_ds_mla(q, dev(flat), bt, starts, sl, dev(mask), 100, 0.07, return_lse=True)       # noqa: E731
    want = call()
    for p in range(76, 75 + n, 3):
        flat[batch.table[0, p // bs], p % bs] = 0xFF
    got = call()
    assert torch.isfinite(got[0]).all() and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("hq,hk", [(1, 0), (4, 1), (20, 3), (23, 1), (24, 1), (25, 0), (28, 4), (40, 9), (49, 24), (97, 2)])
def test_qk_norm_rope_head_counts(g, hq, hk):
    """Head counts around what one, two and more waves of a token hold, in place:
    every head is normed once."""
    rng = np.random.default_rng(hq)
    T, hs = 5, 128
    qk, qk64 = ref.bf16(rng.standard_normal((T, hq + hk, hs)))
    qk = qk.cuda()
    w, w64 = ref.bf16(1 + 0.3 * rng.standard_normal(hs))
    ang = np.arange(9)[:, None] * 2.0 ** -np.arange(hs // 2)
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pos = rng.integers(0, 9, T)
    q, k = qk[:, :hq], qk[:, hq:] if hk else None
    g.qk_norm_rope(q, k, w.cuda(), w.cuda() if hk else None, dev(pos), dev(table), eps=1e-6, q_out=q, k_out=k)
    want, tol = ref.norm_rope(qk64, w64, pos, table.astype(np.float64), hs, float(np.float32(1e-6)), False)
    close(qk, want, tol, "q and k")


@pytest.mark.parametrize("requests,length", [(3, 40), (2, 1700), (1025, 20)])
@pytest.mark.parametrize("hs", [64, 576])
def test_rows_before_the_first_request(g, requests, length, hs):
    """query_starts that begin behind row 0: the rows before are left as they
    were, for short, split and large batches."""
    rng = np.random.default_rng(requests)
    before, n, heads = 37, 2, 2
    batch = Batch(rng, [n] * requests, [length] * requests, 16)
    bt, starts, lens = batch.metadata()
    q, q64 = queries(rng, before + batch.T, heads, hs)
    scale, dv = 0.0625, min(hs, 512)
    kw = dict(out=torch.full((before + batch.T, heads, dv), 7.0, dtype=torch.bfloat16, device="cuda"),
              lse=torch.full((before + batch.T, heads), 7.0, device="cuda"))
    if hs == 576:
        flat = rng.integers(0, 0x38, (batch.nb, 16, 352), dtype=np.uint8)
        g.tree_attention_nvfp4_ds_mla(q, dev(flat), bt, starts + before, lens, None, length, scale, **kw)
    else:
        flat, one = rng.integers(0, 0x38, (batch.nb, 2, 16, 1, hs // 2 + hs // 16), dtype=np.uint8), torch.ones(1, device="cuda")
        g.attention_nvfp4_kv(q, dev(flat), one, one, bt, starts + before, lens, length, scale, **kw)
    assert (kw["out"][:before] == 7).all() and (kw["lse"][:before] == 7).all()
    see = np.repeat(ref.causal(n, length), heads, 0)
    for b in {0, requests // 2, requests - 1}:
        row = batch.table[b]
        if hs == 576:
            k, v, _ = ref.mla_positions(flat.reshape(-1), row, length, 16, batch.nb, 16 * 352, 352)
        else:
            k, v, _ = ref.kv_positions(flat.reshape(-1), g.nvfp4_kv_split_layout(16, 1, hs), row, length, 16, batch.nb, 0, hs)
        at = slice(before + n * b, before + n * (b + 1))
        o, l, ot, lt = ref.attend(q64[at].reshape(-1, hs), k, v, see, scale)
        close(kw["out"][at].reshape(-1, dv), o, ot, f"request {b} out")
        close(kw["lse"][at].reshape(-1), l, lt, f"request {b} lse")
