"""GPU tests of the 8-bit paged cache and of the prompts' attention at the edges
of what their headers allow: value scales over the whole range, values that are
not finite in every form of the prompt kernel, and every form that a call's
sizes select."""
import numpy as np
import pytest
import torch

import serving_refs as ref
from gpu_util import dev
from test_operators_gpu import Batch, close
from test_serving_gpu import cache_view, g, random_codes  # noqa: F401

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


@pytest.mark.parametrize("qlens", [[1, 2], [5, 6], [40, 30]])
def test_cache_least_scales_alone(g, qlens):  # noqa: F811
    rng = np.random.default_rng(1)
    batch = Batch(rng, qlens, [300, 200], 16)
    codes = random_codes(rng, (batch.nb, 2, 16, 1, 64))
    scales = np.full((batch.nb, 2, 1), 2.0 ** -9, np.float32)
    scales[:, 1] = (2.0 ** -rng.integers(96, 101, (batch.nb, 1))).astype(np.float32)
    check_scaled(g, batch, 1, 4, 64, codes, scales, rng.standard_normal((batch.T, 4, 64)), 0.125)
