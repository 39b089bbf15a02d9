"""Checks of the operators around the cache that need no GPU: exported
symbols, refusals on the host before any HIP call, the key-split workspace,
and the references' own definitions."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

import operator_refs as ref
from conftest import ROOT

A16 = 0x10000      # never dereferenced: every call below is refused or empty


@pytest.fixture(scope="module")
def lib():
    from gather_concat_cache_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    from gather_concat_cache_amd import _operators
    return _operators._load()


def declared(header):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(gcache_[a-z0-9_]+)\s*\(", text)))


def test_declared_symbols_are_bound(lib):
    import gather_concat_cache_amd as g
    from gather_concat_cache_amd import _operators
    names = declared("gcache_attention.h") + declared("gcache_pages.h")
    assert sorted(names) == sorted(_operators._SIGS)
    for n in names:
        assert hasattr(lib, n)
        if not n.endswith("workspace_bytes"):
            assert callable(getattr(g, n)) and getattr(g, n) is getattr(g, n[len("gcache_"):])


def test_public_headers_compile_as_c(tmp_path):
    import shutil
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "gcache_attention.h"\n#include "gcache_pages.h"\nint main(void) { gcache_attention_args a; '
                   "gcache_page_state s; return (int)(sizeof a + sizeof s) == 0; }\n")
    cc = shutil.which("gcc")
    subprocess.run([cc, "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                    "/opt/rocm/include", "-fsyntax-only", str(src)], check=True)


def _args(**kw):
    from gather_concat_cache_amd._operators import AttentionArgs
    a = dict(q=A16, out=A16, lse=A16, q_token_stride=1024, q_head_stride=128, out_token_stride=1024,
             out_head_stride=128, lse_token_stride=8, query_starts=A16, seq_lens=A16, block_table=A16,
             block_table_stride=4, total_q=5, max_seq_len=64, num_blocks=9, batch_size=2, num_q_heads=8, block_size=16,
             softmax_scale=0.1, workspace=None, workspace_bytes=0)
    a.update(kw)
    return AttentionArgs(**a)


BAD_ARGS = [
    (dict(total_q=-1), -2), (dict(batch_size=-1), -2), (dict(q=None), -1), (dict(out=None), -1),
    (dict(query_starts=None), -1), (dict(seq_lens=None), -1), (dict(block_table=None), -1), (dict(num_q_heads=0), -2),
    (dict(block_size=0), -2), (dict(block_table_stride=0), -2), (dict(num_blocks=-1), -2), (dict(max_seq_len=-1), -2),
    (dict(workspace_bytes=-4), -2), (dict(total_q=1 << 30), -2), (dict(q_token_stride=-8), -2),
    (dict(out_head_stride=120), -2), (dict(out_token_stride=64), -2), (dict(lse_token_stride=7), -2),
    (dict(softmax_scale=float("nan")), -2), (dict(softmax_scale=float("inf")), -2), (dict(q=A16 + 8), -3),
    (dict(out=A16 + 2), -3), (dict(q_token_stride=1028), -3), (dict(out_head_stride=132), -3),
    (dict(workspace=A16 + 8), -3), (dict(lse=A16 + 2), -3),
]


@pytest.mark.parametrize("change,status", BAD_ARGS)
def test_attention_refusals(lib, change, status):
    import gather_concat_cache_amd as g
    L = g.nvfp4_kv_split_layout(16, 2, 128)
    a = _args(**change)
    assert lib.gcache_attention_nvfp4_kv(C.byref(a), A16, C.byref(L), A16, A16, 2, 128, 0, 0, None) == status
    assert lib.gcache_tree_attention_nvfp4_kv(C.byref(a), A16, C.byref(L), A16, A16, 2, 128, A16, 8, 8, None) == status
    wide = {k: v for k, v in change.items()}
    a = _args(**{**dict(q_head_stride=576, q_token_stride=8 * 576, out_head_stride=512, out_token_stride=8 * 512), **wide})
    if "out_head_stride" not in change and "out_token_stride" not in change:
        assert lib.gcache_tree_attention_nvfp4_ds_mla(C.byref(a), A16, 64 * 352, 352, None, 0, 0, None) == status


def test_attention_cache_refusals(lib):
    import gather_concat_cache_amd as g
    L = g.nvfp4_kv_split_layout(16, 2, 128)
    a = _args()

    def kv(cache=A16, layout=L, ks=A16, vs=A16, hk=2, hs=128, w=0, s=0, args=a):
        return lib.gcache_attention_nvfp4_kv(args and C.byref(args), cache, layout and C.byref(layout), ks, vs, hk, hs, w, s,
                                             None)
    assert kv(args=None) == -1 and kv(cache=None) == -1 and kv(layout=None) == -1 and kv(ks=None) == -1
    assert kv(hs=120) == -2 and kv(hs=0) == -2 and kv(w=-1) == -2 and kv(s=-1) == -2 and kv(hk=3) == -2 and kv(hk=0) == -2
    assert kv(hs=272) == -4
    assert kv(cache=A16 + 8) == -3
    for field, value, status in (("data_head_stride", 60, -3), ("block_stride", -8, -2), ("side_stride", 4, -3),
                                 ("block_stride", (1 << 62), -2)):
        bad = g.NvFp4KvLayout(**{n: getattr(L, n) for n, _ in L._fields_})
        setattr(bad, field, value)
        assert kv(layout=bad) == status, field
    # nothing to do: accepted whatever else the call says
    assert kv(args=_args(total_q=0, q=None)) == 0 and kv(args=_args(batch_size=0, q=None)) == 0
    tree = lib.gcache_tree_attention_nvfp4_kv
    assert tree(C.byref(a), A16, C.byref(L), A16, A16, 2, 128, None, 8, 8, None) == -1
    assert tree(C.byref(a), A16, C.byref(L), A16, A16, 2, 128, A16, 7, 8, None) == -2
    assert tree(C.byref(a), A16, C.byref(L), A16, A16, 2, 128, A16, 7, -1, None) == -2
    m = _args(q_head_stride=576, q_token_stride=8 * 576, out_head_stride=512, out_token_stride=8 * 512)

    def mla(cache=A16, bstr=16 * 352, estr=352, mask=None, mts=0, cols=0):
        return lib.gcache_tree_attention_nvfp4_ds_mla(C.byref(m), cache, bstr, estr, mask, mts, cols, None)
    assert mla(cache=None) == -1 and mla(estr=336) == -2 and mla(bstr=15 * 352) == -2 and mla(cache=A16 + 8) == -3
    assert mla(estr=360, bstr=16 * 360) == -3 and mla(mask=A16, mts=3, cols=4) == -2


def test_workspace_bytes(lib):
    f = lib.gcache_attention_workspace_bytes
    assert f(0, 1, 8, 2, 128, 1000, 0, 0) == 0 and f(4, 0, 8, 2, 128, 1000, 0, 0) == 0
    assert f(4, 1, 8, 3, 128, 1000, 0, 0) == 0                # heads that do not divide
    one = f(1, 1, 8, 2, 128, 1 << 20, 0, 0)
    assert one > 0 and one % (8 * 130 * 4) == 0               # whole splits of (values, maximum, sum)
    assert f(1, 1, 8, 2, 128, 40, 0, 0) == 0                  # too short to split
    assert f(1, 1, 8, 2, 128, 1 << 20, 64, 4) < one           # the window bounds the keys
    for t, b, hq, hk, hs, n in ((1 << 20, 1, 32, 8, 128, 1 << 20), (1 << 24, 7, 64, 1, 576, 1 << 30)):
        assert 0 <= f(t, b, hq, hk, hs, n, 0, 0) < 1 << 40


def test_qk_norm_rope_refusals(lib):
    names = ("q k q_out k_out q_weight k_weight positions cos_sin cs16 max_pos cs_stride T hq hk hs rot inter eps qts "
             "qhs kts khs qots qohs kots kohs stream").split()
    good = dict(q=A16, k=A16, q_out=A16, k_out=A16, q_weight=A16, k_weight=A16, positions=A16, cos_sin=A16, cs16=0,
                max_pos=10, cs_stride=64, T=3, hq=4, hk=2, hs=64, rot=64, inter=0, eps=1e-6, qts=256, qhs=64, kts=128, khs=64,
                qots=256, qohs=64, kots=128, kohs=64, stream=None)

    def call(**kw):
        a = {**good, **kw}
        return lib.gcache_qk_norm_rope(*[a[n] for n in names])
    assert call(T=0, q=None) == 0 and call(T=-1) == -2
    for n in ("q", "k", "q_out", "k_out", "q_weight", "k_weight", "positions", "cos_sin"):
        assert call(**{n: None}) == -1, n
    for kw in (dict(hs=72), dict(hs=0), dict(rot=72), dict(rot=80), dict(rot=-16), dict(hq=0, hk=0), dict(hq=-1),
               dict(eps=-1.0), dict(eps=float("nan")), dict(max_pos=-1), dict(cs_stride=63), dict(qts=-8), dict(qohs=56),
               dict(kots=32), dict(T=1 << 62)):
        assert call(**kw) == -2, kw
    assert call(hs=528, rot=0) == -4
    for kw in (dict(q=A16 + 2), dict(k_out=A16 + 8), dict(q_weight=A16 + 2), dict(positions=A16 + 4), dict(cos_sin=A16 + 2),
               dict(qts=260), dict(khs=68)):
        assert call(**kw) == -3, kw


def test_page_refusals(lib):
    from gather_concat_cache_amd._operators import PageCaches, PageState
    ptrs = (C.c_void_p * 2)(A16, A16 + 64)

    def state(**kw):
        a = dict(block_table=A16, block_table_stride=4, seq_lens=A16, ref_counts=A16, num_blocks=9, num_rows=3, block_size=16)
        a.update(kw)
        return PageState(**a)

    def caches(**kw):
        a = dict(caches=C.cast(ptrs, C.c_void_p), num_caches=2, block_stride=96, page_bytes=96)
        a.update(kw)
        return PageCaches(**a)
    W = lib.gcache_pages_workspace_bytes(9, 3, 2)
    assert W > 0 and lib.gcache_pages_workspace_bytes(-1, 3, 2) == 0

    def fork(s=None, c=None, p=A16, ch=A16, n=2, st=A16, ws=A16, wb=W):
        return lib.gcache_fork_requests(C.byref(s or state()), C.byref(c or caches()), p, ch, n, st, ws, wb, None)

    def extend(s=None, r=A16, nl=A16, n=2, st=A16, ws=A16, wb=W):
        return lib.gcache_extend_requests(C.byref(s or state()), r, nl, n, st, ws, wb, None)

    def free(s=None, r=A16, n=2):
        return lib.gcache_free_requests(C.byref(s or state()), r, n, None)

    def compact(s=None, c=None, m=A16, ws=A16, wb=W):
        return lib.gcache_compact_pages(C.byref(s or state()), C.byref(c or caches()), m, ws, wb, None)

    def copy(c=None, nb=9, s=A16, d=A16, n=2):
        return lib.gcache_copy_pages(C.byref(c or caches()), nb, s, d, n, None)
    for bad, status in ((dict(block_table=None), -1), (dict(seq_lens=None), -1), (dict(ref_counts=None), -1),
                        (dict(num_blocks=0), -2), (dict(num_blocks=1 << 31), -2), (dict(num_rows=0), -2),
                        (dict(block_size=0), -2), (dict(block_table_stride=0), -2), (dict(seq_lens=A16 + 2), -3)):
        for f in (fork, extend, free, compact):
            assert f(s=state(**bad)) == status, (f.__name__, bad)
    for bad, status in ((dict(caches=None), -1), (dict(num_caches=-1), -2), (dict(page_bytes=97), -2), (dict(page_bytes=-1), -2),
                        (dict(block_stride=1 << 62, page_bytes=96), -2)):
        for f in (fork, compact, copy):
            assert f(c=caches(**bad)) == status, (f.__name__, bad)
    none = (C.c_void_p * 2)(A16, None)
    assert fork(c=caches(caches=C.cast(none, C.c_void_p))) == -1
    for f in (fork, extend):
        assert f(n=0) == 0 and f(n=-1) == -2 and f(n=(1 << 22) + 1) == -2 and f(st=None) == -1 and f(ws=None) == -1
        assert f(wb=W - 4) == -2 and f(ws=A16 + 2) == -3
    assert fork(p=None) == -1 and extend(nl=None) == -1 and free(r=None) == -1 and free(n=0) == 0 and free(n=-1) == -2
    assert compact(m=None) == -1 and compact(wb=0) == -2 and compact(m=A16 + 2) == -3
    assert copy(n=0) == 0 and copy(s=None) == -1 and copy(n=-1) == -2 and copy(d=A16 + 1) == -3


def test_binding_refuses_cpu_tensors_and_wrong_types():
    import gather_concat_cache_amd as g
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        g.qk_norm_rope(q, None, q[0, 0], None, i, None)
    with pytest.raises(ValueError):
        g.tree_attention_nvfp4_ds_mla(q, torch.zeros(1, 1, 352, dtype=torch.uint8), i[None], i, i[:1], None, 1, 1.0)
    with pytest.raises(TypeError):
        g.attention_nvfp4_kv(q, q, None, None, i[None], i, i[:1], 1, 1.0)
    with pytest.raises(ValueError):
        g.free_requests(16, i[None], i[:1], i, i)
    with pytest.raises(ValueError):
        g.copy_pages([], i, i)
    with pytest.raises(ValueError):
        g.copy_pages(torch.zeros(2, 4, dtype=torch.uint8), i, i)


def test_reference_decoders_agree_with_torch(orc):
    """The references' own e4m3 and e2m1 tables: against torch's float8 type,
    and an nvfp4 entry against the oracle's dequantizing gather."""
    b = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(b).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(ref.e4m3(b), t, equal_nan=True)
    rng = np.random.default_rng(0)
    e = rng.integers(0, 0x7F, 352, dtype=np.uint8)
    got = orc.gather_nvfp4_ds_mla(e, 1, np.zeros((1, 1), np.int32), np.zeros(1, np.int32), None, 1, 1)
    want, _, _ = ref.mla_positions(e, [0], 1, 1, 1, 352, 352)
    gathered = torch.from_numpy(got.astype(np.int16) if got.dtype != np.uint16 else got.view(np.int16)).view(torch.bfloat16)
    assert np.array_equal(gathered.to(torch.float64).numpy()[0], want[0])


def test_reference_masks():
    assert ref.causal(2, 3).tolist() == [[True, True, False], [True, True, True]]
    assert ref.causal(1, 6, window=2, sinks=1).tolist() == [[True, False, False, False, True, True]]
    assert ref.causal(3, 2).tolist() == [[False, False], [True, False], [True, True]]
    m = np.array([[True, False], [False, True]])
    assert ref.tree(2, 3, m).tolist() == [[True, True, False], [True, False, True]]


def test_reference_page_rules():
    """Hand-worked: lowest free pages first, grants in order, compaction's
    highest page into the lowest hole."""
    i = lambda *v: np.array(v, np.int32)      # noqa: E731
    table, lens, refs = np.full((3, 2), -1, np.int32), i(6, 0, 0), i(0, 0, 1, 0, 1)
    table[0] = [4, 2]
    cache = np.arange(5)[:, None].astype(np.uint8)
    assert ref.fork(table, lens, refs, [0, 0], [1, 1], 4, [cache]).tolist() == [1, 0]
    assert table.tolist() == [[4, 2], [4, 0], [-1, -1]] and refs.tolist() == [1, 0, 1, 0, 2] and cache[0, 0] == 2
    assert ref.extend(table, lens, refs, [2, 2], [8, 1], 4).tolist() == [1, 0]
    assert table[2].tolist() == [1, 3] and lens.tolist() == [6, 6, 8]
    ref.free(table, lens, refs, [0, 0], 4)
    assert refs.tolist() == [1, 1, 0, 1, 1] and lens.tolist() == [0, 6, 8]
    assert ref.compact(table, lens, refs, 4, [cache]).tolist() == [0, 1, -1, 3, 2]
    assert table.tolist() == [[-1, -1], [2, 0], [1, 3]] and cache[2, 0] == 4


# strides of 3 tokens and 4 heads of 64 values: rows that meet, and rows that do not
SHARED = [(64, 64), (128, 64), (64, 128), (192, 64), (72, 64), (64, 184), (128, 256), (192, 128)]
APART = [(256, 64), (64, 192), (512, 128), (80, 240), (320, 72), (1024, 64), (128, 320), (192, 256), (192, 320)]


@pytest.mark.parametrize("strides,ok", [(s, False) for s in SHARED] + [(s, True) for s in APART])
def test_rows_of_an_output_share_no_element(lib, strides, ok):
    """(token stride, head stride) pairs, each at least a row: refused when two
    rows of the output meet, whichever of the two strides is the larger."""
    import gather_concat_cache_amd as g
    T, H, hs = 3, 4, 64
    ts, st = strides
    used = np.zeros(T * ts + H * st + hs, int)
    for t in range(T):
        for h in range(H):
            used[t * ts + h * st:][:hs] += 1
    assert (used.max() == 1) == ok, "the lists above"
    L = g.nvfp4_kv_split_layout(16, 2, hs)
    a = _args(total_q=T, num_q_heads=H, q_head_stride=hs, out_token_stride=ts, out_head_stride=st)
    if ok and torch.cuda.is_available():
        return                                               # accepted: would be launched
    want = (-4, -5) if ok else (-2,)                         # refused for its shape, or for want of a GPU
    assert lib.gcache_attention_nvfp4_kv(C.byref(a), A16, C.byref(L), A16, A16, 2, hs, 0, 0, None) in want
    for heads, out in (((H, 0), (ts, st, 0, 0)), ((0, H), (0, 0, ts, st))):      # q's output, k's
        assert lib.gcache_qk_norm_rope(A16, A16, A16, A16, A16, A16, None, None, 0, 0, 0, T, *heads, hs, 0, 0, 1e-6, 256, 64,
                                       256, 64, *out, None) in want


@pytest.mark.parametrize("rows", [(1 << 31) - 1, (1 << 31) - 127, (1 << 31) - 128])
def test_rows_end_before_int32(lib, rows):
    """The kernels round rows up to tiles of 128 in 32 bits: more than 2^31 -
    128 rows (tokens x heads) are refused before anything is launched."""
    import gather_concat_cache_amd as g
    L = g.nvfp4_kv_split_layout(16, 1, 16)
    a = _args(total_q=1, num_q_heads=rows, q_head_stride=16, out_head_stride=16, lse_token_stride=rows)
    if rows > (1 << 31) - 128:
        assert lib.gcache_attention_nvfp4_kv(C.byref(a), A16, C.byref(L), A16, A16, 1, 16, 0, 0, None) == -2
        assert lib.gcache_attention_workspace_bytes(1, 1, rows, 1, 16, 1 << 20, 0, 0) == 0
    elif not torch.cuda.is_available():
        assert lib.gcache_attention_nvfp4_kv(C.byref(a), A16, C.byref(L), A16, A16, 1, 16, 0, 0, None) in (-4, -5)


def test_stream_of_another_device_is_refused():
    """The kernels run on the device of their tensors: a stream of another one
    is an error, not a launch on some other stream."""
    import types
    from gather_concat_cache_amd import _operators
    other = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError):
        _operators._elsewhere(torch.device("cuda", 0), other)
    assert _operators._elsewhere(torch.device("cuda", 1), other)
