"""ctypes binding of the operators around the cache (include/gcache_attention.h
and include/gcache_pages.h): attention over the quantized pages, query/key
norms with the position rotation, and page ownership.

Argument marshalling only, as in _native: checks of dtype, device and layout,
then one C call on the current stream (or `stream`).  Outputs and scratch that
the caller does not pass are allocated through torch on that stream.
"""
import ctypes as C

import torch

from ._native import (_P, _I32, _I64, NvFp4KvLayout, _check, _dev_tensor, _ds_cache_geometry, _kv_geometry, _ptr,
                      _scale, _stream, load)


class AttentionArgs(C.Structure):
    """gcache_attention_args."""
    _fields_ = [("q", _P), ("out", _P), ("lse", _P),
                ("q_token_stride", _I64), ("q_head_stride", _I64), ("out_token_stride", _I64),
                ("out_head_stride", _I64), ("lse_token_stride", _I64),
                ("query_starts", _P), ("seq_lens", _P), ("block_table", _P), ("block_table_stride", _I64),
                ("total_q", _I64), ("max_seq_len", _I64), ("num_blocks", _I64),
                ("batch_size", _I32), ("num_q_heads", _I32), ("block_size", _I32), ("softmax_scale", C.c_float),
                ("workspace", _P), ("workspace_bytes", _I64)]


class PageState(C.Structure):
    """gcache_page_state."""
    _fields_ = [("block_table", _P), ("block_table_stride", _I64), ("seq_lens", _P), ("ref_counts", _P),
                ("num_blocks", _I64), ("num_rows", _I32), ("block_size", _I32)]


class PageCaches(C.Structure):
    """gcache_page_caches."""
    _fields_ = [("caches", _P), ("num_caches", _I32), ("block_stride", _I64), ("page_bytes", _I64)]


_ARGS, _LAYOUT = C.POINTER(AttentionArgs), C.POINTER(NvFp4KvLayout)
_STATE, _CACHES = C.POINTER(PageState), C.POINTER(PageCaches)
_SIGS = {
    "gcache_qk_norm_rope": (C.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _I32, _I64, _I64, _I64, _I32, _I32, _I32, _I32,
                                      _I32, C.c_float, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64, _P]),
    "gcache_attention_workspace_bytes": (_I64, [_I64, _I32, _I32, _I32, _I32, _I64, _I32, _I32]),
    "gcache_attention_nvfp4_kv": (C.c_int, [_ARGS, _P, _LAYOUT, _P, _P, _I32, _I32, _I32, _I32, _P]),
    "gcache_tree_attention_nvfp4_kv": (C.c_int, [_ARGS, _P, _LAYOUT, _P, _P, _I32, _I32, _P, _I64, _I32, _P]),
    "gcache_tree_attention_nvfp4_ds_mla": (C.c_int, [_ARGS, _P, _I64, _I64, _P, _I64, _I32, _P]),
    "gcache_pages_workspace_bytes": (_I64, [_I64, _I32, _I64]),
    "gcache_copy_pages": (C.c_int, [_CACHES, _I64, _P, _P, _I64, _P]),
    "gcache_fork_requests": (C.c_int, [_STATE, _CACHES, _P, _P, _I64, _P, _P, _I64, _P]),
    "gcache_extend_requests": (C.c_int, [_STATE, _P, _P, _I64, _P, _P, _I64, _P]),
    "gcache_free_requests": (C.c_int, [_STATE, _P, _I64, _P]),
    "gcache_compact_pages": (C.c_int, [_STATE, _CACHES, _P, _P, _I64, _P]),
}

_lib = None


def _load():
    global _lib
    if _lib is None:
        lib = load()
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


class _On:
    """The device of a call's tensors as the current one and, when a stream is
    given, that stream as the current one: what torch allocates inside belongs
    to the stream the kernels run on."""

    def __init__(self, device, stream):
        self.ctx = []
        if device.index != torch.cuda.current_device():
            self.ctx.append(torch.cuda.device(device))
        if stream is not None:
            self.ctx.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.ctx:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.ctx):
            c.__exit__(*exc)


def _vector(t, dtype, name, dev):
    _dev_tensor(t, dtype, name, dev)
    if t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector")
    return t


def _scratch(workspace, nbytes, dev):
    """(tensor to keep until the launch, bytes) of a call's scratch memory."""
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    else:
        _dev_tensor(workspace, torch.uint8, "workspace", dev)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    return workspace, 0 if workspace is None else workspace.numel()


# ---------------------------------------------------------------------------
# norms and rotation
# ---------------------------------------------------------------------------
def qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, eps=1e-6, interleaved=False, q_out=None, k_out=None,
                 stream=None):
    """Root-mean-square norm of every head of q bf16 [T, Hq, hs] and k bf16
    [T, Hk, hs] (weights bf16 [hs]), then the rotation of the first
    cos_sin.shape[1] values by the angles of positions (int64 [T]): cos_sin
    fp32 or bf16 [max_position, rot] holds cos then sin; pairs are (i, i +
    rot/2), or (2i, 2i + 1) when `interleaved`.  cos_sin None: norms only.
    k (with k_weight) may be None.  Returns (q_out, k_out), allocated when not
    given; q_out=q and k_out=k work in place."""
    dev = _dev_tensor(q, torch.bfloat16, "q").device
    T, hs = q.shape[0], q.shape[-1]
    with _On(dev, stream):
        sides = []
        for name, x, w, y in (("q", q, q_weight, q_out), ("k", k, k_weight, k_out)):
            if x is None:
                sides.append((None, None, None, 0, (0, 0, 0, 0)))
                continue
            _dev_tensor(x, torch.bfloat16, name, dev)
            if x.dim() != 3 or x.shape[0] != T or x.shape[2] != hs or (T and x.stride(2) != 1):
                raise ValueError("q and k must be bf16 [T, heads, head_size] with unit last stride")
            _vector(w, torch.bfloat16, f"{name}_weight", dev)
            if w.numel() != hs:
                raise ValueError(f"{name}_weight must hold head_size values")
            if y is None:
                y = torch.empty(x.shape, dtype=torch.bfloat16, device=dev)
            _dev_tensor(y, torch.bfloat16, f"{name}_out", dev)
            if y.shape != x.shape or (T and y.stride(2) != 1):
                raise ValueError(f"{name}_out must have the shape of {name} and unit last stride")
            sides.append((x, y, w, x.shape[1], (x.stride(0), x.stride(1), y.stride(0), y.stride(1))))
        rot = max_pos = cs_stride = 0
        if cos_sin is not None:
            if not isinstance(cos_sin, torch.Tensor) or cos_sin.dtype not in (torch.float32, torch.bfloat16):
                raise TypeError("cos_sin must be an fp32 or bf16 tensor")
            _dev_tensor(cos_sin, cos_sin.dtype, "cos_sin", dev)
            if cos_sin.dim() != 2 or (cos_sin.shape[1] > 1 and cos_sin.stride(1) != 1):
                raise ValueError("cos_sin must be [max_position, rot] with unit last stride")
            max_pos, rot = cos_sin.shape
            cs_stride = max(cos_sin.stride(0), rot)
            if max_pos > 1 and cos_sin.stride(0) < rot:
                raise ValueError("cos_sin rows must not overlap")
            _vector(positions, torch.int64, "positions", dev)
            if positions.numel() != T:
                raise ValueError("positions must hold one position per token")
        (xq, yq, wq, hq, sq), (xk, yk, wk, hk, sk) = sides
        if T == 0 or hq + hk == 0:
            return yq, yk
        st = _load().gcache_qk_norm_rope(
            _ptr(xq), _ptr(xk), _ptr(yq), _ptr(yk), _ptr(wq), _ptr(wk), _ptr(positions) if rot else None,
            _ptr(cos_sin) if rot else None, int(rot > 0 and cos_sin.dtype == torch.bfloat16), max_pos, cs_stride, T, hq,
            hk, hs, rot, int(bool(interleaved)), eps, sq[0], sq[1], sk[0], sk[1], sq[2], sq[3], sk[2], sk[3],
            _stream(dev, stream))
    _check(st, "gcache_qk_norm_rope")
    return yq, yk


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _attention(fn, extra, q, dk, dv, hk, num_blocks, block_size, block_table, query_starts, seq_lens, max_seq_len,
               softmax_scale, window, sinks, out, lse, return_lse, workspace, dev, stream):
    """Marshals gcache_attention_args and calls `fn`(args, *extra, stream)."""
    if q.dim() != 3 or q.shape[2] != dk or q.stride(2) != 1:
        raise ValueError(f"q must be bf16 [T, heads, {dk}] with unit last stride")
    if block_table.dim() != 2 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 [batch, max_blocks] tensor")
    T, hq = q.shape[0], q.shape[1]
    B = seq_lens.numel()
    if query_starts.numel() != B + 1 or block_table.shape[0] < B:
        raise ValueError("query_starts must hold batch + 1 entries and block_table a row per request")
    with _On(dev, stream):
        if out is None:
            out = torch.empty((T, hq, dv), dtype=torch.bfloat16, device=dev)
        else:
            _dev_tensor(out, torch.bfloat16, "out", dev)
            if out.shape != (T, hq, dv) or (out.numel() and out.stride(2) != 1):
                raise ValueError(f"out must be bf16 {(T, hq, dv)} with unit last stride")
        if lse is None:
            lse = torch.empty((T, hq), dtype=torch.float32, device=dev) if return_lse else None
        else:
            _dev_tensor(lse, torch.float32, "lse", dev)
            if lse.shape != (T, hq) or (lse.numel() and hq > 1 and lse.stride(1) != 1):
                raise ValueError(f"lse must be fp32 {(T, hq)} with unit last stride")
        if T and hq and B:
            lib = _load()
            nbytes = 0
            if workspace is None:
                nbytes = lib.gcache_attention_workspace_bytes(T, B, hq, hk, dk, max_seq_len, window, sinks)
            workspace, nbytes = _scratch(workspace, nbytes, dev)
            a = AttentionArgs(q.data_ptr(), out.data_ptr(), _ptr(lse), q.stride(0), q.stride(1), out.stride(0),
                              out.stride(1), 0 if lse is None else max(lse.stride(0), hq), query_starts.data_ptr(),
                              seq_lens.data_ptr(), block_table.data_ptr(), block_table.shape[1], T, max_seq_len,
                              num_blocks, B, hq, block_size, softmax_scale, _ptr(workspace), nbytes)
            _check(getattr(lib, fn)(C.byref(a), *extra, _stream(dev, stream)), fn)
    return (out, lse) if return_lse else out


def _attention_tensors(q, kv_cache, block_table, query_starts, seq_lens):
    dev = _dev_tensor(kv_cache, torch.uint8, "kv_cache").device
    _dev_tensor(q, torch.bfloat16, "q", dev)
    _dev_tensor(block_table, torch.int32, "block_table", dev)
    _vector(query_starts, torch.int32, "query_starts", dev)
    _vector(seq_lens, torch.int32, "seq_lens", dev)
    return dev


def _tree_mask(mask, T, dev):
    if not isinstance(mask, torch.Tensor) or mask.dtype not in (torch.bool, torch.uint8):
        raise TypeError("tree_mask must be a bool or uint8 tensor")
    _dev_tensor(mask, mask.dtype, "tree_mask", dev)
    if mask.dim() != 2 or mask.shape[0] != T or (mask.shape[1] > 1 and mask.stride(1) != 1) \
            or (T > 1 and mask.stride(0) < mask.shape[1]):
        raise ValueError("tree_mask must be [T, columns] with unit last stride")
    return mask.data_ptr(), max(mask.stride(0), mask.shape[1]), mask.shape[1]


def _per_head(kv_cache, q, k_scale, v_scale, layout, dev):
    _scale(k_scale, "k_scale", dev)
    _scale(v_scale, "v_scale", dev)
    if kv_cache.dim() != 5 or q.dim() != 3:
        raise ValueError("kv_cache must be uint8 [num_blocks, 2, block_size, num_kv_heads, full_dim], q [T, heads, hs]")
    hk, hs = kv_cache.shape[3], q.shape[2]
    if hk == 0 or q.shape[1] % hk:
        raise ValueError("the query heads must be a multiple of the cache's heads")
    if hs % 16 or kv_cache.shape[4] != hs // 2 + hs // 16:
        raise ValueError("kv_cache's last dimension must be head_size/2 + head_size/16")
    nb, bs, layout = _kv_geometry(kv_cache, hk, hs, layout)
    return hk, hs, nb, bs, layout


def attention_nvfp4_kv(q, kv_cache, k_scale, v_scale, block_table, query_starts, seq_lens, max_seq_len, softmax_scale,
                       window=None, num_sinks=0, layout=None, out=None, lse=None, return_lse=False, workspace=None,
                       stream=None):
    """Causal attention of packed queries bf16 [T, Hq, hs] over the per-head
    NVFP4 cache, read in place.  Request b's queries are rows query_starts[b]
    .. query_starts[b + 1] - 1 (int32 [B + 1]), the last positions of its
    seq_lens[b] (int32 [B]) cached tokens.  `window`: a query sees the last
    `window` positions up to its own and the first `num_sinks`; None: all.
    max_seq_len (int): the longest sequence expected (sizes the key split
    only).  Returns out bf16 [T, Hq, hs], with lse fp32 [T, Hq] when
    return_lse.  Rows of no request keep what `out` and `lse` held
    (unspecified when they are allocated here); a row that sees nothing is
    zeros with lse -inf."""
    dev = _attention_tensors(q, kv_cache, block_table, query_starts, seq_lens)
    hk, hs, nb, bs, layout = _per_head(kv_cache, q, k_scale, v_scale, layout, dev)
    if window is not None and window < 1:
        raise ValueError("window must be at least 1 (None: no window)")
    w, sinks = (0, 0) if window is None else (window, num_sinks)
    extra = (kv_cache.data_ptr(), C.byref(layout), k_scale.data_ptr(), v_scale.data_ptr(), hk, hs, w, sinks)
    return _attention("gcache_attention_nvfp4_kv", extra, q, hs, hs, hk, nb, bs, block_table, query_starts, seq_lens,
                      max_seq_len, softmax_scale, w, sinks, out, lse, return_lse, workspace, dev, stream)


def tree_attention_nvfp4_kv(q, kv_cache, k_scale, v_scale, block_table, query_starts, seq_lens, tree_mask, max_seq_len,
                            softmax_scale, layout=None, out=None, lse=None, return_lse=False, workspace=None,
                            stream=None):
    """Attention of drafted tokens over the per-head NVFP4 cache: a request's
    queries are its last cached positions; each sees every position before the
    first of them, and query j of its own request where tree_mask (bool or
    uint8 [T, columns]) is set at column j.  Otherwise as
    attention_nvfp4_kv."""
    dev = _attention_tensors(q, kv_cache, block_table, query_starts, seq_lens)
    hk, hs, nb, bs, layout = _per_head(kv_cache, q, k_scale, v_scale, layout, dev)
    extra = (kv_cache.data_ptr(), C.byref(layout), k_scale.data_ptr(), v_scale.data_ptr(), hk, hs,
             *_tree_mask(tree_mask, q.shape[0], dev))
    return _attention("gcache_tree_attention_nvfp4_kv", extra, q, hs, hs, hk, nb, bs, block_table, query_starts,
                      seq_lens, max_seq_len, softmax_scale, 0, 0, out, lse, return_lse, workspace, dev, stream)


def tree_attention_nvfp4_ds_mla(q, kv_cache, block_table, query_starts, seq_lens, tree_mask, max_seq_len, softmax_scale,
                                out=None, lse=None, return_lse=False, workspace=None, stream=None):
    """Attention of drafted tokens over the nvfp4_ds_mla cache uint8
    [num_blocks, block_size, >=352] in absorbed form: q bf16 [T, H, 576] (512
    latent, 64 RoPE values) -> out bf16 [T, H, 512].  tree_mask None: the
    queries are a chain (causal), the form for single tokens too.  Otherwise
    as tree_attention_nvfp4_kv."""
    dev = _attention_tensors(q, kv_cache, block_table, query_starts, seq_lens)
    nb, bs, bstr, estr = _ds_cache_geometry(kv_cache, "kv_cache")
    mask = (None, 0, 0) if tree_mask is None else _tree_mask(tree_mask, q.shape[0], dev)
    return _attention("gcache_tree_attention_nvfp4_ds_mla", (kv_cache.data_ptr(), bstr, estr, *mask), q, 576, 512, 1, nb,
                      bs, block_table, query_starts, seq_lens, max_seq_len, softmax_scale, 0, 0, out, lse, return_lse,
                      workspace, dev, stream)


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def _page_caches(caches):
    """One cache or a sequence of them (one a layer), dim 0 the pages, all of
    one geometry -> (PageCaches and what it points to, num_blocks, device)."""
    caches = [caches] if isinstance(caches, torch.Tensor) else list(caches)
    first = caches[0] if caches else None
    if first is None:
        raise ValueError("caches must name at least one cache")
    geo = None
    for c in caches:
        if not isinstance(c, torch.Tensor) or c.device.type != "cuda" or c.device != first.device:
            raise ValueError("caches must be GPU tensors on one device")
        if geo is None:
            if c.dim() < 2 or min(c.stride()) < 0:
                raise ValueError("a cache must be [num_blocks, ...]")
            geo = (c.shape, c.stride(), c.dtype)
        elif (c.shape, c.stride(), c.dtype) != geo:
            raise ValueError("caches must share one shape, one set of strides and one dtype")
    shape, strides, _ = geo
    item = first.element_size()
    page = 0 if 0 in shape[1:] else item * (1 + sum((n - 1) * s for n, s in zip(shape[1:], strides[1:])))
    stride = strides[0] * item if shape[0] > 1 else max(page, strides[0] * item)
    if page > stride:
        raise ValueError("the pages of a cache must not overlap")
    array = (C.c_void_p * len(caches))(*[c.data_ptr() for c in caches])
    return PageCaches(C.cast(array, C.c_void_p), len(caches), stride, page), array, shape[0], first.device


def _page_state(block_size, block_table, seq_lens, ref_counts, dev=None):
    dev = _dev_tensor(block_table, torch.int32, "block_table", dev).device
    if block_table.dim() != 2 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 [rows, max_blocks] tensor")
    _vector(seq_lens, torch.int32, "seq_lens", dev)
    _vector(ref_counts, torch.int32, "ref_counts", dev)
    if seq_lens.numel() != block_table.shape[0]:
        raise ValueError("seq_lens must hold one length per row of block_table")
    return PageState(block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(), ref_counts.data_ptr(),
                     ref_counts.numel(), block_table.shape[0], block_size), dev


def _requests(names, tensors, dev):
    for name, t in zip(names, tensors):
        _vector(t, torch.int32, name, dev)
    if any(t.numel() != tensors[0].numel() for t in tensors):
        raise ValueError(f"{' and '.join(names)} must be of one length")
    return tensors[0].numel()


def _status(status, n, dev):
    if status is None:
        return torch.empty(n, dtype=torch.int32, device=dev)
    _vector(status, torch.int32, "status", dev)
    if status.numel() != n:
        raise ValueError("status must hold one entry per request")
    return status


def copy_pages(caches, src, dst, stream=None):
    """Copy pages src[i] -> dst[i] (int32 vectors) in every cache: a tensor
    [num_blocks, ...] or a sequence of such tensors of one geometry.
    Destinations are distinct and none is a source."""
    pc, _keep, nb, dev = _page_caches(caches)
    n = _requests(("src", "dst"), (src, dst), dev)
    with _On(dev, stream):
        st = _load().gcache_copy_pages(C.byref(pc), nb, src.data_ptr(), dst.data_ptr(), n, _stream(dev, stream))
    _check(st, "gcache_copy_pages")


def fork_requests(caches, block_size, block_table, seq_lens, ref_counts, parent_rows, child_rows, status=None,
                  workspace=None, stream=None):
    """Make the empty rows child_rows[i] copies of rows parent_rows[i]: full
    pages are shared, the partial last page is copied to a free one in every
    cache.  State: block_table int32 [rows, max_blocks], seq_lens int32 [rows],
    ref_counts int32 [num_blocks] (0: free).  Returns status int32: 1, or 0
    where the fork was refused (gcache_pages.h says when)."""
    pc, _keep, nb, dev = _page_caches(caches)
    ps, dev = _page_state(block_size, block_table, seq_lens, ref_counts, dev)
    if nb != ref_counts.numel():
        raise ValueError("ref_counts must hold one count per page of the caches")
    n = _requests(("parent_rows", "child_rows"), (parent_rows, child_rows), dev)
    with _On(dev, stream):
        status = _status(status, n, dev)
        if n:
            lib = _load()
            ws, nbytes = _scratch(workspace, lib.gcache_pages_workspace_bytes(nb, ps.num_rows, n), dev)
            _check(lib.gcache_fork_requests(C.byref(ps), C.byref(pc), parent_rows.data_ptr(), child_rows.data_ptr(), n,
                                            status.data_ptr(), _ptr(ws), nbytes, _stream(dev, stream)),
                   "gcache_fork_requests")
    return status


def extend_requests(block_size, block_table, seq_lens, ref_counts, rows, new_lens, status=None, workspace=None,
                    stream=None):
    """Grow rows[i] to new_lens[i] tokens, taking the lowest free pages.
    Returns status int32: 1, or 0 where the request was refused."""
    ps, dev = _page_state(block_size, block_table, seq_lens, ref_counts)
    n = _requests(("rows", "new_lens"), (rows, new_lens), dev)
    with _On(dev, stream):
        status = _status(status, n, dev)
        if n:
            lib = _load()
            ws, nbytes = _scratch(workspace, lib.gcache_pages_workspace_bytes(ps.num_blocks, ps.num_rows, n), dev)
            _check(lib.gcache_extend_requests(C.byref(ps), rows.data_ptr(), new_lens.data_ptr(), n, status.data_ptr(),
                                              _ptr(ws), nbytes, _stream(dev, stream)), "gcache_extend_requests")
    return status


def free_requests(block_size, block_table, seq_lens, ref_counts, rows, stream=None):
    """End rows[i]: their pages lose one user, the rows become empty."""
    ps, dev = _page_state(block_size, block_table, seq_lens, ref_counts)
    n = _requests(("rows",), (rows,), dev)
    with _On(dev, stream):
        st = _load().gcache_free_requests(C.byref(ps), rows.data_ptr(), n, _stream(dev, stream)) if n else 0
    _check(st, "gcache_free_requests")


def compact_pages(caches, block_size, block_table, seq_lens, ref_counts, page_map=None, workspace=None, stream=None):
    """Move the live pages into the lowest page ids, in every cache, and rename
    them in the tables.  Returns page_map int32 [num_blocks]: the new id of
    each page, -1 for free ones."""
    pc, _keep, nb, dev = _page_caches(caches)
    ps, dev = _page_state(block_size, block_table, seq_lens, ref_counts, dev)
    if nb != ref_counts.numel():
        raise ValueError("ref_counts must hold one count per page of the caches")
    with _On(dev, stream):
        if page_map is None:
            page_map = torch.empty(nb, dtype=torch.int32, device=dev)
        _vector(page_map, torch.int32, "page_map", dev)
        if page_map.numel() != nb:
            raise ValueError("page_map must hold one entry per page")
        lib = _load()
        ws, nbytes = _scratch(workspace, lib.gcache_pages_workspace_bytes(nb, ps.num_rows, 0), dev)
        _check(lib.gcache_compact_pages(C.byref(ps), C.byref(pc), page_map.data_ptr(), _ptr(ws), nbytes,
                                        _stream(dev, stream)), "gcache_compact_pages")
    return page_map
