"""ctypes binding of the operators around the cache (include/gcache_attention.h
and include/gcache_pages.h): attention over the quantized pages, query/key
norms with the position rotation, and page ownership.

Argument marshalling only, as in _native: checks of dtype, device and layout,
then one C call on the current stream (or `stream`).  Outputs and scratch that
the caller does not pass are allocated through torch on that stream.
"""
import ctypes as C
import functools

import torch

from ._native import (_P, _I32, _I64, NvFp4KvLayout, _check, _dev_tensor, _ds_cache_geometry, _kv_geometry, _ptr, load,
                      nvfp4_kv_split_layout)

_BF16, _I32T, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


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

_INT32_MAX = 2 ** 31 - 1
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


# the current stream's handle, without building a Stream object a call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _elsewhere(dev, stream):
    """True when a call's stream or device is not the current one: the call is
    then repeated inside _on()."""
    if stream is not None and stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return stream is not None or dev.index != torch.cuda.current_device()


class _on:
    """The device of a call's tensors as the current one and, when a stream is
    given, that stream as the current one: what torch allocates inside belongs
    to the stream the kernels run on."""

    def __init__(self, device, stream):
        self.ctx = [torch.cuda.device(device)]
        if stream is not None:
            self.ctx.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.ctx:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.ctx):
            c.__exit__(*exc)


def _want(t, dtype, name, dev):
    """A GPU tensor of one dtype on one device."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != dev:
        _dev_tensor(t, dtype, name, dev)


def _vector(t, dtype, name, dev):
    _want(t, dtype, name, dev)
    if t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector")


def _scalar(t, name, dev):
    _want(t, _F32, name, dev)
    if t.numel() != 1:
        raise ValueError(f"{name} must hold one fp32 value")


def _scratch(workspace, nbytes, dev):
    """(tensor to keep until the launch, bytes) of a call's scratch memory."""
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=_U8, device=dev) if nbytes else None
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
    dev = _dev_tensor(q, _BF16, "q").device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return qk_norm_rope(q, k, q_weight, k_weight, positions, cos_sin, eps, interleaved, q_out, k_out)
    if q.dim() != 3:
        raise ValueError("q and k must be bf16 [T, heads, head_size] with unit last stride")
    T, hq, hs = q.shape
    xq, yq, q_out = _norm_side(q, q_weight, q_out, "q", T, hs, dev)
    hk, xk, yk, k_ptrs = 0, (0, 0), (0, 0), (None, None, None)
    if k is not None:
        xk, yk, k_out = _norm_side(k, k_weight, k_out, "k", T, hs, dev)
        hk, k_ptrs = k.shape[1], (k.data_ptr(), k_out.data_ptr(), k_weight.data_ptr())
    else:
        k_out = None
    rot = max_pos = cs_stride = bf16 = 0
    pos_ptr = cs_ptr = None
    if cos_sin is not None:
        bf16 = int(getattr(cos_sin, "dtype", None) is _BF16)
        _want(cos_sin, _BF16 if bf16 else _F32, "cos_sin", dev)
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [max_position, rot] with unit last stride")
        max_pos, rot = cos_sin.shape
        cs_stride, unit = cos_sin.stride()
        if (unit != 1 and rot > 1) or (max_pos > 1 and cs_stride < rot):
            raise ValueError("cos_sin must be [max_position, rot] with unit last stride and rows that do not overlap")
        _vector(positions, torch.int64, "positions", dev)
        if positions.numel() != T:
            raise ValueError("positions must hold one position per token")
        if rot:
            cs_stride, pos_ptr, cs_ptr = max(cs_stride, rot), positions.data_ptr(), cos_sin.data_ptr()
    if T and hq + hk:
        st = _load().gcache_qk_norm_rope(
            q.data_ptr(), k_ptrs[0], q_out.data_ptr(), k_ptrs[1], q_weight.data_ptr(), k_ptrs[2], pos_ptr, cs_ptr, bf16,
            max_pos, cs_stride, T, hq, hk, hs, rot, 1 if interleaved else 0, eps, xq[0], xq[1], xk[0], xk[1], yq[0], yq[1],
            yk[0], yk[1], _raw_stream(dev.index))
        if st:
            _check(st, "gcache_qk_norm_rope")
    return q_out, k_out


def _norm_side(x, w, y, name, T, hs, dev):
    """Checks of one side: (token and head strides of x, of y, y)."""
    _want(x, _BF16, name, dev)
    _vector(w, _BF16, name + "_weight", dev)
    shape = x.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != hs:
        raise ValueError("q and k must be bf16 [T, heads, head_size] with unit last stride")
    if w.numel() != hs:
        raise ValueError(f"{name}_weight must hold head_size values")
    sx = x.stride()
    if y is None:
        y = torch.empty(shape, dtype=_BF16, device=dev)
    else:
        _want(y, _BF16, name + "_out", dev)
        if y.shape != shape:
            raise ValueError(f"{name}_out must have the shape of {name}")
    sy = y.stride()
    if T and (sx[2] != 1 or sy[2] != 1):
        raise ValueError(f"{name} and {name}_out must have unit last stride")
    return sx, sy, y


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _attention(fn, extra, q, dk, dv, hk, num_blocks, block_size, block_table, query_starts, seq_lens, max_seq_len,
               softmax_scale, window, sinks, out, lse, return_lse, workspace, dev):
    """Checks the shared tensors, marshals gcache_attention_args and calls
    `fn`(args, *extra, stream)."""
    _want(q, _BF16, "q", dev)
    _want(block_table, _I32T, "block_table", dev)
    _vector(query_starts, _I32T, "query_starts", dev)
    _vector(seq_lens, _I32T, "seq_lens", dev)
    qs = q.stride()
    if len(qs) != 3 or q.shape[2] != dk or qs[2] != 1:
        raise ValueError(f"q must be bf16 [T, heads, {dk}] with unit last stride")
    if block_table.dim() != 2 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 [batch, max_blocks] tensor")
    T, hq, _ = q.shape
    B = seq_lens.numel()
    if query_starts.numel() != B + 1 or block_table.shape[0] < B:
        raise ValueError("query_starts must hold batch + 1 entries and block_table a row per request")
    if B > _INT32_MAX or hq > _INT32_MAX or block_size > _INT32_MAX:
        raise ValueError("requests, heads and block size must be within int32")
    if out is None:
        out = torch.empty((T, hq, dv), dtype=_BF16, device=dev)
    else:
        _want(out, _BF16, "out", dev)
        if out.shape != (T, hq, dv):
            raise ValueError(f"out must be bf16 {(T, hq, dv)}")
    os = out.stride()
    lse_ptr = lse_ts = 0
    if lse is None:
        if return_lse:
            lse = torch.empty((T, hq), dtype=_F32, device=dev)
    else:
        _want(lse, _F32, "lse", dev)
        if lse.shape != (T, hq):
            raise ValueError(f"lse must be fp32 {(T, hq)}")
    if lse is not None:
        lse_ts, unit = lse.stride()
        lse_ptr = lse.data_ptr()
        if (T > 1 and lse_ts < hq) or (hq > 1 and unit != 1):
            raise ValueError("lse must have unit last stride and rows that do not overlap")
        lse_ts = max(lse_ts, hq)
    if T and hq and B:
        if os[2] != 1:
            raise ValueError("out must have unit last stride")
        lib = _load()
        nbytes = 0
        if workspace is None:
            nbytes = lib.gcache_attention_workspace_bytes(T, B, hq, hk, dk, max_seq_len, window, sinks)
        workspace, nbytes = _scratch(workspace, nbytes, dev)
        a = AttentionArgs(q.data_ptr(), out.data_ptr(), lse_ptr, qs[0], qs[1], os[0], os[1], lse_ts,
                          query_starts.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(), block_table.shape[1], T,
                          max_seq_len, num_blocks, B, hq, block_size, softmax_scale, _ptr(workspace), nbytes)
        st = getattr(lib, fn)(C.byref(a), *extra, _raw_stream(dev.index))
        if st:
            _check(st, fn)
    return (out, lse) if return_lse else out


_NO_COLUMNS = 16                 # stands for a mask that no byte of is read


def _tree_mask(mask, T, dev):
    if not isinstance(mask, torch.Tensor) or mask.dtype not in (torch.bool, _U8):
        raise TypeError("tree_mask must be a bool or uint8 tensor")
    _want(mask, mask.dtype, "tree_mask", dev)
    if mask.dim() != 2 or mask.shape[0] != T:
        raise ValueError("tree_mask must be [T, columns] with unit last stride")
    cols = mask.shape[1]
    row, unit = mask.stride()
    if (cols > 1 and unit != 1) or (T > 1 and row < cols):
        raise ValueError("tree_mask must be [T, columns] with unit last stride and rows that do not overlap")
    # a mask without columns has no memory, and no pointer would mean a chain
    return mask.data_ptr() or _NO_COLUMNS, max(row, cols), min(cols, _INT32_MAX)


_split_layout = functools.lru_cache(maxsize=64)(nvfp4_kv_split_layout)     # of sizes; not handed out


def _per_head(kv_cache, q, k_scale, v_scale, layout, dev):
    _scalar(k_scale, "k_scale", dev)
    _scalar(v_scale, "v_scale", dev)
    if kv_cache.dim() != 5 or kv_cache.shape[1] != 2 or q.dim() != 3:
        raise ValueError("kv_cache must be uint8 [num_blocks, 2, block_size, num_kv_heads, full_dim], q [T, heads, hs]")
    nb, _, bs, hk, full = kv_cache.shape
    hs = q.shape[2]
    if hk == 0 or q.shape[1] % hk:
        raise ValueError("the query heads must be a multiple of the cache's heads")
    if hs % 16 or full != hs // 2 + hs // 16:
        raise ValueError("kv_cache's last dimension must be head_size/2 + head_size/16")
    if layout is None:
        if not kv_cache.is_contiguous():
            raise ValueError("the default split layout needs a contiguous kv_cache")
        return hk, hs, nb, bs, _split_layout(bs, hk, hs)
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
    only; the split follows all lengths of the batch, so a row's last bits may
    change with the other requests).  Returns out bf16 [T, Hq, hs], with lse fp32 [T, Hq] when
    return_lse.  Rows of no request keep what `out` and `lse` held
    (unspecified when they are allocated here); a row that sees nothing is
    zeros with lse -inf."""
    dev = _dev_tensor(kv_cache, _U8, "kv_cache").device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attention_nvfp4_kv(q, kv_cache, k_scale, v_scale, block_table, query_starts, seq_lens, max_seq_len,
                                      softmax_scale, window, num_sinks, layout, out, lse, return_lse, workspace)
    _want(q, _BF16, "q", dev)
    hk, hs, nb, bs, layout = _per_head(kv_cache, q, k_scale, v_scale, layout, dev)
    if window is not None and window < 1:
        raise ValueError("window must be at least 1 (None: no window)")
    # no position reaches int32's end, so larger numbers mean the same as it (ctypes would keep their low bits)
    w, sinks = (0, 0) if window is None else (min(window, _INT32_MAX), max(min(num_sinks, _INT32_MAX), -1))
    extra = (kv_cache.data_ptr(), C.byref(layout), k_scale.data_ptr(), v_scale.data_ptr(), hk, hs, w, sinks)
    return _attention("gcache_attention_nvfp4_kv", extra, q, hs, hs, hk, nb, bs, block_table, query_starts, seq_lens,
                      max_seq_len, softmax_scale, w, sinks, out, lse, return_lse, workspace, dev)


def tree_attention_nvfp4_kv(q, kv_cache, k_scale, v_scale, block_table, query_starts, seq_lens, tree_mask, max_seq_len,
                            softmax_scale, layout=None, out=None, lse=None, return_lse=False, workspace=None,
                            stream=None):
    """Attention of drafted tokens over the per-head NVFP4 cache: a request's
    queries are its last cached positions; each sees every position before the
    first of them, and query j of its own request where tree_mask (bool or
    uint8 [T, columns]) is set at column j.  Otherwise as
    attention_nvfp4_kv."""
    dev = _dev_tensor(kv_cache, _U8, "kv_cache").device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return tree_attention_nvfp4_kv(q, kv_cache, k_scale, v_scale, block_table, query_starts, seq_lens, tree_mask,
                                           max_seq_len, softmax_scale, layout, out, lse, return_lse, workspace)
    _want(q, _BF16, "q", dev)
    hk, hs, nb, bs, layout = _per_head(kv_cache, q, k_scale, v_scale, layout, dev)
    extra = (kv_cache.data_ptr(), C.byref(layout), k_scale.data_ptr(), v_scale.data_ptr(), hk, hs,
             *_tree_mask(tree_mask, q.shape[0], dev))
    return _attention("gcache_tree_attention_nvfp4_kv", extra, q, hs, hs, hk, nb, bs, block_table, query_starts,
                      seq_lens, max_seq_len, softmax_scale, 0, 0, out, lse, return_lse, workspace, dev)


def tree_attention_nvfp4_ds_mla(q, kv_cache, block_table, query_starts, seq_lens, tree_mask, max_seq_len, softmax_scale,
                                out=None, lse=None, return_lse=False, workspace=None, stream=None):
    """Attention of drafted tokens over the nvfp4_ds_mla cache uint8
    [num_blocks, block_size, >=352] in absorbed form: q bf16 [T, H, 576] (512
    latent, 64 RoPE values) -> out bf16 [T, H, 512].  tree_mask None: the
    queries are a chain (causal), the form for single tokens too.  Otherwise
    as tree_attention_nvfp4_kv."""
    dev = _dev_tensor(kv_cache, _U8, "kv_cache").device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return tree_attention_nvfp4_ds_mla(q, kv_cache, block_table, query_starts, seq_lens, tree_mask, max_seq_len,
                                               softmax_scale, out, lse, return_lse, workspace)
    _want(q, _BF16, "q", dev)
    nb, bs, bstr, estr = _ds_cache_geometry(kv_cache, "kv_cache")
    mask = (None, 0, 0) if tree_mask is None else _tree_mask(tree_mask, q.shape[0], dev)
    return _attention("gcache_tree_attention_nvfp4_ds_mla", (kv_cache.data_ptr(), bstr, estr, *mask), q, 576, 512, 1, nb,
                      bs, block_table, query_starts, seq_lens, max_seq_len, softmax_scale, 0, 0, out, lse, return_lse,
                      workspace, dev)


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def _page_caches(caches):
    """One cache or a sequence of them (one a layer), dim 0 the pages, all of
    one geometry -> (PageCaches and what it points to, num_blocks, device)."""
    caches = [caches] if isinstance(caches, torch.Tensor) else list(caches)
    if not caches:
        raise ValueError("caches must name at least one cache")
    first = caches[0]
    if not isinstance(first, torch.Tensor) or first.device.type != "cuda":
        raise ValueError("caches must be GPU tensors on one device")
    shape, strides, dtype, dev = first.shape, first.stride(), first.dtype, first.device
    if len(shape) < 2:
        raise ValueError("a cache must be [num_blocks, ...]")
    for c in caches:
        if c.shape != shape or c.stride() != strides or c.dtype is not dtype or c.device != dev:
            raise ValueError("caches must be GPU tensors on one device, of one shape, strides and dtype")
    item = first.element_size()
    page = 0 if 0 in shape[1:] else item * (1 + sum((n - 1) * s for n, s in zip(shape[1:], strides[1:])))
    stride = strides[0] * item if shape[0] > 1 else max(page, strides[0] * item)
    if page > stride:
        raise ValueError("the pages of a cache must not overlap")
    array = (C.c_void_p * len(caches))(*[c.data_ptr() for c in caches])
    return PageCaches(C.addressof(array), len(caches), stride, page), array, shape[0], dev


def _page_state(block_size, block_table, seq_lens, ref_counts, dev=None):
    dev = _dev_tensor(block_table, _I32T, "block_table", dev).device
    if block_table.dim() != 2 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 [rows, max_blocks] tensor")
    _vector(seq_lens, _I32T, "seq_lens", dev)
    _vector(ref_counts, _I32T, "ref_counts", dev)
    if seq_lens.numel() != block_table.shape[0]:
        raise ValueError("seq_lens must hold one length per row of block_table")
    if not 1 <= block_size <= _INT32_MAX or block_table.shape[0] > _INT32_MAX:
        raise ValueError("block_size must be positive, it and the rows of block_table within int32")
    return PageState(block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(), ref_counts.data_ptr(),
                     ref_counts.numel(), block_table.shape[0], block_size), dev


def _requests(names, tensors, dev):
    for name, t in zip(names, tensors):
        _vector(t, _I32T, name, dev)
    if any(t.numel() != tensors[0].numel() for t in tensors):
        raise ValueError(f"{' and '.join(names)} must be of one length")
    return tensors[0].numel()


def _status(status, n, dev):
    if status is None:
        return torch.empty(n, dtype=_I32T, device=dev)
    _vector(status, _I32T, "status", dev)
    if status.numel() != n:
        raise ValueError("status must hold one entry per request")
    return status


def copy_pages(caches, src, dst, stream=None):
    """Copy pages src[i] -> dst[i] (int32 vectors) in every cache: a tensor
    [num_blocks, ...] or a sequence of such tensors of one geometry.  A page
    goes from its first element to its last, padding between them included
    (for forks and compaction too); bytes between pages stay.  Destinations
    are distinct and none is a source."""
    pc, _keep, nb, dev = _page_caches(caches)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return copy_pages(caches, src, dst)
    n = _requests(("src", "dst"), (src, dst), dev)
    _check(_load().gcache_copy_pages(C.byref(pc), nb, src.data_ptr(), dst.data_ptr(), n, _raw_stream(dev.index)),
           "gcache_copy_pages")


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
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return fork_requests(caches, block_size, block_table, seq_lens, ref_counts, parent_rows, child_rows, status,
                                 workspace)
    n = _requests(("parent_rows", "child_rows"), (parent_rows, child_rows), dev)
    status = _status(status, n, dev)
    if n:
        lib = _load()
        ws, nbytes = _scratch(workspace, lib.gcache_pages_workspace_bytes(nb, ps.num_rows, n), dev)
        _check(lib.gcache_fork_requests(C.byref(ps), C.byref(pc), parent_rows.data_ptr(), child_rows.data_ptr(), n,
                                        status.data_ptr(), _ptr(ws), nbytes, _raw_stream(dev.index)),
               "gcache_fork_requests")
    return status


def extend_requests(block_size, block_table, seq_lens, ref_counts, rows, new_lens, status=None, workspace=None,
                    stream=None):
    """Grow rows[i] to new_lens[i] tokens, taking the lowest free pages.
    Returns status int32: 1, or 0 where the request was refused."""
    ps, dev = _page_state(block_size, block_table, seq_lens, ref_counts)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return extend_requests(block_size, block_table, seq_lens, ref_counts, rows, new_lens, status, workspace)
    n = _requests(("rows", "new_lens"), (rows, new_lens), dev)
    status = _status(status, n, dev)
    if n:
        lib = _load()
        ws, nbytes = _scratch(workspace, lib.gcache_pages_workspace_bytes(ps.num_blocks, ps.num_rows, n), dev)
        _check(lib.gcache_extend_requests(C.byref(ps), rows.data_ptr(), new_lens.data_ptr(), n, status.data_ptr(), _ptr(ws),
                                          nbytes, _raw_stream(dev.index)), "gcache_extend_requests")
    return status


def free_requests(block_size, block_table, seq_lens, ref_counts, rows, stream=None):
    """End rows[i]: their pages lose one user, the rows become empty."""
    ps, dev = _page_state(block_size, block_table, seq_lens, ref_counts)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return free_requests(block_size, block_table, seq_lens, ref_counts, rows)
    n = _requests(("rows",), (rows,), dev)
    if n:
        _check(_load().gcache_free_requests(C.byref(ps), rows.data_ptr(), n, _raw_stream(dev.index)), "gcache_free_requests")


def compact_pages(caches, block_size, block_table, seq_lens, ref_counts, page_map=None, workspace=None, stream=None):
    """Move the live pages into the lowest page ids, in every cache, and rename
    them in the tables.  Returns page_map int32 [num_blocks]: the new id of
    each page, -1 for free ones."""
    pc, _keep, nb, dev = _page_caches(caches)
    ps, dev = _page_state(block_size, block_table, seq_lens, ref_counts, dev)
    if nb != ref_counts.numel():
        raise ValueError("ref_counts must hold one count per page of the caches")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return compact_pages(caches, block_size, block_table, seq_lens, ref_counts, page_map, workspace)
    if page_map is None:
        page_map = torch.empty(nb, dtype=_I32T, device=dev)
    _vector(page_map, _I32T, "page_map", dev)
    if page_map.numel() != nb:
        raise ValueError("page_map must hold one entry per page")
    lib = _load()
    ws, nbytes = _scratch(workspace, lib.gcache_pages_workspace_bytes(nb, ps.num_rows, 0), dev)
    _check(lib.gcache_compact_pages(C.byref(ps), C.byref(pc), page_map.data_ptr(), _ptr(ws), nbytes,
                                    _raw_stream(dev.index)), "gcache_compact_pages")
    return page_map
