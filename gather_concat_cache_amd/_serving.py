"""ctypes binding of the 8-bit paged cache and of the prompts' attention
(include/gcache_fp8_kv.h and include/gcache_prompt.h).

Argument marshalling only, as in _operators: checks of dtype, device and
layout, then one C call on the current stream (or `stream`).  Outputs and
scratch that the caller does not pass are allocated through torch on that
stream.
"""
import ctypes as C

import torch

from ._native import _I32, _I64, _P, _check, _dev_tensor, _ptr, load
from ._operators import (_BF16, _F32, _I32T, _INT32_MAX, _U8, _attention, _elsewhere, _on, _raw_stream, _scratch, _tree_mask,
                         _vector, _want, AttentionArgs)

_E4M3 = torch.float8_e4m3fn


class Fp8KvLayout(C.Structure):
    """gcache_fp8_kv_layout."""
    _fields_ = [(n, _I64) for n in ("token_stride", "head_stride", "side_stride", "block_stride", "scale_head_stride",
                                    "scale_side_stride", "scale_block_stride")]


class AppendArgs(C.Structure):
    """gcache_append_args."""
    _fields_ = ([(n, _P) for n in ("q", "k", "v", "q_out", "k_out")]
                + [(f"{n}_{s}_stride", _I64) for n in ("q", "k", "v", "q_out", "k_out") for s in ("token", "head")]
                + [("query_starts", _P), ("seq_lens", _P), ("block_table", _P), ("block_table_stride", _I64),
                   ("positions", _P), ("cos_sin", _P), ("max_position", _I64), ("cos_sin_stride", _I64),
                   ("num_tokens", _I64), ("num_blocks", _I64)]
                + [(n, _I32) for n in ("batch_size", "num_q_heads", "num_kv_heads", "head_size", "block_size", "rot",
                                       "interleaved", "cos_sin_bf16")])


class PromptArgs(C.Structure):
    """gcache_prompt_args."""
    _fields_ = ([(n, _P) for n in ("q", "k", "v", "out", "lse")]
                + [(f"{n}_{s}_stride", _I64) for n in ("q", "k", "v", "out") for s in ("token", "head")]
                + [("lse_token_stride", _I64), ("query_starts", _P), ("key_starts", _P), ("total_q", _I64),
                   ("total_k", _I64), ("max_key_len", _I64)]
                + [(n, _I32) for n in ("batch_size", "num_q_heads", "num_kv_heads", "key_size", "value_size")]
                + [("softmax_scale", C.c_float)]
                + [(n, _I32) for n in ("causal", "window", "num_sinks", "accumulate")]
                + [("workspace", _P), ("workspace_bytes", _I64)])


_LAYOUT = C.POINTER(Fp8KvLayout)
_SIGS = {
    "gcache_rope_append_fp8_kv": (C.c_int, [C.POINTER(AppendArgs), _P, _P, _LAYOUT, _P]),
    "gcache_attention_fp8_kv": (C.c_int, [C.POINTER(AttentionArgs), _P, _P, _LAYOUT, _I32, _I32, _I32, _I32, _P, _I64, _I32,
                                          _P]),
    "gcache_attention_fp8_kv_workspace_bytes": (_I64, [_I64, _I32, _I32, _I32, _I32, _I64, _I32, _I32]),
    "gcache_prompt_attention": (C.c_int, [C.POINTER(PromptArgs), _P]),
    "gcache_prompt_workspace_bytes": (_I64, [_I64, _I32, _I32, _I32, _I32, _I32, _I64, _I32, _I32]),
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


def _fp8_cache(kv_cache, kv_scales):
    """kv_cache e4m3 (or uint8) [num_blocks, 2, block_size, heads, head_size]
    and kv_scales fp32 [num_blocks, 2, heads], any strides -> (device, sizes,
    layout)."""
    if not isinstance(kv_cache, torch.Tensor) or kv_cache.dtype not in (_E4M3, _U8):
        raise TypeError("kv_cache must be a float8_e4m3fn or uint8 tensor")
    dev = _dev_tensor(kv_cache, kv_cache.dtype, "kv_cache").device
    _want(kv_scales, _F32, "kv_scales", dev)
    shape = kv_cache.shape
    if len(shape) != 5 or shape[1] != 2 or (kv_cache.numel() and kv_cache.stride(4) != 1):
        raise ValueError("kv_cache must be [num_blocks, 2, block_size, num_kv_heads, head_size] with unit last stride")
    nb, _, bs, hk, hs = shape
    if kv_scales.shape != (nb, 2, hk):
        raise ValueError("kv_scales must be fp32 [num_blocks, 2, num_kv_heads]")
    if bs > _INT32_MAX or hk > _INT32_MAX or hs > _INT32_MAX:
        raise ValueError("heads, head and block size must be within int32")
    # a dimension of one entry has no step
    b, side, t, h, _ = [s if n > 1 else 0 for n, s in zip(shape, kv_cache.stride())]
    sb, ss, sh = [s if n > 1 else 0 for n, s in zip(kv_scales.shape, kv_scales.stride())]
    return dev, nb, bs, hk, hs, Fp8KvLayout(t, h, side, b, sh, ss, sb)


def _head_rows(x, name, dev, T=None, heads=None, size=None):
    """bf16 [T, heads, size] with unit last stride -> token and head strides."""
    _want(x, _BF16, name, dev)
    shape = x.shape
    if len(shape) != 3 or (T is not None and shape[0] != T) or (heads is not None and shape[1] != heads) or \
            (size is not None and shape[2] != size):
        want = ["T" if T is None else T, "heads" if heads is None else heads, "head_size" if size is None else size]
        raise ValueError(f"{name} must be bf16 [{want[0]}, {want[1]}, {want[2]}] with unit last stride")
    ts, hs, unit = x.stride()
    if unit != 1 and shape[2] > 1 and x.numel():
        raise ValueError(f"{name} must have unit last stride")
    return ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0


def _starts(query_starts, name, B, dev):
    _vector(query_starts, _I32T, name, dev)
    if query_starts.numel() != B + 1:
        raise ValueError(f"{name} must hold batch + 1 entries")


def rope_append_fp8_kv(q, k, v, kv_cache, kv_scales, block_table, query_starts, seq_lens, cos_sin, positions=None,
                       interleaved=False, q_out=None, k_out=None, return_k=False, stream=None):
    """Rotate the queries and keys of new tokens and append keys and values to
    the 8-bit paged cache.  q bf16 [T, Hq, hs] (None: no queries), k and v bf16
    [T, Hk, hs] are packed: request b's tokens are rows query_starts[b] ..
    query_starts[b + 1] - 1 (int32 [B + 1]), the last of its seq_lens[b] (int32
    [B]) positions, in the pages that block_table int32 [B, max_blocks] names.
    kv_cache: float8_e4m3fn or uint8 [num_blocks, 2, block_size, Hk, hs];
    kv_scales: fp32 [num_blocks, 2, Hk], one scale for each page, side and
    head, which the call sets (gcache_fp8_kv.h says how).  cos_sin fp32 or bf16
    [max_position, rot] holds cos then sin of the rotation's angles; its row is
    the token's position, or positions[t] (int64 [T]); pairs are (i, i + rot/2),
    or (2i, 2i + 1) when `interleaved`; cos_sin None: no rotation.  Returns
    (q_out, k_out): the rotated queries, and the rotated keys when k_out is
    given or return_k is set.  q_out=q and k_out=k work in place; rows of no
    request keep what the outputs held."""
    dev, nb, bs, hk, hs, layout = _fp8_cache(kv_cache, kv_scales)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return rope_append_fp8_kv(q, k, v, kv_cache, kv_scales, block_table, query_starts, seq_lens, cos_sin, positions,
                                      interleaved, q_out, k_out, return_k)
    if hk == 0:
        raise ValueError("the cache must have heads")
    ks = _head_rows(k, "k", dev, None, hk, hs)
    T = k.shape[0]
    vs = _head_rows(v, "v", dev, T, hk, hs)
    hq, qs, qos, q_ptr, qo_ptr = 0, (0, 0), (0, 0), None, None
    if q is not None:
        qs = _head_rows(q, "q", dev, T, None, hs)
        hq = q.shape[1]
        if q_out is None:
            q_out = torch.empty((T, hq, hs), dtype=_BF16, device=dev)
        qos = _head_rows(q_out, "q_out", dev, T, hq, hs)
        q_ptr, qo_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    kos = (0, 0)
    if k_out is None and return_k:
        k_out = torch.empty((T, hk, hs), dtype=_BF16, device=dev)
    if k_out is not None:
        kos = _head_rows(k_out, "k_out", dev, T, hk, hs)
    _vector(seq_lens, _I32T, "seq_lens", dev)
    B = seq_lens.numel()
    _starts(query_starts, "query_starts", B, dev)
    _want(block_table, _I32T, "block_table", dev)
    if block_table.dim() != 2 or not block_table.is_contiguous() or block_table.shape[0] < B:
        raise ValueError("block_table must be a contiguous int32 [batch, max_blocks] tensor")
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
        if rot > hs:
            raise ValueError("cos_sin must hold at most head_size values a row")
        # an empty table has no memory, but every position is outside of it
        cs_stride, cs_ptr = max(cs_stride, rot), cos_sin.data_ptr() or kv_scales.data_ptr()
    if positions is not None:
        _vector(positions, torch.int64, "positions", dev)
        if positions.numel() != T:
            raise ValueError("positions must hold one position per token")
        pos_ptr = positions.data_ptr()
    if T > _INT32_MAX or B > _INT32_MAX or hq > _INT32_MAX:
        raise ValueError("tokens, requests and heads must be within int32")
    if T and B:
        a = AppendArgs(q_ptr if hq else None, k.data_ptr(), v.data_ptr(), qo_ptr if hq else None, _ptr(k_out), *qs, *ks, *vs,
                       *qos, *kos, query_starts.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
                       block_table.shape[1], pos_ptr, cs_ptr, max_pos, cs_stride, T, nb, B, hq, hk, hs, bs, rot,
                       1 if interleaved else 0, bf16)
        st = _load().gcache_rope_append_fp8_kv(C.byref(a), kv_cache.data_ptr(), kv_scales.data_ptr(), C.byref(layout),
                                               _raw_stream(dev.index))
        if st:
            _check(st, "gcache_rope_append_fp8_kv")
    return q_out, k_out


def attention_fp8_kv(q, kv_cache, kv_scales, block_table, query_starts, seq_lens, max_seq_len, softmax_scale, window=None,
                     num_sinks=0, tree_mask=None, out=None, lse=None, return_lse=False, workspace=None, stream=None):
    """Attention of packed queries bf16 [T, Hq, hs] over the 8-bit paged cache
    (as in rope_append_fp8_kv), read in place: causal, with `window` and
    num_sinks as in attention_nvfp4_kv, or over drafted tokens with a tree_mask
    as in tree_attention_nvfp4_kv (without a window then).  Everything else as
    in attention_nvfp4_kv: returns out bf16 [T, Hq, hs], with lse fp32 [T, Hq]
    when return_lse."""
    dev, nb, bs, hk, hs, layout = _fp8_cache(kv_cache, kv_scales)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attention_fp8_kv(q, kv_cache, kv_scales, block_table, query_starts, seq_lens, max_seq_len, softmax_scale,
                                    window, num_sinks, tree_mask, out, lse, return_lse, workspace)
    _want(q, _BF16, "q", dev)
    if q.dim() != 3 or hk == 0 or q.shape[1] % hk:
        raise ValueError("q must be bf16 [T, heads, head_size], its heads a multiple of the cache's")
    if window is not None and window < 1:
        raise ValueError("window must be at least 1 (None: no window)")
    if window is not None and tree_mask is not None:
        raise ValueError("a tree_mask goes without a window")
    # no position reaches int32's end, so larger numbers mean the same as it
    w, sinks = (0, 0) if window is None else (min(window, _INT32_MAX), max(min(num_sinks, _INT32_MAX), -1))
    mask = (None, 0, 0) if tree_mask is None else _tree_mask(tree_mask, q.shape[0], dev)
    _load()
    extra = (kv_cache.data_ptr(), kv_scales.data_ptr(), C.byref(layout), hk, hs, w, sinks, *mask)
    return _attention("gcache_attention_fp8_kv", extra, q, hs, hs, hk, nb, bs, block_table, query_starts, seq_lens,
                      max_seq_len, softmax_scale, w, sinks, out, lse, return_lse, workspace, dev,
                      "gcache_attention_fp8_kv_workspace_bytes")


def prompt_attention(q, k, v, query_starts, key_starts, max_key_len, softmax_scale, causal=True, window=None, num_sinks=0,
                     out=None, lse=None, return_lse=False, accumulate=False, workspace=None, stream=None):
    """Attention of packed prompts: queries bf16 [Tq, Hq, dk] over keys bf16
    [Tk, Hk, dk] and values bf16 [Tk, Hk, dv].  Request b's queries are rows
    query_starts[b] .. query_starts[b + 1] - 1, its keys rows key_starts[b] ..
    key_starts[b + 1] - 1 (both int32 [B + 1]).  `causal`: the queries are the
    last positions of the keys (with `window`, each sees the last `window` keys
    up to its own and the first num_sinks); otherwise every query sees every key
    of its request, as over a gathered chunk of its context.  max_key_len (int):
    the most keys expected of a request (sizes the key split only).
    `accumulate`: out and lse, both given, hold the attention over other keys
    and get that over both.  Returns out bf16 [Tq, Hq, dv], with lse fp32 [Tq,
    Hq] when return_lse.  Rows of no request keep what `out` and `lse` held
    (unspecified when they are allocated here); a row that sees nothing is
    zeros with lse -inf."""
    dev = _dev_tensor(q, _BF16, "q").device
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return prompt_attention(q, k, v, query_starts, key_starts, max_key_len, softmax_scale, causal, window, num_sinks,
                                    out, lse, return_lse, accumulate, workspace)
    qs = _head_rows(q, "q", dev)
    T, hq, dk = q.shape
    ks = _head_rows(k, "k", dev, None, None, dk)
    Tk, hk, _ = k.shape
    vs = _head_rows(v, "v", dev, Tk, hk)
    dv = v.shape[2]
    if hk == 0 or hq % hk:
        raise ValueError("the query heads must be a multiple of the key heads")
    _vector(query_starts, _I32T, "query_starts", dev)
    B = query_starts.numel() - 1
    if B < 0:
        raise ValueError("query_starts must hold batch + 1 entries")
    _starts(key_starts, "key_starts", B, dev)
    if window is not None and (window < 1 or not causal):
        raise ValueError("window must be at least 1 (None: no window), and needs the causal order")
    w, sinks = (0, 0) if window is None else (min(window, _INT32_MAX), max(min(num_sinks, _INT32_MAX), -1))
    if accumulate and (out is None or lse is None):
        raise ValueError("accumulate needs the out and lse of the other keys")
    if out is None:
        out = torch.empty((T, hq, dv), dtype=_BF16, device=dev)
    os = _head_rows(out, "out", dev, T, hq, dv)
    if lse is None and return_lse:
        lse = torch.empty((T, hq), dtype=_F32, device=dev)
    lse_ts = 0
    if lse is not None:
        _want(lse, _F32, "lse", dev)
        if lse.shape != (T, hq):
            raise ValueError(f"lse must be fp32 {(T, hq)}")
        lse_ts, unit = lse.stride()
        if (T > 1 and lse_ts < hq) or (hq > 1 and unit != 1):
            raise ValueError("lse must have unit last stride and rows that do not overlap")
        lse_ts = max(lse_ts, hq)
    if max(T, Tk, B, hq, dk, dv) > _INT32_MAX:
        raise ValueError("tokens, requests, heads and head sizes must be within int32")
    if T and hq and B:
        lib = _load()
        nbytes = 0
        if workspace is None:
            nbytes = lib.gcache_prompt_workspace_bytes(T, B, hq, hk, dk, dv, max_key_len, w, max(sinks, 0))
        workspace, nbytes = _scratch(workspace, nbytes, dev)
        a = PromptArgs(q.data_ptr(), k.data_ptr() or None, v.data_ptr() or None, out.data_ptr(), _ptr(lse), *qs, *ks, *vs, *os,
                       lse_ts, query_starts.data_ptr(), key_starts.data_ptr(), T, Tk, max_key_len, B, hq, hk, dk, dv,
                       softmax_scale, 1 if causal else 0, w, sinks, 1 if accumulate else 0, _ptr(workspace), nbytes)
        st = lib.gcache_prompt_attention(C.byref(a), _raw_stream(dev.index))
        if st:
            _check(st, "gcache_prompt_attention")
    return (out, lse) if return_lse else out
