"""gather_concat_cache_amd -- quantized paged KV-cache write and gather-upconvert
for AMD Instinct MI355X (gfx950), with the attention that reads the pages in
place, the norm and rotation before the write, and the ownership of pages; an
8-bit paged cache with its append and attention; and the attention of prompts.

The computation lives in libgcache.so (hand-written HIP kernels behind the C
ABI of the headers in include/); this package only marshals torch tensors (device
memory and streams) into those calls.  Each function is exported under the
C name and under the C name without the ``gcache_`` prefix.
"""
from ._native import (FP8_DS_MLA, LIB_PATH, NVFP4_DS_MLA, GcacheError, NvFp4KvLayout,
                      cache_gather_bf16, cache_gather_upconvert_fp8_ds_mla, cache_gather_upconvert_nvfp4_ds_mla,
                      cache_write_fp8_ds_mla, cache_write_nvfp4_ds_mla, context_chunks,
                      convert_req_index_to_global_index, entry_bytes,
                      gather_context_chunked,
                      gather_upconvert_nvfp4_kv, load, nvfp4_full_dim, nvfp4_kv_split_layout, nvfp4_kv_split_views,
                      reshape_and_cache_nvfp4, time_next_launch)
from ._operators import (attention_nvfp4_kv, compact_pages, copy_pages, extend_requests, fork_requests, free_requests,
                         qk_norm_rope, tree_attention_nvfp4_ds_mla, tree_attention_nvfp4_kv)
from ._serving import attention_fp8_kv, prompt_attention, rope_append_fp8_kv

__all__ = [
    "NVFP4_DS_MLA", "FP8_DS_MLA", "LIB_PATH", "GcacheError", "NvFp4KvLayout", "load",
    "entry_bytes", "nvfp4_full_dim", "nvfp4_kv_split_layout", "nvfp4_kv_split_views",
    "cache_write_nvfp4_ds_mla", "cache_write_fp8_ds_mla",
    "cache_gather_upconvert_nvfp4_ds_mla", "cache_gather_upconvert_fp8_ds_mla", "cache_gather_bf16",
    "reshape_and_cache_nvfp4", "gather_upconvert_nvfp4_kv",
    "context_chunks", "gather_context_chunked", "convert_req_index_to_global_index", "time_next_launch",
    "qk_norm_rope", "attention_nvfp4_kv", "tree_attention_nvfp4_kv", "tree_attention_nvfp4_ds_mla",
    "rope_append_fp8_kv", "attention_fp8_kv", "prompt_attention",
    "copy_pages", "fork_requests", "extend_requests", "free_requests", "compact_pages",
]

# The same functions under the C entry points' own names.
gcache_entry_bytes = entry_bytes
gcache_nvfp4_full_dim = nvfp4_full_dim
gcache_nvfp4_kv_split_layout = nvfp4_kv_split_layout
gcache_cache_write_nvfp4_ds_mla = cache_write_nvfp4_ds_mla
gcache_cache_write_fp8_ds_mla = cache_write_fp8_ds_mla
gcache_cache_gather_upconvert_nvfp4_ds_mla = cache_gather_upconvert_nvfp4_ds_mla
gcache_cache_gather_upconvert_fp8_ds_mla = cache_gather_upconvert_fp8_ds_mla
gcache_cache_gather_bf16 = cache_gather_bf16
gcache_reshape_and_cache_nvfp4 = reshape_and_cache_nvfp4
gcache_gather_upconvert_nvfp4_kv = gather_upconvert_nvfp4_kv
gcache_convert_req_index_to_global_index = convert_req_index_to_global_index
gcache_time_next_launch = time_next_launch
gcache_qk_norm_rope = qk_norm_rope
gcache_attention_nvfp4_kv = attention_nvfp4_kv
gcache_tree_attention_nvfp4_kv = tree_attention_nvfp4_kv
gcache_tree_attention_nvfp4_ds_mla = tree_attention_nvfp4_ds_mla
gcache_copy_pages = copy_pages
gcache_fork_requests = fork_requests
gcache_extend_requests = extend_requests
gcache_free_requests = free_requests
gcache_compact_pages = compact_pages
gcache_rope_append_fp8_kv = rope_append_fp8_kv
gcache_attention_fp8_kv = attention_fp8_kv
gcache_prompt_attention = prompt_attention
__all__ += [n for n in list(globals()) if n.startswith("gcache_")]

load()   # fail at import time when libgcache.so has not been built
