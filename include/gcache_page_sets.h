/*
 * gcache_page_sets.h -- C ABI of libgcache.so, continued: the operators of
 * gcache_pages.h that move pages, for pages that lie in several arrays of
 * different geometry.  A page of the 8-bit cache (gcache_fp8_kv.h) is its codes
 * in kv_cache and its scales in kv_scales: a fork or a compaction that takes
 * the codes along without the scales leaves the page with other values.
 *
 * sets: HOST array of num_sets gcache_page_caches, each with a geometry
 * (block_stride, page_bytes) of its own and all with the same num_blocks pages.
 * One set is the call of gcache_pages.h.  Everything else as there.
 */
#ifndef GCACHE_PAGE_SETS_H
#define GCACHE_PAGE_SETS_H

#include "gcache_pages.h"

#ifdef __cplusplus
extern "C" {
#endif

int gcache_copy_page_sets(const gcache_page_caches* sets, int32_t num_sets, int64_t num_blocks, const int32_t* src,
                          const int32_t* dst, int64_t num_pairs, hipStream_t stream);

int gcache_fork_page_sets(const gcache_page_state* state, const gcache_page_caches* sets, int32_t num_sets,
                          const int32_t* parent_rows, const int32_t* child_rows, int64_t num_forks, int32_t* status,
                          void* workspace, int64_t workspace_bytes, hipStream_t stream);

int gcache_compact_page_sets(const gcache_page_state* state, const gcache_page_caches* sets, int32_t num_sets,
                             int32_t* page_map, void* workspace, int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* GCACHE_PAGE_SETS_H */
