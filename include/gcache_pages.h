/*
 * gcache_pages.h -- C ABI of libgcache.so, continued: which request owns which
 * cache page, kept on the device so that a serving step never waits for the
 * host: fork, extend and free requests, compact the pages, copy pages.
 *
 * State, owned by the caller:
 *   block_table  int32 [num_rows, block_table_stride], a row a request
 *   seq_lens     int32 [num_rows]: tokens of the row; its first
 *                ceil(seq_lens / block_size) entries are its pages
 *   ref_counts   int32 [num_blocks]: users of a page (rows, or the caller's own
 *                for pages it wants kept); 0 is free
 *   caches       HOST array of num_caches device pointers (one cache a layer,
 *                any format), read during the call; all with the same
 *                num_blocks, block_stride and page_bytes (the bytes of a page
 *                that are copied, <= block_stride); pages that lie in arrays of
 *                several geometries go through gcache_page_sets.h
 * A page that a row fills only partly belongs to that row alone: a fork shares
 * the full pages and copies the partial one, so rows may append without
 * looking at counts.
 *
 * Pages are granted lowest id first, to the requests of a call in their order:
 * request i is granted when the pages of the valid requests 0..i together are
 * free, else refused (status 0) and left as it was.  Results do not depend on
 * timing.  Two calls on the same state must be ordered by the caller.
 *
 * Page ids outside [0, num_blocks) in a table are carried along and never
 * counted or copied.  The conventions of gcache.h hold otherwise; every call
 * can be captured in a HIP graph.
 *
 * Requirements: num_blocks in [1, 2^31), num_rows >= 1, block_size >= 1,
 * block_table_stride >= 1, at most 2^22 requests or pairs a call; workspace of
 * gcache_pages_workspace_bytes() bytes, 4-byte aligned (scratch).
 */
#ifndef GCACHE_PAGES_H
#define GCACHE_PAGES_H

#include "gcache.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int32_t* block_table;
    int64_t block_table_stride;
    int32_t* seq_lens;
    int32_t* ref_counts;
    int64_t num_blocks;
    int32_t num_rows, block_size;
} gcache_page_state;

typedef struct {
    void* const* caches;         /* host array */
    int32_t num_caches;
    int64_t block_stride, page_bytes;
} gcache_page_caches;

int64_t gcache_pages_workspace_bytes(int64_t num_blocks, int32_t num_rows, int64_t num_requests);

/* Pages src[i] -> dst[i] in every cache, i < num_pairs (device int32 arrays).
 * Pairs with an id outside [0, num_blocks) are skipped.  Destinations are
 * distinct and none is a source (else their bytes are unspecified). */
int gcache_copy_pages(const gcache_page_caches* caches, int64_t num_blocks, const int32_t* src,
                      const int32_t* dst, int64_t num_pairs, hipStream_t stream);

/* Row child_rows[i] becomes a copy of row parent_rows[i] (as both are before
 * the call).  Refused (status 0): a row out of range, parent == child, a child
 * that is not empty (seq_lens != 0), a child named by an earlier valid fork, a
 * parent longer than the table, no free page for the partial last page. */
int gcache_fork_requests(const gcache_page_state* state, const gcache_page_caches* caches,
                         const int32_t* parent_rows, const int32_t* child_rows, int64_t num_forks,
                         int32_t* status, void* workspace, int64_t workspace_bytes,
                         hipStream_t stream);

/* Row rows[i] grows to new_lens[i] tokens.  Refused: a row out of range or
 * named by an earlier valid request, new_lens below seq_lens or past the
 * table, not enough free pages. */
int gcache_extend_requests(const gcache_page_state* state, const int32_t* rows,
                           const int32_t* new_lens, int64_t num_requests, int32_t* status,
                           void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* Rows end: their pages lose one user (never below 0), their entries become
 * -1, seq_lens 0.  A row named twice is freed once; rows out of range are
 * skipped. */
int gcache_free_requests(const gcache_page_state* state, const int32_t* rows, int64_t num_requests,
                         hipStream_t stream);

/* With L live pages (ref_counts > 0), those with ids >= L move into the free
 * ids below L, the highest id into the lowest hole, in every cache; tables and
 * counts follow.  page_map int32 [num_blocks] gets each page's new id, -1 for
 * free pages (for the caller's own tables).  A table entry that names a free
 * page becomes -1. */
int gcache_compact_pages(const gcache_page_state* state, const gcache_page_caches* caches,
                         int32_t* page_map, void* workspace, int64_t workspace_bytes,
                         hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* GCACHE_PAGES_H */
