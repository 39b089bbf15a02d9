/*
 * gcache_fp8_kv.h -- C ABI of libgcache.so, continued: a paged cache of e4m3
 * keys and values with a scale for each page, side and head; appending to it,
 * with the position rotation on the way, and the attention that reads it.
 *
 * The conventions of gcache.h hold: device pointers owned by the caller, host
 * validation before any launch, the caller's stream, no allocation and no
 * synchronization.  Every call can be captured in a HIP graph.  Status codes
 * are gcache_status.
 *
 * The cache.  Position p of a request is in page block_table[p / block_size] at
 * token p % block_size.  The value of dim i of (page, side, token, head) is
 *     e4m3(kv_cache[page * block_stride + side * side_stride
 *                   + token * token_stride + head * head_stride + i])
 *     * kv_scales[page * scale_block_stride + side * scale_side_stride
 *                 + head * scale_head_stride],      side 0: keys, 1: values.
 * A scale counts as the nearest number within 2^-100 .. 2^121 (what is not a
 * positive number as 2^-100).
 * A page is its codes and its scales: what copies, forks or compacts pages has to
 * move both (gcache_page_sets.h, with a set for kv_cache and one for kv_scales),
 * or the scales lie within the page's bytes: kv_scales = kv_cache + the bytes of a
 * page's codes, scale_block_stride = block_stride / 4.
 */
#ifndef GCACHE_FP8_KV_H
#define GCACHE_FP8_KV_H

#include "gcache_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t token_stride, head_stride, side_stride, block_stride;   /* bytes, multiples of 16 */
    int64_t scale_head_stride, scale_side_stride, scale_block_stride;   /* floats */
} gcache_fp8_kv_layout;

/*
 * Append the new tokens of packed requests, keys rotated, and rotate their
 * queries.  Request b has the tokens query_starts[b] .. query_starts[b + 1] - 1
 * of q, k and v; they are the last of its seq_lens[b] positions.  As in
 * gcache_qk_norm_rope, without the norm:
 *     pair (a, b) = (x_i, x_{i + rot/2})     (interleaved == 0), i < rot/2
 *                or (x_{2i}, x_{2i+1})       (interleaved != 0)
 *     (a, b) -> (a cos_i - b sin_i, b cos_i + a sin_i)
 * with cos_i = cos_sin[r, i], sin_i = cos_sin[r, rot/2 + i], where r is
 * positions[token], or the token's position when positions is NULL; values
 * from rot on stay.  binary32, one rounding to bf16 (q_out, k_out) or to e4m3
 * (the cache).  A token whose r is outside [0, max_position) gets zero rows
 * of q and k.
 *
 * The scale of (page, side, head) follows from the page's tokens of this call,
 *     need = max(|x|) / 448, within 2^-100 .. 2^120:
 * a page whose first token is this call's gets need; a page with older tokens
 * keeps its scale, doubled k times, with the least k >= 0 that reaches need,
 * and its older codes are divided by 2^k (exact, but for e4m3's subnormal
 * numbers, which are rounded).  Codes are e4m3(x * (1 / scale)), rounded to
 * nearest even and clamped to +-448; inputs are finite.
 *
 *  q             bf16 [num_tokens, num_q_heads, head_size] or NULL (num_q_heads 0)
 *  k, v          bf16 [num_tokens, num_kv_heads, head_size]; token and head
 *                strides in elements, multiples of 8; all 16-byte aligned
 *  q_out, k_out  like q, k, no two rows sharing an element; may be q and k
 *                themselves (same strides), else they must not overlap the
 *                inputs; k_out may be NULL
 *  kv_cache      16-byte aligned; no two rows of a layout may share a byte
 *  kv_scales     fp32
 * A token at a negative position, behind the table's row or in a page outside
 * [0, num_blocks) is not written to the cache (its q_out and k_out are).
 * Tokens outside [query_starts[0], query_starts[batch]) are left as they were,
 * and so is every byte and scale of pages without a new token.  A page that
 * gets tokens belongs to one request (the pages operators see to that); two
 * requests of a call that append to one page race.
 * Requirements: head_size a multiple of 16, 16 .. 256 (larger:
 * GCACHE_ERR_UNSUPPORTED); rot a multiple of 16, 0 .. head_size (0: cos_sin
 * and positions are not read); num_tokens * heads <= 2^31 - 128; block_size
 * <= 65536; query_starts non-decreasing.
 */
typedef struct {
    const void *q, *k, *v;
    void *q_out, *k_out;
    int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride;
    int64_t q_out_token_stride, q_out_head_stride, k_out_token_stride, k_out_head_stride;
    const int32_t* query_starts; /* [batch_size + 1] */
    const int32_t* seq_lens;     /* [batch_size], the new tokens among them */
    const int32_t* block_table;  /* [batch_size, block_table_stride] */
    int64_t block_table_stride;
    const int64_t* positions;    /* [num_tokens] or NULL */
    const void* cos_sin;         /* fp32 or bf16 [max_position, >= rot] */
    int64_t max_position, cos_sin_stride;
    int64_t num_tokens, num_blocks;
    int32_t batch_size, num_q_heads, num_kv_heads, head_size, block_size;
    int32_t rot, interleaved, cos_sin_bf16;
} gcache_append_args;

int gcache_rope_append_fp8_kv(const gcache_append_args* args, void* kv_cache, float* kv_scales,
                              const gcache_fp8_kv_layout* layout, hipStream_t stream);

/*
 * Attention over the cache, read in place: as gcache_attention_nvfp4_kv (causal,
 * with a sliding window and sinks) or, with a tree_mask, as
 * gcache_tree_attention_nvfp4_kv (window 0 then).  An e4m3 NaN code (no write
 * makes one) that a row does not see cannot reach it; a row that sees one may
 * take it as a NaN or as 0.
 * Any value scale is right; rows that see one outside 2^-40 .. 2^24 (of pages of
 * zeros, for instance) may take up to three times as long where a request has
 * more than 32 rows a kv head.
 * Requirements: as there, head_size a multiple of 16 up to 256; the layout's
 * strides as above; fewer than 2^31 workgroups, which is certain when (batch_size
 * + 8) * num_kv_heads <= 2^30 (more: GCACHE_ERR_SHAPE).  Workspace:
 * gcache_attention_fp8_kv_workspace_bytes().
 */
int gcache_attention_fp8_kv(const gcache_attention_args* args, const void* kv_cache, const float* kv_scales,
                            const gcache_fp8_kv_layout* layout, int32_t num_kv_heads, int32_t head_size,
                            int32_t window, int32_t num_sinks, const uint8_t* tree_mask, int64_t tree_mask_stride,
                            int32_t mask_columns, hipStream_t stream);
int64_t gcache_attention_fp8_kv_workspace_bytes(int64_t total_q, int32_t batch_size, int32_t num_q_heads,
                                                int32_t num_kv_heads, int32_t head_size, int64_t max_seq_len,
                                                int32_t window, int32_t num_sinks);

#ifdef __cplusplus
}
#endif
#endif /* GCACHE_FP8_KV_H */
