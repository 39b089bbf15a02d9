/*
 * gcache_attention.h -- C ABI of libgcache.so, continued: attention that reads
 * the quantized paged caches of gcache.h in place, and the norm and rotation
 * of the queries and keys before the cache write.
 *
 * The conventions of gcache.h hold: device pointers owned by the caller, host
 * validation before any launch, the caller's stream, no allocation and no
 * synchronization.  Every call can be captured in a HIP graph.  Status codes
 * are gcache_status.
 */
#ifndef GCACHE_ATTENTION_H
#define GCACHE_ATTENTION_H

#include "gcache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Norm of every query and key head with the position rotation in the same
 * pass.  For token t and head h of q (weight q_weight) and of k (k_weight):
 *     n_i = x_i * w_i / sqrt(mean(x^2) + eps)
 *     pair (a, b) = (n_i, n_{i + rot/2})     (interleaved == 0), i < rot/2
 *                or (n_{2i}, n_{2i+1})       (interleaved != 0)
 *     (a, b) -> (a cos_i - b sin_i, b cos_i + a sin_i)
 * with cos_i = cos_sin[positions[t], i] and sin_i = cos_sin[positions[t],
 * rot/2 + i]; values from rot on are only normed.  binary32 throughout, one
 * rounding to bf16.  A token whose position is outside [0, max_position) gets
 * zero rows (with rot == 0 positions and cos_sin are not read and may be NULL).
 *
 *  q, k          bf16 [num_tokens, heads, head_size], token and head strides
 *                in elements (multiples of 8), 16-byte aligned
 *  q_out, k_out  likewise, no two rows sharing an element; may be q and k
 *                themselves (same strides), else they must not overlap the
 *                inputs
 *  q_weight, k_weight  bf16 [head_size], 16-byte aligned
 *  positions     int64 [num_tokens]
 *  cos_sin       fp32 (cos_sin_bf16 == 0) or bf16 [max_position, >= rot], row
 *                stride in elements
 * Requirements: head_size a multiple of 16, 16 .. 512; rot a multiple of 16,
 * 0 .. head_size; num_q_heads, num_kv_heads >= 0 and not both 0 (the
 * pointers of a side without heads may be NULL); eps >= 0.
 */
int gcache_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out,
                        const void* q_weight, const void* k_weight, const int64_t* positions,
                        const void* cos_sin, int32_t cos_sin_bf16, int64_t max_position,
                        int64_t cos_sin_stride, int64_t num_tokens, int32_t num_q_heads,
                        int32_t num_kv_heads, int32_t head_size, int32_t rot, int32_t interleaved,
                        float eps, int64_t q_token_stride, int64_t q_head_stride,
                        int64_t k_token_stride, int64_t k_head_stride, int64_t q_out_token_stride,
                        int64_t q_out_head_stride, int64_t k_out_token_stride,
                        int64_t k_out_head_stride, hipStream_t stream);

/*
 * What an attention call works on.  Request b has the packed query tokens
 * query_starts[b] .. query_starts[b + 1] - 1 and seq_lens[b] cached tokens,
 * the queries' own among them: its query i stands at position
 * seq_lens[b] - query_len + i, and position p is in cache block
 * block_table[b, p / block_size] at offset p % block_size.
 *   Query head h uses key/value head h / (num_q_heads / num_kv_heads).
 *   Hidden from every row: positions from seq_lens[b] on, positions whose
 *   block-table index is >= block_table_stride or whose block id is outside
 *   [0, num_blocks).  A row that sees nothing (also: a query at a negative
 *   position) gets zeros and lse = -infinity.  Rows outside
 *   [query_starts[0], query_starts[batch]) are left as they were.
 *   query_starts must be non-decreasing (values are clamped to
 *   [0, total_q]; otherwise rows belong to unspecified requests).
 *   Hidden positions cannot reach an output, whatever their bytes: a block
 *   scale that holds the e4m3 NaN code (no write makes one) counts as 0.
 *   max_seq_len: the largest seq_lens the caller expects.  It only sizes the
 *   split of the keys; longer sequences are computed all the same.  The split
 *   follows the lengths of the whole batch: equal calls give equal bits, but
 *   the last bits of a row may change with the other requests.
 *   workspace: gcache_attention_workspace_bytes() bytes, 16-byte aligned, or
 *   less, or NULL: with less the keys are split into fewer parts.  Its content
 *   is scratch; two calls that may run at the same time need two.
 */
typedef struct {
    const void* q;               /* bf16 [total_q, num_q_heads, key size] */
    void* out;                   /* bf16 [total_q, num_q_heads, value size] */
    float* lse;                  /* [total_q, >= num_q_heads] natural log of the row's sum of
                                    exp(logit), or NULL */
    int64_t q_token_stride, q_head_stride;       /* elements, multiples of 8 */
    int64_t out_token_stride, out_head_stride;   /* likewise; no two rows may share an element */
    int64_t lse_token_stride;                    /* elements */
    const int32_t* query_starts; /* [batch_size + 1] */
    const int32_t* seq_lens;     /* [batch_size] */
    const int32_t* block_table;  /* [batch_size, block_table_stride] */
    int64_t block_table_stride;
    int64_t total_q;
    int64_t max_seq_len;
    int64_t num_blocks;
    int32_t batch_size, num_q_heads, block_size;
    float softmax_scale;         /* logit = softmax_scale * q . k */
    void* workspace;
    int64_t workspace_bytes;
} gcache_attention_args;

/* Bytes of workspace that let an attention call split its keys as it wants
 * (0 when it would not split).  For the DS-MLA cache: num_kv_heads = 1,
 * head_size = 576.  window and num_sinks as in the call, 0 without a window. */
int64_t gcache_attention_workspace_bytes(int64_t total_q, int32_t batch_size, int32_t num_q_heads,
                                         int32_t num_kv_heads, int32_t head_size,
                                         int64_t max_seq_len, int32_t window, int32_t num_sinks);

/*
 * Attention over the per-head NVFP4 cache with a sliding window and sinks.
 * Query at position i sees position j when j <= i and (window == 0, or
 * j < num_sinks, or i - j < window).  window == 0: plain causal attention.
 * k_scale, v_scale, layout and the alignment of the cache: as in
 * gcache_reshape_and_cache_nvfp4.
 * Requirements: head_size a multiple of 16, at most 256 (larger:
 * GCACHE_ERR_UNSUPPORTED); num_q_heads a multiple of num_kv_heads;
 * total_q * num_q_heads <= 2^31 - 128 (in every attention call); q, out 16-byte
 * aligned.
 */
int gcache_attention_nvfp4_kv(const gcache_attention_args* args, const void* kv_cache,
                              const gcache_nvfp4_kv_layout* layout, const float* k_scale,
                              const float* v_scale, int32_t num_kv_heads, int32_t head_size,
                              int32_t window, int32_t num_sinks, hipStream_t stream);

/*
 * The same cache, queries that are a tree of drafted tokens: a request's
 * queries are the last query_len positions of its sequence, in any order in
 * which the draft was written.  Query i of the request sees every position
 * before the first query, and of the queries' positions those j with
 * tree_mask[token of i, j] != 0 (its ancestors and itself, for a tree; any
 * mask is allowed).
 *  tree_mask  uint8 [total_q, mask_columns], row stride tree_mask_stride;
 *             columns from mask_columns on are hidden
 */
int gcache_tree_attention_nvfp4_kv(const gcache_attention_args* args, const void* kv_cache,
                                   const gcache_nvfp4_kv_layout* layout, const float* k_scale,
                                   const float* v_scale, int32_t num_kv_heads, int32_t head_size,
                                   const uint8_t* tree_mask, int64_t tree_mask_stride,
                                   int32_t mask_columns, hipStream_t stream);

/*
 * Tree attention over the nvfp4_ds_mla cache (gcache_cache_write_nvfp4_ds_mla's
 * 352-byte entries) in absorbed form: q is bf16 [total_q, heads, 576] (the 512
 * latent values, then 64 RoPE values), every head reads the same entries,
 *     logit = softmax_scale * (q[0:512] . nope + q[512:576] . rope)
 * and out is bf16 [total_q, heads, 512], the weighted sum of the NoPE parts.
 * tree_mask NULL: the queries are a chain (causal), which is also the form for
 * single tokens.  kv_cache, block_stride and entry_stride (bytes): as in the
 * nvfp4_ds_mla gather.
 */
int gcache_tree_attention_nvfp4_ds_mla(const gcache_attention_args* args, const void* kv_cache,
                                       int64_t block_stride, int64_t entry_stride,
                                       const uint8_t* tree_mask, int64_t tree_mask_stride,
                                       int32_t mask_columns, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* GCACHE_ATTENTION_H */
