/*
 * gcache_prompt.h -- C ABI of libgcache.so, continued: attention of whole
 * prompts, bf16 queries over bf16 keys and values in packed sequences of
 * different lengths; also of queries over a gathered chunk of context.
 *
 * The conventions of gcache.h hold: device pointers owned by the caller, host
 * validation before any launch, the caller's stream, no allocation and no
 * synchronization.  Every call can be captured in a HIP graph.  Status codes
 * are gcache_status.
 */
#ifndef GCACHE_PROMPT_H
#define GCACHE_PROMPT_H

#include "gcache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Request b has the query rows query_starts[b] .. query_starts[b + 1] - 1 and
 * the key rows key_starts[b] .. key_starts[b + 1] - 1.  Query head h uses
 * key/value head h / (num_q_heads / num_kv_heads).
 *   causal != 0: query i of n stands at position m - n + i of the m keys and
 *     sees key j when j <= that and (window == 0, or j < num_sinks, or position
 *     - j < window).  A query at a negative position sees nothing.
 *   causal == 0: every query sees every key of its request (window must be 0).
 *   out = sum of softmax(softmax_scale * q . k) v, binary32 sums, weights
 *   rounded to bf16 for the second product; lse the natural log of the row's
 *   sum of exp(logit).  A row that sees nothing gets zeros and lse -infinity.
 *   accumulate != 0: out and lse hold an earlier part of the row (another chunk
 *   of its keys) and get the attention over both; a part whose lse is -infinity
 *   does not count, whatever its row holds.
 * Keys and values that a row does not see cannot reach it, infinities and NaN
 * among them; a row that sees a value that is not finite gets one in its dim (the
 * infinity, or a NaN where it sees a NaN, infinities of both signs, or one whose
 * weight is 0 in binary32), and one that sees a NaN key NaNs in all.
 * Rows outside [query_starts[0], query_starts[batch]) are left as they were.
 * query_starts and key_starts must be non-decreasing (values are clamped to
 * [0, total_q] and [0, total_k]; otherwise rows belong to unspecified requests).
 *   max_key_len: the most keys of a request the caller expects; it (and total_k,
 *   which tells even lengths) only sizes the split of the keys.  The split follows the lengths of the whole batch:
 *   equal calls give equal bits, but the last bits of a row may change with the
 *   other requests.
 *   workspace: gcache_prompt_workspace_bytes() bytes, 16-byte aligned, or less,
 *   or NULL: with less the keys are split into fewer parts.  Its content is
 *   scratch; two calls that may run at the same time need two.
 * Requirements: key_size (q and k) and value_size (v and out) multiples of 8,
 * 8 .. 256 (larger: GCACHE_ERR_UNSUPPORTED); strides in elements, multiples of
 * 8; everything 16-byte aligned; token strides of k and v at most 2^23
 * (larger: GCACHE_ERR_UNSUPPORTED); no two rows of out share an element, and
 * out must not overlap the inputs; num_q_heads a multiple of num_kv_heads;
 * total_q * num_q_heads <= 2^31 - 128; total_q + total_k <= 2^31 - 256; fewer than
 * 2^31 workgroups, which is certain when (batch_size + 8) * num_kv_heads <= 2^30
 * (more: GCACHE_ERR_SHAPE).
 */
typedef struct {
    const void* q;               /* bf16 [total_q, num_q_heads, key_size] */
    const void* k;               /* bf16 [total_k, num_kv_heads, key_size] */
    const void* v;               /* bf16 [total_k, num_kv_heads, value_size] */
    void* out;                   /* bf16 [total_q, num_q_heads, value_size] */
    float* lse;                  /* [total_q, >= num_q_heads], or NULL (not with accumulate) */
    int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride;
    int64_t out_token_stride, out_head_stride, lse_token_stride;
    const int32_t* query_starts; /* [batch_size + 1] */
    const int32_t* key_starts;   /* [batch_size + 1] */
    int64_t total_q, total_k, max_key_len;
    int32_t batch_size, num_q_heads, num_kv_heads, key_size, value_size;
    float softmax_scale;
    int32_t causal, window, num_sinks, accumulate;
    void* workspace;
    int64_t workspace_bytes;
} gcache_prompt_args;

int gcache_prompt_attention(const gcache_prompt_args* args, hipStream_t stream);

/* Bytes of workspace that let a call split its keys as it wants (0 when it
 * would not split). */
int64_t gcache_prompt_workspace_bytes(int64_t total_q, int32_t batch_size, int32_t num_q_heads, int32_t num_kv_heads,
                                      int32_t key_size, int32_t value_size, int64_t max_key_len, int32_t window,
                                      int32_t num_sinks);

#ifdef __cplusplus
}
#endif
#endif /* GCACHE_PROMPT_H */
