// gcache_operators.h -- parameter blocks and launchers of the operators
// around the cache: attention over quantized pages, query/key norms with the
// position rotation, and page bookkeeping.  The extern "C" entry points in
// operators_abi.hip validate arguments, fill one of these and launch.
#pragma once

#include "gcache_internal.h"

namespace gcache {

struct AttnParams {
    const uint16_t* q;           // bf16 [total_q, hq, dk]
    uint16_t* out;               // bf16 [total_q, hq, dv]
    float* lse;                  // [total_q, hq] or nullptr
    int64_t q_ts, q_hs, o_ts, o_hs, lse_ts;   // element strides
    const uint8_t* cache;
    const int32_t* block_table;
    int64_t bt_stride;
    const int32_t* qs;           // query_starts [batch + 1]
    const int32_t* seq_lens;     // [batch]
    int32_t batch, total_q;
    int32_t hq, hk, group, hs;   // group = hq / hk
    int64_t num_blocks;
    BlockDiv div;                // block_size
    KvLayout L;                  // DS-MLA: entries are the data rows, their scales 320 bytes in
    // set by the launcher: num_blocks clamped to int32, strides that fit 32
    // bits where pages are walked 16 keys at a time
    int32_t blocks;
    uint32_t data_offset, scale_offset, data_token, scale_token;
    const float* gscale[2];      // per-head: k_scale, v_scale; nullptr otherwise
    float scale_log2;            // softmax_scale * log2(e)
    int32_t window;              // > 0: keys behind pos - window are hidden unless sinks
    int32_t sinks;
    const uint8_t* mask;         // tree mask [total_q, mask_cols] or nullptr
    int64_t mask_ts;
    int32_t mask_cols;
    int32_t tiles;               // row tiles of one kv head (upper bound)
    int32_t units;               // work units of one kv head (>= tiles)
    int32_t splits;              // key splits of a request (upper bound)
    int32_t key_tiles;           // 32-key tiles that a row tile sees (bound from max_seq_len and the window)
    float* ws_o;                 // [splits, total_q * hq, dv]
    float* ws_ml;                // [splits, total_q * hq, 2]
    int32_t* ws_chunk;           // [1] key tiles of a split, from the attention kernel to the join
    int32_t row_tile;            // rows of a row tile (set by the launcher, for the join)
    uint32_t group_mul, group_shift;     // division by group (set by the launcher): see row_token()
};

// Attention of packed prompts: the same, with keys and values in packed rows.
// hs is the value size; block_table, cache, L and gscale are unused.
struct PromptParams : AttnParams {
    const uint16_t* k;           // bf16 [total_k, hk, dk]
    const uint16_t* v;           // bf16 [total_k, hk, hs]
    int64_t k_ts, k_hs, v_ts, v_hs;      // element strides
    const int32_t* ks;           // key_starts [batch + 1]
    int32_t total_k, dk;
    int32_t causal;
    int32_t accumulate;          // join with what out and lse hold
};

// Rows per workgroup (16 to 128), work units and key splits of a call; filled
// by plan_attention from sizes that the host knows.
struct AttnPlan {
    int32_t row_tiles;           // 16-row tiles per workgroup
    int32_t tiles, units, splits, key_tiles;
    int64_t ws_floats;           // workspace of that many splits
};
AttnPlan plan_attention(int64_t total_q, int32_t batch, int32_t hq, int32_t hk, int32_t dp, int32_t dv,
                        int64_t max_seq_len, int32_t window, int32_t sinks, int64_t ws_floats_avail);
AttnPlan plan_attention_rows(int row_tiles, int64_t slots, int64_t total_q, int32_t batch, int32_t hq, int32_t hk,
                             int32_t dv, int64_t max_seq_len, int32_t window, int32_t sinks, int64_t ws_floats_avail,
                             bool even = false);
AttnPlan plan_attention_fp8(int64_t total_q, int32_t batch, int32_t hq, int32_t hk, int32_t hs, int64_t max_seq_len,
                            int32_t window, int32_t sinks, int64_t ws_floats_avail);
AttnPlan plan_attention_prompt(int64_t total_q, int32_t batch, int32_t hq, int32_t hk, int32_t dk, int32_t dv,
                               int64_t max_key_len, int32_t window, int32_t sinks, int64_t ws_floats_avail, bool even);
hipError_t launch_attention_fp8(const AttnParams& p, int row_tiles, hipStream_t s);
hipError_t launch_attention_prompt(const PromptParams& p, hipStream_t s);
hipError_t launch_attention_kv(const AttnParams& p, int row_tiles, hipStream_t s);
hipError_t launch_attention_ds_mla(const AttnParams& p, int row_tiles, hipStream_t s);

struct QkNormRopeParams {
    const uint16_t* x[2];        // q, k: bf16 [T, heads, hs]
    uint16_t* y[2];
    int64_t x_ts[2], x_hs[2], y_ts[2], y_hs[2];
    const uint16_t* w[2];        // bf16 [hs]
    int32_t heads[2];
    int32_t hs, rot, interleaved;
    const int64_t* positions;    // [T]
    const void* cos_sin;         // [max_pos, rot]: cos then sin
    int64_t cs_stride, max_pos;
    int32_t cs_bf16;
    float eps;
    int64_t num_tokens;
    int32_t waves_per_token, sets;   // set by the launcher, as is
    float inv_hs;
};
hipError_t launch_qk_norm_rope(const QkNormRopeParams& p, hipStream_t s);

struct AppendParams {
    const uint16_t *q, *k, *v;   // bf16 [T, heads, hs]
    uint16_t *qo, *ko;           // ko may be nullptr
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs, ko_ts, ko_hs;
    uint8_t* cache;
    int64_t token_stride, head_stride, side_stride, block_stride;    // bytes
    float* scales;
    int64_t s_head, s_side, s_block;
    const int32_t *qs, *lens, *block_table;
    int64_t bt_stride, num_blocks;
    const int64_t* positions;    // [T] or nullptr
    const void* cos_sin;
    int64_t max_pos, cs_stride;
    int32_t cs_bf16, interleaved, rot, hs, hq, hk, batch;
    int32_t num_tokens;
    BlockDiv div;
    // set by the launcher
    int32_t chunk_heads, head_chunks, wave_rows;     // heads of a workgroup; rows of a wave
    int32_t by_token, q_waves;
    int64_t page_groups;
};
hipError_t launch_rope_append(const AppendParams& p, hipStream_t s);

constexpr int kMaxCaches = 64;   // cache pointers carried by one launch
struct CacheList {
    uint8_t* base[kMaxCaches];
    int32_t n;
    int64_t num_blocks, block_stride, page_bytes;
};
struct PageTable {
    int32_t* table;              // [num_rows, >= stride]
    int64_t stride;
    int32_t num_rows;
    int32_t* lens;               // [num_rows]
    int32_t* refs;               // [num_blocks]
    int32_t num_blocks, block_size;
};
hipError_t launch_copy_pages(const CacheList& c, const int32_t* src, const int32_t* dst, int64_t n, hipStream_t s,
                             bool first, bool last);

// Fork and extend: requests of one call, and their workspace.
struct GrantParams {
    PageTable t;
    const int32_t* a;            // fork: parent rows; extend: rows
    const int32_t* b;            // fork: child rows; extend: new lengths
    int32_t n;
    int32_t* status;             // [n]
    int32_t* claim;              // [num_rows] lowest request number of a row
    int32_t* upto;               // [n] pages of the requests up to this one, -1: more than num_blocks
    int32_t* len;                // [n] the request's tokens, -1 when it is refused
    int32_t* free_ids;           // [num_blocks] the lowest free pages
};
hipError_t launch_fork_plan(const GrantParams& g, hipStream_t s);
hipError_t launch_fork_apply(const GrantParams& g, const CacheList& c, bool rows, hipStream_t s, bool last);
hipError_t launch_extend(const GrantParams& g, hipStream_t s);
hipError_t launch_free(const PageTable& t, const int32_t* rows, int32_t n, hipStream_t s);

constexpr int kCompactIds = 4096;   // page ids of one workgroup of the compaction plan
struct CompactParams {
    PageTable t;
    int32_t* page_map;           // [num_blocks]
    int32_t* counts;             // [ceil(num_blocks / kCompactIds)] live pages
    int32_t* holes;              // [num_blocks]
    int32_t* movers;             // [num_blocks]
    int32_t* moves;              // [1] entries of holes and movers
};
hipError_t launch_compact_plan(const CompactParams& c, hipStream_t s);
hipError_t launch_compact_move(const CompactParams& c, const CacheList& l, hipStream_t s);
hipError_t launch_compact_finish(const CompactParams& c, hipStream_t s);

// Launch `groups` workgroups of kernel(params, group0) as launch_groups does,
// as one part of a sequence of launches: only its first and last pieces of
// all take the timing hook's start and stop.
template <typename P>
inline hipError_t launch_span(void (*kernel)(P, int64_t), int64_t groups, int threads, hipStream_t s, bool first,
                              bool last, const P& p) {
    const int64_t kMaxBlocks = int64_t(1) << 22;         // 256 lanes each: below 2^32 work-items
    for (int64_t b0 = 0; b0 < groups; b0 += kMaxBlocks) {
        const int64_t nb = groups - b0 < kMaxBlocks ? groups - b0 : kMaxBlocks;
        int64_t group0 = b0;
        void* args[] = {const_cast<P*>(&p), &group0};
        const hipError_t e = launch_piece(reinterpret_cast<const void*>(kernel), nb, threads, args, s, first && b0 == 0,
                                          last && b0 + nb >= groups);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace gcache
