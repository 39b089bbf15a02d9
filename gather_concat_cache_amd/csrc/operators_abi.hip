// operators_abi.hip -- the extern "C" entry points of gcache_attention.h and
// gcache_pages.h: host checks, then one short sequence of launches on the
// caller's stream.  Nothing here allocates, frees or synchronizes.
#include <atomic>
#include <cmath>
#include <cstring>
#include <utility>

#include "../../include/gcache_attention.h"
#include "../../include/gcache_pages.h"
#include "gcache_operators.h"

using namespace gcache;

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxRequests = int64_t(1) << 22;
constexpr int64_t kMaxRows = INT32_MAX - 127;   // attention: query tokens x heads, rounded up to tiles of 128 in 32 bits
std::atomic<int> g_arch_state[kMaxDevices];   // 0 unknown, 1 gfx950, -1 other

int check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return GCACHE_ERR_DEVICE;
    if (dev >= kMaxDevices) return GCACHE_ERR_UNSUPPORTED;
    int state = g_arch_state[dev].load(std::memory_order_relaxed);
    if (state == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GCACHE_ERR_DEVICE;
        state = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
        g_arch_state[dev].store(state, std::memory_order_relaxed);
    }
    return state > 0 ? GCACHE_OK : GCACHE_ERR_UNSUPPORTED;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }
int launched(hipError_t e) { return e == hipSuccess ? GCACHE_OK : GCACHE_ERR_LAUNCH; }

BlockDiv make_div(int32_t block_size) {
    BlockDiv d{block_size, -1};
    if ((block_size & (block_size - 1)) == 0) d.shift = __builtin_ctz((unsigned)block_size);
    return d;
}

// Rows of n values at t * token_stride + h * head_stride (t < tokens, h <
// heads) share no element.  Nearly always all heads of a token, or all tokens
// of a head, end before the next begins; else two rows h heads and t tokens
// apart meet where |h * head_stride - t * token_stride| < n.
bool rows_apart(int64_t tokens, int64_t heads, int64_t token_stride, int64_t head_stride, int64_t n) {
    if (tokens < 1 || heads < 1) return true;
    if ((tokens > 1 && token_stride < n) || (heads > 1 && head_stride < n)) return false;
    if (tokens == 1 || heads == 1) return true;
    typedef __int128 wide;                               // products of two 64-bit sizes
    if ((wide)(heads - 1) * head_stride + n <= token_stride || (wide)(tokens - 1) * token_stride + n <= head_stride) return true;
    if (heads > tokens) {                                // step over the fewer
        std::swap(heads, tokens);
        std::swap(head_stride, token_stride);
    }
    for (int64_t h = 1; h < heads; h++) {
        const wide at = (wide)h * head_stride, t = at / token_stride;    // the rows around `at` are t and t + 1
        if ((t < tokens && at - t * token_stride < n) || (t + 1 < tokens && (t + 1) * token_stride - at < n)) return false;
    }
    return true;
}

// Head dims a kernel works with: 64, 128, 256, or 512 for the latent cache.
int padded_dim(int32_t head_size) { return head_size <= 64 ? 64 : head_size <= 128 ? 128 : head_size <= 256 ? 256 : 512; }

// Checks shared by the attention calls, and the parameters they fill.
int attention_args(const gcache_attention_args* a, int32_t hk, int32_t dv, AttnParams* p) {
    if (a->total_q < 0 || a->batch_size < 0) return GCACHE_ERR_SHAPE;
    if (!a->q || !a->out || !a->query_starts || !a->seq_lens || !a->block_table) return GCACHE_ERR_NULL;
    int64_t rows;
    if (a->num_q_heads <= 0 || hk <= 0 || a->num_q_heads % hk || a->block_size <= 0 ||
        a->block_table_stride <= 0 || a->num_blocks < 0 || a->max_seq_len < 0 || a->workspace_bytes < 0 ||
        !mul_ok(a->total_q, a->num_q_heads, &rows) || rows > kMaxRows)
        return GCACHE_ERR_SHAPE;
    int64_t tmp;
    if (!mul_ok(a->block_table_stride, a->block_size, &tmp) || !mul_ok(a->block_table_stride, a->batch_size, &tmp))
        return GCACHE_ERR_SHAPE;
    if (a->q_token_stride < 0 || a->q_head_stride < 0 || a->out_token_stride < 0 || a->out_head_stride < 0 ||
        a->lse_token_stride < 0)
        return GCACHE_ERR_SHAPE;
    if (!std::isfinite(a->softmax_scale)) return GCACHE_ERR_SHAPE;
    if (!aligned(a->q, 16) || !aligned(a->out, 16) || a->q_token_stride % 8 || a->q_head_stride % 8 ||
        a->out_token_stride % 8 || a->out_head_stride % 8 || !aligned(a->lse, 4) || !aligned(a->query_starts, 4) ||
        !aligned(a->seq_lens, 4) || !aligned(a->block_table, 4) || !aligned(a->workspace, 16))
        return GCACHE_ERR_ALIGN;
    // rows of an output must not share elements
    if (!rows_apart(a->total_q, a->num_q_heads, a->out_token_stride, a->out_head_stride, dv) ||
        (a->lse && a->total_q > 1 && a->lse_token_stride < a->num_q_heads))
        return GCACHE_ERR_SHAPE;
    p->q = static_cast<const uint16_t*>(a->q);
    p->out = static_cast<uint16_t*>(a->out);
    p->lse = a->lse;
    p->q_ts = a->q_token_stride;
    p->q_hs = a->q_head_stride;
    p->o_ts = a->out_token_stride;
    p->o_hs = a->out_head_stride;
    p->lse_ts = a->lse_token_stride;
    p->block_table = a->block_table;
    p->bt_stride = a->block_table_stride;
    p->qs = a->query_starts;
    p->seq_lens = a->seq_lens;
    p->batch = a->batch_size;
    p->total_q = (int32_t)a->total_q;
    p->hq = a->num_q_heads;
    p->hk = hk;
    p->group = a->num_q_heads / hk;
    p->hs = dv;
    p->num_blocks = a->num_blocks;
    p->div = make_div(a->block_size);
    p->gscale[0] = p->gscale[1] = nullptr;
    p->scale_log2 = (float)(a->softmax_scale * 1.4426950408889634);
    p->window = p->sinks = 0;
    p->mask = nullptr;
    p->mask_ts = 0;
    p->mask_cols = 0;
    p->row_tile = 0;
    return GCACHE_OK;
}

AttnPlan set_plan(const gcache_attention_args* a, int dp, AttnParams* p) {
    const int64_t have = a->workspace ? a->workspace_bytes / (int64_t)sizeof(float) : 0;
    const AttnPlan plan = plan_attention(p->total_q, p->batch, p->hq, p->hk, dp, p->hs, a->max_seq_len, p->window,
                                         p->sinks, have);
    p->tiles = plan.tiles;
    p->units = plan.units;
    p->splits = plan.splits;
    p->key_tiles = plan.key_tiles;
    p->ws_o = static_cast<float*>(a->workspace);
    const int64_t rows = (int64_t)plan.splits * p->total_q * p->hq;
    p->ws_ml = p->ws_o ? p->ws_o + rows * p->hs : nullptr;
    p->ws_chunk = p->ws_o ? reinterpret_cast<int32_t*>(p->ws_ml + 2 * rows) : nullptr;
    return plan;
}

int kv_attention(const gcache_attention_args* a, const void* kv_cache, const gcache_nvfp4_kv_layout* L,
                 const float* k_scale, const float* v_scale, int32_t hk, int32_t hs, int32_t window, int32_t sinks,
                 const uint8_t* mask, int64_t mask_ts, int32_t mask_cols, hipStream_t stream) {
    if (!a) return GCACHE_ERR_NULL;
    if ((a->total_q == 0 && a->batch_size >= 0) || (a->batch_size == 0 && a->total_q >= 0)) return GCACHE_OK;
    if ((!kv_cache && a->num_blocks > 0) || !L || !k_scale || !v_scale) return GCACHE_ERR_NULL;
    if (hs <= 0 || hs % 16 || window < 0 || sinks < 0) return GCACHE_ERR_SHAPE;
    if (hs > 256) return GCACHE_ERR_UNSUPPORTED;
    AttnParams p;
    int rc = attention_args(a, hk, hs, &p);
    if (rc) return rc;
    const int64_t v[8] = {L->data_offset, L->data_token_stride, L->data_head_stride, L->scale_offset,
                          L->scale_token_stride, L->scale_head_stride, L->side_stride, L->block_stride};
    for (int64_t x : v)
        if (x < 0) return GCACHE_ERR_SHAPE;
    int64_t tmp;
    if (!mul_ok(a->num_blocks, L->block_stride, &tmp)) return GCACHE_ERR_SHAPE;
    if (!aligned(kv_cache, 16) || L->data_offset % 8 || L->data_token_stride % 8 || L->data_head_stride % 8 ||
        L->side_stride % 8 || L->block_stride % 8)
        return GCACHE_ERR_ALIGN;
    if ((rc = check_device())) return rc;
    p.cache = static_cast<const uint8_t*>(kv_cache);
    p.L = KvLayout{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
    p.gscale[0] = k_scale;
    p.gscale[1] = v_scale;
    p.window = window;
    p.sinks = sinks;
    p.mask = mask;
    p.mask_ts = mask_ts;
    p.mask_cols = mask_cols;
    const AttnPlan plan = set_plan(a, padded_dim(hs), &p);
    return launched(launch_attention_kv(p, plan.row_tiles, stream));
}

int check_state(const gcache_page_state* s, PageTable* t) {
    if (!s) return GCACHE_ERR_NULL;
    if (!s->block_table || !s->seq_lens || !s->ref_counts) return GCACHE_ERR_NULL;
    int64_t tmp;
    if (s->num_blocks < 1 || s->num_blocks > INT32_MAX || s->num_rows < 1 || s->block_size < 1 ||
        s->block_table_stride < 1 || !mul_ok(s->num_rows, s->block_table_stride, &tmp))
        return GCACHE_ERR_SHAPE;
    if (!aligned(s->block_table, 4) || !aligned(s->seq_lens, 4) || !aligned(s->ref_counts, 4)) return GCACHE_ERR_ALIGN;
    *t = PageTable{s->block_table, s->block_table_stride, s->num_rows, s->seq_lens, s->ref_counts,
                   (int32_t)s->num_blocks, s->block_size};
    return GCACHE_OK;
}

int check_caches(const gcache_page_caches* c, int64_t num_blocks) {
    if (!c) return GCACHE_ERR_NULL;
    if (c->num_caches < 0) return GCACHE_ERR_SHAPE;
    if (c->num_caches == 0) return GCACHE_OK;
    if (!c->caches) return GCACHE_ERR_NULL;
    int64_t tmp;
    if (num_blocks < 0 || c->page_bytes < 0 || c->page_bytes > c->block_stride ||
        !mul_ok(num_blocks, c->block_stride, &tmp))
        return GCACHE_ERR_SHAPE;
    for (int i = 0; i < c->num_caches; i++)
        if (!c->caches[i]) return GCACHE_ERR_NULL;
    return GCACHE_OK;
}

// The caches from `at` on that one launch carries.
CacheList cache_list(const gcache_page_caches* c, int64_t num_blocks, int at) {
    CacheList l;
    l.n = c->num_caches - at < kMaxCaches ? c->num_caches - at : kMaxCaches;
    for (int i = 0; i < kMaxCaches; i++) l.base[i] = static_cast<uint8_t*>(i < l.n ? c->caches[at + i] : nullptr);
    l.num_blocks = num_blocks;
    l.block_stride = c->block_stride;
    l.page_bytes = c->page_bytes;
    return l;
}

int grant_params(const PageTable& t, const int32_t* a, const int32_t* b, int64_t n, int32_t* status, void* ws,
                 int64_t ws_bytes, GrantParams* g) {
    if (!a || !b || !status || !ws) return GCACHE_ERR_NULL;
    if (n > kMaxRequests || ws_bytes < gcache_pages_workspace_bytes(t.num_blocks, t.num_rows, n)) return GCACHE_ERR_SHAPE;
    if (!aligned(a, 4) || !aligned(b, 4) || !aligned(status, 4) || !aligned(ws, 4)) return GCACHE_ERR_ALIGN;
    int32_t* w = static_cast<int32_t*>(ws);
    *g = GrantParams{t, a, b, (int32_t)n, status, w, w + t.num_rows, w + t.num_rows + n, w + t.num_rows + 2 * n};
    return GCACHE_OK;
}

}  // namespace

extern "C" {

int gcache_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const void* q_weight,
                        const void* k_weight, const int64_t* positions, const void* cos_sin, int32_t cos_sin_bf16,
                        int64_t max_position, int64_t cos_sin_stride, int64_t num_tokens, int32_t num_q_heads,
                        int32_t num_kv_heads, int32_t head_size, int32_t rot, int32_t interleaved, float eps,
                        int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                        int64_t q_out_token_stride, int64_t q_out_head_stride, int64_t k_out_token_stride,
                        int64_t k_out_head_stride, hipStream_t stream) {
    if (num_tokens < 0) return GCACHE_ERR_SHAPE;
    if (num_tokens == 0) return GCACHE_OK;
    int64_t heads = (int64_t)num_q_heads + num_kv_heads, waves;
    if (num_q_heads < 0 || num_kv_heads < 0 || heads == 0 || heads > INT32_MAX / 4 || head_size < 16 || head_size % 16 ||
        rot < 0 || rot % 16 || rot > head_size || !mul_ok(num_tokens, heads, &waves) || !(eps >= 0.0f) || !std::isfinite(eps))
        return GCACHE_ERR_SHAPE;
    if (head_size > 512) return GCACHE_ERR_UNSUPPORTED;
    if ((num_q_heads && (!q || !q_out || !q_weight)) || (num_kv_heads && (!k || !k_out || !k_weight)) ||
        (rot && (!positions || !cos_sin)))
        return GCACHE_ERR_NULL;
    if (rot && (max_position < 0 || cos_sin_stride < rot)) return GCACHE_ERR_SHAPE;
    const int64_t st[8] = {q_token_stride, q_head_stride, k_token_stride, k_head_stride,
                           q_out_token_stride, q_out_head_stride, k_out_token_stride, k_out_head_stride};
    for (int i = 0; i < 8; i++) {
        if ((i / 2) % 2 ? !num_kv_heads : !num_q_heads) continue;
        if (st[i] < 0) return GCACHE_ERR_SHAPE;
        if (st[i] % 8) return GCACHE_ERR_ALIGN;
    }
    // rows of an output must not share elements
    for (int i = 0; i < 2; i++)
        if (!rows_apart(num_tokens, i ? num_kv_heads : num_q_heads, st[4 + 2 * i], st[5 + 2 * i], head_size))
            return GCACHE_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(q_weight, 16) ||
        !aligned(k_weight, 16) || !aligned(positions, 8) || !aligned(cos_sin, cos_sin_bf16 ? 2 : 4))
        return GCACHE_ERR_ALIGN;
    const int rc = check_device();
    if (rc) return rc;
    QkNormRopeParams p;
    const void* x[2] = {q, k};
    void* y[2] = {q_out, k_out};
    const void* w[2] = {q_weight, k_weight};
    for (int i = 0; i < 2; i++) {
        p.x[i] = static_cast<const uint16_t*>(x[i]);
        p.y[i] = static_cast<uint16_t*>(y[i]);
        p.w[i] = static_cast<const uint16_t*>(w[i]);
        p.x_ts[i] = st[2 * i];
        p.x_hs[i] = st[2 * i + 1];
        p.y_ts[i] = st[4 + 2 * i];
        p.y_hs[i] = st[5 + 2 * i];
    }
    p.heads[0] = num_q_heads;
    p.heads[1] = num_kv_heads;
    p.hs = head_size;
    p.rot = rot;
    p.interleaved = interleaved != 0;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.cs_stride = cos_sin_stride;
    p.max_pos = max_position;
    p.cs_bf16 = cos_sin_bf16 != 0;
    p.eps = eps;
    p.num_tokens = num_tokens;
    return launched(launch_qk_norm_rope(p, stream));
}

int64_t gcache_attention_workspace_bytes(int64_t total_q, int32_t batch_size, int32_t num_q_heads,
                                         int32_t num_kv_heads, int32_t head_size, int64_t max_seq_len, int32_t window,
                                         int32_t num_sinks) {
    if (total_q <= 0 || batch_size <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
        head_size <= 0 || max_seq_len < 0 || window < 0 || num_sinks < 0 || total_q > kMaxRows / num_q_heads)
        return 0;
    const int dp = padded_dim(head_size);
    const int32_t dv = head_size > 256 ? kNope : head_size;
    const AttnPlan p = plan_attention(total_q, batch_size, num_q_heads, num_kv_heads, dp, dv, max_seq_len, window,
                                      num_sinks, INT64_MAX);
    return p.ws_floats * (int64_t)sizeof(float);
}

int gcache_attention_nvfp4_kv(const gcache_attention_args* args, const void* kv_cache,
                              const gcache_nvfp4_kv_layout* layout, const float* k_scale, const float* v_scale,
                              int32_t num_kv_heads, int32_t head_size, int32_t window, int32_t num_sinks,
                              hipStream_t stream) {
    return kv_attention(args, kv_cache, layout, k_scale, v_scale, num_kv_heads, head_size, window, num_sinks, nullptr, 0,
                        0, stream);
}

int gcache_tree_attention_nvfp4_kv(const gcache_attention_args* args, const void* kv_cache,
                                   const gcache_nvfp4_kv_layout* layout, const float* k_scale, const float* v_scale,
                                   int32_t num_kv_heads, int32_t head_size, const uint8_t* tree_mask,
                                   int64_t tree_mask_stride, int32_t mask_columns, hipStream_t stream) {
    if (args && args->total_q > 0) {
        if (!tree_mask) return GCACHE_ERR_NULL;
        if (mask_columns < 0 || tree_mask_stride < mask_columns) return GCACHE_ERR_SHAPE;
    }
    return kv_attention(args, kv_cache, layout, k_scale, v_scale, num_kv_heads, head_size, 0, 0, tree_mask,
                        tree_mask_stride, mask_columns, stream);
}

int gcache_tree_attention_nvfp4_ds_mla(const gcache_attention_args* a, const void* kv_cache, int64_t block_stride,
                                       int64_t entry_stride, const uint8_t* tree_mask, int64_t tree_mask_stride,
                                       int32_t mask_columns, hipStream_t stream) {
    if (!a) return GCACHE_ERR_NULL;
    if ((a->total_q == 0 && a->batch_size >= 0) || (a->batch_size == 0 && a->total_q >= 0)) return GCACHE_OK;
    if (!kv_cache && a->num_blocks > 0) return GCACHE_ERR_NULL;
    if (tree_mask && (mask_columns < 0 || tree_mask_stride < mask_columns)) return GCACHE_ERR_SHAPE;
    AttnParams p;
    int rc = attention_args(a, 1, kNope, &p);
    if (rc) return rc;
    int64_t need;
    if (entry_stride < kNvEntry || !mul_ok(a->block_size, entry_stride, &need) || block_stride < need ||
        !mul_ok(a->num_blocks, block_stride, &need))
        return GCACHE_ERR_SHAPE;
    if (!aligned(kv_cache, 16) || block_stride % 16 || entry_stride % 16) return GCACHE_ERR_ALIGN;
    if ((rc = check_device())) return rc;
    p.cache = static_cast<const uint8_t*>(kv_cache);
    p.L = KvLayout{0, entry_stride, 0, kNvScaleOff, entry_stride, 0, 0, block_stride};
    p.mask = tree_mask;
    p.mask_ts = tree_mask_stride;
    p.mask_cols = tree_mask ? mask_columns : 0;
    const AttnPlan plan = set_plan(a, kNope, &p);
    return launched(launch_attention_ds_mla(p, plan.row_tiles, stream));
}

int64_t gcache_pages_workspace_bytes(int64_t num_blocks, int32_t num_rows, int64_t num_requests) {
    if (num_blocks < 0 || num_blocks > INT32_MAX || num_rows < 0 || num_requests < 0 || num_requests > kMaxRequests)
        return 0;
    const int64_t grant = num_rows + 2 * num_requests + num_blocks;
    const int64_t compact = num_blocks / kCompactIds + 1 + 2 * num_blocks + 1;
    return (grant > compact ? grant : compact) * (int64_t)sizeof(int32_t);
}

int gcache_copy_pages(const gcache_page_caches* caches, int64_t num_blocks, const int32_t* src, const int32_t* dst,
                      int64_t num_pairs, hipStream_t stream) {
    if (num_pairs < 0 || num_pairs > kMaxRequests || num_blocks < 0 || num_blocks > INT32_MAX) return GCACHE_ERR_SHAPE;
    int rc = check_caches(caches, num_blocks);
    if (rc) return rc;
    if (num_pairs == 0 || caches->num_caches == 0 || caches->page_bytes == 0 || num_blocks == 0) return GCACHE_OK;
    if (!src || !dst) return GCACHE_ERR_NULL;
    if (!aligned(src, 4) || !aligned(dst, 4)) return GCACHE_ERR_ALIGN;
    if ((rc = check_device())) return rc;
    for (int at = 0; at < caches->num_caches; at += kMaxCaches) {
        const hipError_t e = launch_copy_pages(cache_list(caches, num_blocks, at), src, dst, num_pairs, stream, at == 0,
                                               at + kMaxCaches >= caches->num_caches);
        if (e != hipSuccess) return GCACHE_ERR_LAUNCH;
    }
    return GCACHE_OK;
}

int gcache_fork_requests(const gcache_page_state* state, const gcache_page_caches* caches, const int32_t* parent_rows,
                         const int32_t* child_rows, int64_t num_forks, int32_t* status, void* workspace,
                         int64_t workspace_bytes, hipStream_t stream) {
    if (num_forks < 0) return GCACHE_ERR_SHAPE;
    PageTable t;
    int rc = check_state(state, &t);
    if (rc) return rc;
    if ((rc = check_caches(caches, t.num_blocks))) return rc;
    if (num_forks == 0) return GCACHE_OK;
    GrantParams g;
    if ((rc = grant_params(t, parent_rows, child_rows, num_forks, status, workspace, workspace_bytes, &g))) return rc;
    if ((rc = check_device())) return rc;
    hipError_t e = launch_fork_plan(g, stream);
    const int n = caches->page_bytes > 0 ? caches->num_caches : 0;
    for (int at = 0; (at < n || at == 0) && e == hipSuccess; at += kMaxCaches)
        e = launch_fork_apply(g, cache_list(caches, n ? t.num_blocks : 0, at), at == 0, stream, at + kMaxCaches >= n);
    return launched(e);
}

int gcache_extend_requests(const gcache_page_state* state, const int32_t* rows, const int32_t* new_lens,
                           int64_t num_requests, int32_t* status, void* workspace, int64_t workspace_bytes,
                           hipStream_t stream) {
    if (num_requests < 0) return GCACHE_ERR_SHAPE;
    PageTable t;
    int rc = check_state(state, &t);
    if (rc) return rc;
    if (num_requests == 0) return GCACHE_OK;
    GrantParams g;
    if ((rc = grant_params(t, rows, new_lens, num_requests, status, workspace, workspace_bytes, &g))) return rc;
    if ((rc = check_device())) return rc;
    return launched(launch_extend(g, stream));
}

int gcache_free_requests(const gcache_page_state* state, const int32_t* rows, int64_t num_requests,
                         hipStream_t stream) {
    if (num_requests < 0 || num_requests > kMaxRequests) return GCACHE_ERR_SHAPE;
    PageTable t;
    int rc = check_state(state, &t);
    if (rc) return rc;
    if (num_requests == 0) return GCACHE_OK;
    if (!rows) return GCACHE_ERR_NULL;
    if (!aligned(rows, 4)) return GCACHE_ERR_ALIGN;
    if ((rc = check_device())) return rc;
    return launched(launch_free(t, rows, (int32_t)num_requests, stream));
}

int gcache_compact_pages(const gcache_page_state* state, const gcache_page_caches* caches, int32_t* page_map,
                         void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    PageTable t;
    int rc = check_state(state, &t);
    if (rc) return rc;
    if ((rc = check_caches(caches, t.num_blocks))) return rc;
    if (!page_map || !workspace) return GCACHE_ERR_NULL;
    if (workspace_bytes < gcache_pages_workspace_bytes(t.num_blocks, t.num_rows, 0)) return GCACHE_ERR_SHAPE;
    if (!aligned(page_map, 4) || !aligned(workspace, 4)) return GCACHE_ERR_ALIGN;
    if ((rc = check_device())) return rc;
    int32_t* w = static_cast<int32_t*>(workspace);
    const int64_t groups = t.num_blocks / kCompactIds + 1;
    CompactParams c{t, page_map, w, w + groups, w + groups + t.num_blocks, w + groups + 2 * (int64_t)t.num_blocks};
    hipError_t e = launch_compact_plan(c, stream);
    const int n = caches->page_bytes > 0 ? caches->num_caches : 0;
    for (int at = 0; at < n && e == hipSuccess; at += kMaxCaches)
        e = launch_compact_move(c, cache_list(caches, t.num_blocks, at), stream);
    if (e == hipSuccess) e = launch_compact_finish(c, stream);
    return launched(e);
}

}  // extern "C"
