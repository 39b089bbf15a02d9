// operators_abi.hip -- the extern "C" entry points of gcache_attention.h,
// gcache_fp8_kv.h, gcache_prompt.h, gcache_pages.h and gcache_page_sets.h: host
// checks, then one short sequence of launches on the caller's stream.  Nothing here allocates,
// frees or synchronizes.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <utility>

#include "../../include/gcache_attention.h"
#include "../../include/gcache_fp8_kv.h"
#include "../../include/gcache_page_sets.h"
#include "../../include/gcache_pages.h"
#include "../../include/gcache_prompt.h"
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

// The plan's sizes and the workspace's parts.
void use_plan(const AttnPlan& plan, void* workspace, AttnParams* p) {
    p->tiles = plan.tiles;
    p->units = plan.units;
    p->splits = plan.splits;
    p->key_tiles = plan.key_tiles;
    p->ws_o = static_cast<float*>(workspace);
    const int64_t rows = (int64_t)plan.splits * p->total_q * p->hq;
    p->ws_ml = p->ws_o ? p->ws_o + rows * p->hs : nullptr;
    p->ws_chunk = p->ws_o ? reinterpret_cast<int32_t*>(p->ws_ml + 2 * rows) : nullptr;
}

int64_t workspace_floats(const void* workspace, int64_t bytes) { return workspace ? bytes / (int64_t)sizeof(float) : 0; }

AttnPlan set_plan(const gcache_attention_args* a, int dp, AttnParams* p) {
    const AttnPlan plan = plan_attention(p->total_q, p->batch, p->hq, p->hk, dp, p->hs, a->max_seq_len, p->window,
                                         p->sinks, workspace_floats(a->workspace, a->workspace_bytes));
    use_plan(plan, a->workspace, p);
    return plan;
}

// Rows of n elements, repeated `count` times `stride` apart in each of several
// dimensions, share no element: in the order of their strides, each dimension's
// steps are as long as what lies inside it.
struct Dim {
    int64_t count, stride;
};
bool nested(Dim* d, int dims, int64_t n) {
    std::sort(d, d + dims, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    for (int i = 0; i < dims; i++) {
        if (d[i].count <= 1) continue;
        if (d[i].stride < n) return false;
        int64_t span;
        if (!mul_ok(d[i].count - 1, d[i].stride, &span) || __builtin_add_overflow(span, n, &n)) return false;
    }
    return true;
}

int check_fp8_layout(const gcache_fp8_kv_layout* L, const void* cache, const float* scales, int64_t num_blocks, bool written,
                     int32_t hk, int32_t hs, int32_t block_size) {
    const int64_t s[7] = {L->token_stride, L->head_stride, L->side_stride, L->block_stride,
                          L->scale_head_stride, L->scale_side_stride, L->scale_block_stride};
    int64_t tmp;
    for (int64_t x : s)
        if (x < 0 || !mul_ok(x, 2, &tmp)) return GCACHE_ERR_SHAPE;
    if (!mul_ok(num_blocks, L->block_stride, &tmp) || !mul_ok(num_blocks, L->scale_block_stride, &tmp) ||
        !mul_ok(hk, L->head_stride, &tmp) || !mul_ok(hk, L->scale_head_stride, &tmp) ||
        !mul_ok(block_size, L->token_stride, &tmp))
        return GCACHE_ERR_SHAPE;
    if (!aligned(cache, 16) || !aligned(scales, 4)) return GCACHE_ERR_ALIGN;
    for (int i = 0; i < 4; i++)
        if (s[i] % 16) return GCACHE_ERR_ALIGN;
    Dim data[4] = {{block_size, s[0]}, {hk, s[1]}, {2, s[2]}, {num_blocks, s[3]}};
    Dim scale[3] = {{hk, s[4]}, {2, s[5]}, {num_blocks, s[6]}};
    if (written && (!nested(data, 4, hs) || !nested(scale, 3, 1))) return GCACHE_ERR_SHAPE;
    return GCACHE_OK;
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

int check_sets(const gcache_page_caches* sets, int32_t num_sets, int64_t num_blocks) {
    if (num_sets < 0) return GCACHE_ERR_SHAPE;
    if (num_sets > 0 && !sets) return GCACHE_ERR_NULL;
    for (int i = 0; i < num_sets; i++)
        if (const int rc = check_caches(sets + i, num_blocks)) return rc;
    return GCACHE_OK;
}
// Caches of a set that have bytes to move.
int moved_caches(const gcache_page_caches& c) { return c.page_bytes > 0 ? c.num_caches : 0; }

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

// run(list, first, last) for each launch's caches, of all sets.
template <typename Run>
void each_list(const gcache_page_caches* sets, int32_t num_sets, int64_t num_blocks, Run run) {
    int64_t left = 0, done = 0;
    for (int i = 0; i < num_sets; i++) left += moved_caches(sets[i]);
    for (int i = 0; i < num_sets; i++) {
        const int n = moved_caches(sets[i]);
        for (int at = 0; at < n; at += kMaxCaches) {
            const CacheList l = cache_list(sets + i, num_blocks, at);
            run(l, done == 0, done + l.n == left);
            done += l.n;
        }
    }
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

int gcache_rope_append_fp8_kv(const gcache_append_args* a, void* kv_cache, float* kv_scales,
                              const gcache_fp8_kv_layout* L, hipStream_t stream) {
    if (!a) return GCACHE_ERR_NULL;
    if (a->num_tokens < 0 || a->batch_size < 0) return GCACHE_ERR_SHAPE;
    if (a->num_tokens == 0 || a->batch_size == 0) return GCACHE_OK;
    if (!L || !a->k || !a->v || (a->num_q_heads > 0 && (!a->q || !a->q_out)) || !a->query_starts || !a->seq_lens ||
        !a->block_table || (a->num_blocks > 0 && (!kv_cache || !kv_scales)) || (a->rot > 0 && !a->cos_sin))
        return GCACHE_ERR_NULL;
    int64_t tmp;
    const int64_t heads = (int64_t)a->num_q_heads + a->num_kv_heads;
    if (a->num_q_heads < 0 || a->num_kv_heads <= 0 || a->head_size < 16 || a->head_size % 16 || a->rot < 0 || a->rot % 16 ||
        a->rot > a->head_size || a->block_size <= 0 || a->block_size > 65536 || a->block_table_stride <= 0 ||
        a->num_blocks < 0 || !mul_ok(a->num_tokens, heads, &tmp) || tmp > kMaxRows ||
        !mul_ok(a->block_table_stride, a->batch_size, &tmp) || !mul_ok(a->block_table_stride, a->block_size, &tmp) ||
        (a->rot > 0 && (a->max_position < 0 || a->cos_sin_stride < a->rot)))
        return GCACHE_ERR_SHAPE;
    if (a->head_size > 256) return GCACHE_ERR_UNSUPPORTED;
    const bool sides[5] = {a->num_q_heads > 0, true, true, a->num_q_heads > 0, a->k_out != nullptr};   // q, k, v, q_out, k_out
    const int64_t st[10] = {a->q_token_stride, a->q_head_stride, a->k_token_stride, a->k_head_stride, a->v_token_stride,
                            a->v_head_stride, a->q_out_token_stride, a->q_out_head_stride, a->k_out_token_stride,
                            a->k_out_head_stride};
    const void* at[5] = {a->q, a->k, a->v, a->q_out, a->k_out};
    for (int i = 0; i < 10; i++) {
        if (!sides[i / 2]) continue;
        if (st[i] < 0) return GCACHE_ERR_SHAPE;
        if (st[i] % 8 || !aligned(at[i / 2], 16)) return GCACHE_ERR_ALIGN;
    }
    for (int i = 3; i < 5; i++)                          // rows of an output must not share elements
        if (sides[i] && !rows_apart(a->num_tokens, i == 3 ? a->num_q_heads : a->num_kv_heads, st[2 * i], st[2 * i + 1], a->head_size))
            return GCACHE_ERR_SHAPE;
    if (!aligned(a->query_starts, 4) || !aligned(a->seq_lens, 4) || !aligned(a->block_table, 4) ||
        (a->rot > 0 && (!aligned(a->positions, 8) || !aligned(a->cos_sin, a->cos_sin_bf16 ? 2 : 4))))
        return GCACHE_ERR_ALIGN;
    int rc = check_fp8_layout(L, kv_cache, kv_scales, a->num_blocks, true, a->num_kv_heads, a->head_size, a->block_size);
    if (rc) return rc;
    if ((rc = check_device())) return rc;
    AppendParams p;
    p.q = static_cast<const uint16_t*>(a->q);
    p.k = static_cast<const uint16_t*>(a->k);
    p.v = static_cast<const uint16_t*>(a->v);
    p.qo = static_cast<uint16_t*>(a->q_out);
    p.ko = static_cast<uint16_t*>(a->k_out);
    p.q_ts = st[0];
    p.q_hs = st[1];
    p.k_ts = st[2];
    p.k_hs = st[3];
    p.v_ts = st[4];
    p.v_hs = st[5];
    p.qo_ts = st[6];
    p.qo_hs = st[7];
    p.ko_ts = st[8];
    p.ko_hs = st[9];
    p.cache = static_cast<uint8_t*>(kv_cache);
    p.token_stride = L->token_stride;
    p.head_stride = L->head_stride;
    p.side_stride = L->side_stride;
    p.block_stride = L->block_stride;
    p.scales = kv_scales;
    p.s_head = L->scale_head_stride;
    p.s_side = L->scale_side_stride;
    p.s_block = L->scale_block_stride;
    p.qs = a->query_starts;
    p.lens = a->seq_lens;
    p.block_table = a->block_table;
    p.bt_stride = a->block_table_stride;
    p.num_blocks = a->num_blocks;
    p.positions = a->rot > 0 ? a->positions : nullptr;   // (without a rotation neither is read)
    p.cos_sin = a->rot > 0 ? a->cos_sin : nullptr;
    p.max_pos = a->max_position;
    p.cs_stride = a->cos_sin_stride;
    p.cs_bf16 = a->cos_sin_bf16 != 0;
    p.interleaved = a->interleaved != 0;
    p.rot = a->rot;
    p.hs = a->head_size;
    p.hq = a->num_q_heads;
    p.hk = a->num_kv_heads;
    p.batch = a->batch_size;
    p.num_tokens = (int32_t)a->num_tokens;
    p.div = make_div(a->block_size);
    return launched(launch_rope_append(p, stream));
}

int gcache_attention_fp8_kv(const gcache_attention_args* a, const void* kv_cache, const float* kv_scales,
                            const gcache_fp8_kv_layout* L, int32_t hk, int32_t hs, int32_t window, int32_t num_sinks,
                            const uint8_t* tree_mask, int64_t tree_mask_stride, int32_t mask_columns, hipStream_t stream) {
    if (!a) return GCACHE_ERR_NULL;
    if ((a->total_q == 0 && a->batch_size >= 0) || (a->batch_size == 0 && a->total_q >= 0)) return GCACHE_OK;
    if (!L || (a->num_blocks > 0 && (!kv_cache || !kv_scales))) return GCACHE_ERR_NULL;
    if (hs <= 0 || hs % 16 || window < 0 || num_sinks < 0 ||
        (tree_mask && (window > 0 || mask_columns < 0 || tree_mask_stride < mask_columns)))
        return GCACHE_ERR_SHAPE;
    if (hs > 256) return GCACHE_ERR_UNSUPPORTED;
    AttnParams p;
    int rc = attention_args(a, hk, hs, &p);
    if (rc) return rc;
    if ((rc = check_fp8_layout(L, kv_cache, kv_scales, a->num_blocks, false, hk, hs, a->block_size))) return rc;
    if ((rc = check_device())) return rc;
    p.cache = static_cast<const uint8_t*>(kv_cache);
    // the scales' strides in floats: see raw_scale()
    p.L = KvLayout{0, L->token_stride, L->head_stride, L->scale_side_stride, L->scale_block_stride, L->scale_head_stride,
                   L->side_stride, L->block_stride};
    p.gscale[0] = kv_scales;
    p.window = window;
    p.sinks = num_sinks;
    p.mask = tree_mask;
    p.mask_ts = tree_mask_stride;
    p.mask_cols = tree_mask ? mask_columns : 0;
    const AttnPlan plan = plan_attention_fp8(p.total_q, p.batch, p.hq, hk, hs, a->max_seq_len, window, num_sinks,
                                             workspace_floats(a->workspace, a->workspace_bytes));
    use_plan(plan, a->workspace, &p);
    if (((int64_t)p.units + 7) * hk > INT32_MAX) return GCACHE_ERR_SHAPE;    // workgroups are numbered in 32 bits
    return launched(launch_attention_fp8(p, plan.row_tiles, stream));
}

int64_t gcache_attention_fp8_kv_workspace_bytes(int64_t total_q, int32_t batch_size, int32_t num_q_heads,
                                                int32_t num_kv_heads, int32_t head_size, int64_t max_seq_len,
                                                int32_t window, int32_t num_sinks) {
    if (total_q <= 0 || batch_size <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
        head_size <= 0 || max_seq_len < 0 || window < 0 || num_sinks < 0 || total_q > kMaxRows / num_q_heads)
        return 0;
    return plan_attention_fp8(total_q, batch_size, num_q_heads, num_kv_heads, head_size, max_seq_len, window, num_sinks,
                              INT64_MAX).ws_floats * (int64_t)sizeof(float);
}

int gcache_prompt_attention(const gcache_prompt_args* a, hipStream_t stream) {
    if (!a) return GCACHE_ERR_NULL;
    if (a->total_q < 0 || a->batch_size < 0 || a->total_k < 0) return GCACHE_ERR_SHAPE;
    if (a->total_q == 0 || a->batch_size == 0) return GCACHE_OK;
    if (!a->q || !a->out || !a->query_starts || !a->key_starts || (a->total_k > 0 && (!a->k || !a->v)) ||
        (a->accumulate && !a->lse))
        return GCACHE_ERR_NULL;
    int64_t rows;
    if (a->num_q_heads <= 0 || a->num_kv_heads <= 0 || a->num_q_heads % a->num_kv_heads || a->key_size < 8 ||
        a->key_size % 8 || a->value_size < 8 || a->value_size % 8 || a->max_key_len < 0 || a->workspace_bytes < 0 ||
        a->window < 0 || a->num_sinks < 0 || (!a->causal && a->window > 0) || !std::isfinite(a->softmax_scale) ||
        !mul_ok(a->total_q, a->num_q_heads, &rows) || rows > kMaxRows || a->total_k > INT32_MAX - 255 - a->total_q)
        return GCACHE_ERR_SHAPE;
    const int64_t st[8] = {a->q_token_stride, a->q_head_stride, a->k_token_stride, a->k_head_stride, a->v_token_stride,
                           a->v_head_stride, a->out_token_stride, a->out_head_stride};
    const void* at[4] = {a->q, a->k, a->v, a->out};
    for (int i = 0; i < 8; i++) {
        if (st[i] < 0) return GCACHE_ERR_SHAPE;
        if (st[i] % 8 || !aligned(at[i / 2], 16)) return GCACHE_ERR_ALIGN;
    }
    if (a->lse_token_stride < 0 || !rows_apart(a->total_q, a->num_q_heads, st[6], st[7], a->value_size) ||
        (a->lse && a->total_q > 1 && a->lse_token_stride < a->num_q_heads))
        return GCACHE_ERR_SHAPE;
    if (!aligned(a->lse, 4) || !aligned(a->query_starts, 4) || !aligned(a->key_starts, 4) || !aligned(a->workspace, 16))
        return GCACHE_ERR_ALIGN;
    if (a->key_size > 256 || a->value_size > 256 || a->k_token_stride > (1 << 23) || a->v_token_stride > (1 << 23))
        return GCACHE_ERR_UNSUPPORTED;
    const int rc = check_device();
    if (rc) return rc;
    PromptParams p{};
    p.q = static_cast<const uint16_t*>(a->q);
    p.k = static_cast<const uint16_t*>(a->k);
    p.v = static_cast<const uint16_t*>(a->v);
    p.out = static_cast<uint16_t*>(a->out);
    p.lse = a->lse;
    p.q_ts = st[0];
    p.q_hs = st[1];
    p.k_ts = st[2];
    p.k_hs = st[3];
    p.v_ts = st[4];
    p.v_hs = st[5];
    p.o_ts = st[6];
    p.o_hs = st[7];
    p.lse_ts = a->lse_token_stride;
    p.qs = a->query_starts;
    p.ks = a->key_starts;
    p.batch = a->batch_size;
    p.total_q = (int32_t)a->total_q;
    p.total_k = (int32_t)a->total_k;
    p.hq = a->num_q_heads;
    p.hk = a->num_kv_heads;
    p.group = a->num_q_heads / a->num_kv_heads;
    p.dk = a->key_size;
    p.hs = a->value_size;
    p.scale_log2 = (float)(a->softmax_scale * 1.4426950408889634);
    p.window = a->window;
    p.sinks = a->num_sinks;
    p.causal = a->causal != 0;
    p.accumulate = a->accumulate != 0;
    p.div = make_div(1);
    // Chunks of context whose mean is at least 3/4 of the longest are split as if all were alike.  Against the split that
    // batches of unknown lengths get, us, 192 / 128 dims: 176 and 256 row tiles over 2048 keys 52 and 53 against 57 and
    // 66, 272 and 336 over 4096 121 and 130 against 125 and 139, 224 and 256 over 16384 301 and 328 against 313 and 339, 384
    // over 8192 268 against 290; 128 dims, 336 over 4096 105 against 121, 480 and 512 alike.  Lengths that differ, 384
    // tiles: 7200, 5800 and 5400 keys 222 against 240; twice 8192 and 2048 225 against 237; but one of three long, 8192 and
    // twice 5120 241 against 235, and 128 dims, 4096, 2500 and 2900 100 against 93.  The lengths are on the device, so the
    // host cannot tell the last two from the others.
    const bool even = !a->causal && a->max_key_len <= 4 * a->total_k / (3 * (int64_t)a->batch_size);
    const AttnPlan plan = plan_attention_prompt(p.total_q, p.batch, p.hq, p.hk, p.dk, p.hs, a->max_key_len, p.window, p.sinks,
                                                workspace_floats(a->workspace, a->workspace_bytes), even);
    use_plan(plan, a->workspace, &p);
    if (((int64_t)p.units + 7) * p.hk > INT32_MAX) return GCACHE_ERR_SHAPE;  // workgroups are numbered in 32 bits
    return launched(launch_attention_prompt(p, stream));
}

int64_t gcache_prompt_workspace_bytes(int64_t total_q, int32_t batch_size, int32_t num_q_heads, int32_t num_kv_heads,
                                      int32_t key_size, int32_t value_size, int64_t max_key_len, int32_t window,
                                      int32_t num_sinks) {
    if (total_q <= 0 || batch_size <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
        key_size <= 0 || value_size <= 0 || max_key_len < 0 || window < 0 || num_sinks < 0 || total_q > kMaxRows / num_q_heads)
        return 0;
    return plan_attention_prompt(total_q, batch_size, num_q_heads, num_kv_heads, key_size, value_size, max_key_len, window,
                                 num_sinks, INT64_MAX, false).ws_floats * (int64_t)sizeof(float);
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
    return gcache_copy_page_sets(caches, 1, num_blocks, src, dst, num_pairs, stream);
}

int gcache_copy_page_sets(const gcache_page_caches* sets, int32_t num_sets, int64_t num_blocks, const int32_t* src,
                          const int32_t* dst, int64_t num_pairs, hipStream_t stream) {
    if (num_pairs < 0 || num_pairs > kMaxRequests || num_blocks < 0 || num_blocks > INT32_MAX) return GCACHE_ERR_SHAPE;
    int rc = check_sets(sets, num_sets, num_blocks);
    if (rc) return rc;
    bool any = false;
    for (int i = 0; i < num_sets; i++) any = any || moved_caches(sets[i]) > 0;
    if (num_pairs == 0 || !any || num_blocks == 0) return GCACHE_OK;
    if (!src || !dst) return GCACHE_ERR_NULL;
    if (!aligned(src, 4) || !aligned(dst, 4)) return GCACHE_ERR_ALIGN;
    if ((rc = check_device())) return rc;
    hipError_t e = hipSuccess;
    each_list(sets, num_sets, num_blocks, [&](const CacheList& l, bool first, bool last) {
        if (e == hipSuccess) e = launch_copy_pages(l, src, dst, num_pairs, stream, first, last);
    });
    return launched(e);
}

int gcache_fork_requests(const gcache_page_state* state, const gcache_page_caches* caches, const int32_t* parent_rows,
                         const int32_t* child_rows, int64_t num_forks, int32_t* status, void* workspace,
                         int64_t workspace_bytes, hipStream_t stream) {
    return gcache_fork_page_sets(state, caches, 1, parent_rows, child_rows, num_forks, status, workspace, workspace_bytes,
                                 stream);
}

int gcache_fork_page_sets(const gcache_page_state* state, const gcache_page_caches* sets, int32_t num_sets,
                          const int32_t* parent_rows, const int32_t* child_rows, int64_t num_forks, int32_t* status,
                          void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (num_forks < 0) return GCACHE_ERR_SHAPE;
    PageTable t;
    int rc = check_state(state, &t);
    if (rc) return rc;
    if ((rc = check_sets(sets, num_sets, t.num_blocks))) return rc;
    if (num_forks == 0) return GCACHE_OK;
    GrantParams g;
    if ((rc = grant_params(t, parent_rows, child_rows, num_forks, status, workspace, workspace_bytes, &g))) return rc;
    if ((rc = check_device())) return rc;
    hipError_t e = launch_fork_plan(g, stream);
    // the first launch does the rows too, also where no cache has bytes to move
    bool rows = true;
    each_list(sets, num_sets, t.num_blocks, [&](const CacheList& l, bool first, bool last) {
        rows = false;
        if (e == hipSuccess) e = launch_fork_apply(g, l, first, stream, last);
    });
    if (rows && e == hipSuccess) e = launch_fork_apply(g, CacheList{}, true, stream, true);
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
    return gcache_compact_page_sets(state, caches, 1, page_map, workspace, workspace_bytes, stream);
}

int gcache_compact_page_sets(const gcache_page_state* state, const gcache_page_caches* sets, int32_t num_sets,
                             int32_t* page_map, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    PageTable t;
    int rc = check_state(state, &t);
    if (rc) return rc;
    if ((rc = check_sets(sets, num_sets, t.num_blocks))) return rc;
    if (!page_map || !workspace) return GCACHE_ERR_NULL;
    if (workspace_bytes < gcache_pages_workspace_bytes(t.num_blocks, t.num_rows, 0)) return GCACHE_ERR_SHAPE;
    if (!aligned(page_map, 4) || !aligned(workspace, 4)) return GCACHE_ERR_ALIGN;
    if ((rc = check_device())) return rc;
    int32_t* w = static_cast<int32_t*>(workspace);
    const int64_t groups = t.num_blocks / kCompactIds + 1;
    CompactParams c{t, page_map, w, w + groups, w + groups + t.num_blocks, w + groups + 2 * (int64_t)t.num_blocks};
    hipError_t e = launch_compact_plan(c, stream);
    each_list(sets, num_sets, t.num_blocks, [&](const CacheList& l, bool, bool) {
        if (e == hipSuccess) e = launch_compact_move(c, l, stream);
    });
    if (e == hipSuccess) e = launch_compact_finish(c, stream);
    return launched(e);
}

}  // extern "C"
