// attention_plan.hip -- host side of the attention calls: which kernel, how
// many key splits, the launch sequence; and the kernel that joins the splits.
#include "attention_device.h"

namespace gcache {

// Join the key splits of a row: one wave per (token, head).  The splits'
// maxima and sums are read by a lane each and reduced across the wave; the
// weighted rows follow with four loads in flight.  Bound by memory: the parts
// of 761 tokens of 32 heads of 128, seven each on average, take 26 us.
constexpr int kMaxSplits = 256;
// Rows and planned splits (half of the bound p.splits) for a workgroup a row: 1
// token of 16 heads over 65536 latent keys 34 us against 54 with a wave a row, 8
// x 1 over 32768 48 against 54; but 2048 rows of 3 splits 46 against 44.
constexpr int kWideRows = 2048, kWideSplits = 32;

// WIDE: the four waves of a workgroup share a row, each with every fourth
// split, so a single token's many splits are not read in one wave's sequence.
template <bool WIDE>
__global__ __launch_bounds__(kBlockThreads) void k_attention_join(AttnParams p, int64_t wg0) {
    __shared__ float s_w[kWavesPerBlock][kMaxSplits];
    __shared__ f32x4 s_acc[WIDE ? kWavesPerBlock : 1][WIDE ? kNope / 4 : 1];
    const int lane = lane_id();
    const int RT = p.row_tile;
    const int64_t id = WIDE ? wg0 + blockIdx.x : (wg0 + blockIdx.x) * kWavesPerBlock + wave_id();
    const int64_t rows = (int64_t)p.total_q * p.hq;
    if (id >= rows) return;
    const int token = (int)(id / p.hq), head = (int)(id % p.hq);
    int lo = 0, hi = p.batch;                            // the last request that starts at or before token
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (query_start(p, mid) <= token) lo = mid;
        else hi = mid;
    }
    RowTile t;
    t.b = lo;
    t.q0 = query_start(p, lo);
    t.qlen = query_start(p, lo + 1) - t.q0;
    const int tl = token - t.q0;
    if (tl < 0 || tl >= t.qlen) return;                  // a row of no request
    const int row = tl * p.group + head % p.group;
    t.row0 = row / RT * RT;
    t.rows = (int)min((int64_t)RT, (int64_t)t.qlen * p.group - t.row0);
    tile_range(p, t);
    const int chunk = *p.ws_chunk;
    if (t.total <= chunk) return;                        // written by its only workgroup
    const int n = min((t.total - 1) / chunk + 1, request_splits(request_work(p, t.b), chunk));
    float* wts = s_w[wave_id()];                         // this wave's own
    float mk[kMaxSplits / kWave], lk[kMaxSplits / kWave], mm = kNegInf, ll = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxSplits / kWave; i++) {
        const int k = i * kWave + lane;
        mk[i] = kNegInf;
        lk[i] = 0.0f;
        if (k < n) {
            const float2 ml = *reinterpret_cast<const float2*>(p.ws_ml + 2 * (k * rows + id));
            mk[i] = ml.x;
            lk[i] = ml.y;
        }
        mm = fmaxf(mm, mk[i]);
    }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) mm = fmaxf(mm, __shfl_xor(mm, d));
#pragma unroll
    for (int i = 0; i < kMaxSplits / kWave; i++) {
        const float wt = mk[i] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mk[i] - mm);
        ll = __builtin_fmaf(wt, lk[i], ll);
        if (i * kWave + lane < n) wts[i * kWave + lane] = wt;
    }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) ll += __shfl_xor(ll, d);
    const float scale = ll == 0.0f ? 0.0f : (p.gscale[1] ? *p.gscale[1] : 1.0f) / ll;
    __builtin_amdgcn_wave_barrier();
    constexpr int STEP = WIDE ? kWavesPerBlock : 1;
    const auto write = [&](int d, const f32x4& x) {
        *reinterpret_cast<u32x2*>(p.out + (int64_t)token * p.o_ts + (int64_t)head * p.o_hs + d) =
            u32x2{pack_bf16x2(x[0] * scale, x[1] * scale), pack_bf16x2(x[2] * scale, x[3] * scale)};
    };
    for (int d = 4 * lane; d < p.hs; d += 4 * kWave) {
        f32x4 acc = {0, 0, 0, 0};
        const float* src = p.ws_o + id * p.hs + d;
        int k = WIDE ? wave_id() : 0;
        for (; k + 3 * STEP < n; k += 4 * STEP) {
            f32x4 x[4];
#pragma unroll
            for (int u = 0; u < 4; u++) x[u] = *reinterpret_cast<const f32x4*>(src + (k + u * STEP) * rows * p.hs);
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const float wt = wts[k + u * STEP];
#pragma unroll
                for (int i = 0; i < 4; i++) acc[i] = __builtin_fmaf(wt, x[u][i], acc[i]);
            }
        }
        for (; k < n; k += STEP) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(src + k * rows * p.hs);
#pragma unroll
            for (int i = 0; i < 4; i++) acc[i] = __builtin_fmaf(wts[k], x[i], acc[i]);
        }
        if (WIDE) s_acc[wave_id()][d / 4] = acc;
        else write(d, acc);
    }
    if (WIDE) {
        __syncthreads();
        const int c = threadIdx.x;
        if (4 * c < p.hs) write(4 * c, (s_acc[0][c] + s_acc[WIDE ? 1 : 0][c]) + (s_acc[WIDE ? 2 : 0][c] + s_acc[WIDE ? 3 : 0][c]));
        if (c > 0) return;
    }
    if (lane == 0 && p.lse)
        p.lse[(int64_t)token * p.lse_ts + head] =
            row_lse(mm, ll);
}

AttnPlan plan_attention(int64_t total_q, int32_t batch, int32_t hq, int32_t hk, int32_t dp, int32_t dv,
                        int64_t max_seq_len, int32_t window, int32_t sinks, int64_t ws_floats_avail) {
    AttnPlan a;
    const int64_t group = hq / hk, rows = total_q * group;
    const int64_t mean = (rows + batch - 1) / batch;     // rows of a request and kv head
    // Rows of a workgroup, measured over 8192 keys, group 4, at equal splits:
    //   16 against 32 rows (per head, 64 x 1 token)                169 us against 206
    //   32 against 16 (32 x 8 tokens; two tiles read the keys twice)  112 against 163
    //   32 in the few-rows kernel against the rows kernel          112 against 164
    //   head size 256, 16 rows twice against the rows kernel       122 against 177
    //   64 rows, few-rows kernel against the rows kernel           203 against 185
    //   latent, 32 rows: 16 twice against the 64-row kernel         82 against 85
    //   latent, 64 rows: 16 four times against the 64-row kernel   128 against 93
    a.row_tiles = mean <= 16 || (dp >= 256 && mean <= 32) ? 1 : mean <= 32 ? 2 : dp > 256 ? 4 : 8;
    const int64_t rt = 16 * a.row_tiles;
    a.tiles = (int32_t)((rows + (rt - 1) * batch) / rt);
    // 32-key tiles that a row tile can see (a bound; only the split depends on it)
    int64_t kt = (max_seq_len + kTileKeys - 1) / kTileKeys;
    if (window > 0) {
        const int64_t seen = ((int64_t)window + rt / group + 1 + sinks) / kTileKeys + 3;
        if (seen < kt) kt = seen;
    }
    if (kt > INT32_MAX / kTileKeys) kt = INT32_MAX / kTileKeys;
    if (kt < 1) kt = 1;
    // Work units: rounds of resident workgroups x (key tiles of a split + what a
    // split costs besides: its start, and its part of the output, written and
    // read again) + half a split for the ragged end, in units of one tile's
    // time, for requests of equal length; the kernels size the splits so that
    // other lengths give as many.  The cost of a split was found by sweeping it:
    // 12, 32 and 96 tiles for many rows give 589, 499 and 503 us for 32 x 32
    // latent tokens over 8192 keys, 235, 215 and 216 for 16 x 64 per-head ones;
    // 6 and 20 for few rows 130 and 121 for 128 x 1 latent tokens.
    const int64_t groups = (mean + rt - 1) / rt * batch * hk;
    const bool few = a.row_tiles <= 2;
    const int64_t slots = 256 * (!few ? (dp <= 128 ? 2 : 1) : a.row_tiles * dp <= 128 ? 3 : 2);
    const int64_t extra = few ? 24 : 40;
    const auto rounds = [&](int64_t units) { return (units + slots - 1) / slots; };
    const int64_t per = total_q * hq * (dv + 2);         // floats of a split; one more split's room holds the chunk
    const int64_t room = per > 0 ? ws_floats_avail / per - 1 : 0;
    int64_t top = kt / 4 < kMaxSplits ? kt / 4 : kMaxSplits;    // at least a tile for each of four waves
    if (top > room) top = room;
    int64_t most = top;
    if (most > 8 * slots / groups) most = 8 * slots / groups;   // eight rounds are even enough
    if (!counts_requests(batch, hk)) most = 1;
    int64_t splits = 1, best = rounds(groups) * kt + kt / 2;
    for (int64_t n = 2; n <= most; n += n < 16 ? 1 : n / 16) {
        const int64_t c = ((kt + n - 1) / n + 3) / 4 * 4, m = (kt + c - 1) / c;
        const int64_t cost = rounds(groups * m) * (c + extra) + c / 2;
        if (cost < best) {
            best = cost;
            splits = m;
        }
    }
    a.key_tiles = (int32_t)kt;
    a.units = a.tiles;
    // whole rounds: uneven requests fill them (a launch that is smaller than one stays as it is)
    int64_t units = splits * groups;
    if (units > slots) units = rounds(units) * slots;
    if (splits > 1 && units / hk > a.tiles) a.units = (int32_t)(units / hk);
    // requests longer than the mean are split further
    a.splits = (int32_t)(splits == 1 ? 1 : 2 * splits < top ? 2 * splits : top);
    a.ws_floats = splits > 1 ? (a.splits + 1) * per : 0;
    return a;
}

// 16 keys of one page, with the head and side offsets, within 32 bits.
bool uniform_pages(const AttnParams& p) {
    const int64_t room = INT32_MAX / 4;
    return p.div.size % 16 == 0 && p.L.data_offset < room && p.L.scale_offset < room &&
           p.L.data_token_stride < room / p.div.size && p.L.scale_token_stride < room / p.div.size &&
           p.L.data_head_stride < room / p.hk && p.L.scale_head_stride < room / p.hk && p.L.side_stride < room;
}

hipError_t launch_attention_parts(void (*kernel)(AttnParams, int64_t), int waves, int row_tile, const AttnParams& in,
                                  hipStream_t s) {
    AttnParams p = in;
    p.blocks = (int32_t)(p.num_blocks < INT32_MAX ? p.num_blocks : INT32_MAX);
    p.data_offset = (uint32_t)p.L.data_offset;
    p.scale_offset = (uint32_t)p.L.scale_offset;
    p.data_token = (uint32_t)p.L.data_token_stride;
    p.scale_token = (uint32_t)p.L.scale_token_stride;
    p.row_tile = row_tile;
    const int64_t units = p.units;
    const bool join = p.splits > 1;
    const hipError_t e = launch_span(kernel, (units + 7) / 8 * 8 * p.hk, waves * kWave, s, true, !join, p);
    if (e != hipSuccess || !join) return e;
    const int64_t rows = (int64_t)p.total_q * p.hq;
    if (rows <= kWideRows && p.splits >= kWideSplits) return launch_span(k_attention_join<true>, rows, kBlockThreads, s, false, true, p);
    return launch_span(k_attention_join<false>, (rows + kWavesPerBlock - 1) / kWavesPerBlock, kBlockThreads, s, false, true, p);
}

}  // namespace gcache
