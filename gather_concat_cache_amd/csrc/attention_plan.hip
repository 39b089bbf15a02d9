// attention_plan.hip -- host side of the attention calls: which kernel, how
// many key splits, the launch sequence.
#include "attention_join.h"

namespace gcache {

AttnPlan plan_attention(int64_t total_q, int32_t batch, int32_t hq, int32_t hk, int32_t dp, int32_t dv,
                        int64_t max_seq_len, int32_t window, int32_t sinks, int64_t ws_floats_avail) {
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
    const int row_tiles = mean <= 16 || (dp >= 256 && mean <= 32) ? 1 : mean <= 32 ? 2 : dp > 256 ? 4 : 8;
    const int64_t slots = 256 * (row_tiles > 2 ? (dp <= 128 ? 2 : 1) : row_tiles * dp <= 128 ? 3 : 2);
    return plan_attention_rows(row_tiles, slots, total_q, batch, hq, hk, dv, max_seq_len, window, sinks, ws_floats_avail);
}

AttnPlan plan_attention_rows(int row_tiles, int64_t slots, int64_t total_q, int32_t batch, int32_t hq, int32_t hk,
                             int32_t dv, int64_t max_seq_len, int32_t window, int32_t sinks, int64_t ws_floats_avail,
                             bool even) {
    AttnPlan a;
    const int64_t group = hq / hk, rows = total_q * group;
    const int64_t mean = (rows + batch - 1) / batch;     // rows of a request and kv head
    a.row_tiles = row_tiles;
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
    // even: all row tiles see about as many keys, so the ragged end is a quarter.
    const int64_t ragged = even ? 4 : 2;
    const int64_t groups = (mean + rt - 1) / rt * batch * hk;
    const bool few = a.row_tiles <= 2;
    const int64_t extra = few ? 24 : 40;
    const auto rounds = [&](int64_t units) { return (units + slots - 1) / slots; };
    const int64_t per = total_q * hq * (dv + 2);         // floats of a split; one more split's room holds the chunk
    const int64_t room = per > 0 ? ws_floats_avail / per - 1 : 0;
    int64_t top = kt / 4 < kMaxSplits ? kt / 4 : kMaxSplits;    // at least a tile for each of four waves
    if (top > room) top = room;
    int64_t most = top;
    if (most > 8 * slots / groups) most = 8 * slots / groups;   // eight rounds are even enough
    if (!counts_requests(batch, hk)) most = 1;
    int64_t splits = 1, best = rounds(groups) * kt + kt / ragged;
    for (int64_t n = 2; n <= most; n += n < 16 ? 1 : n / 16) {
        const int64_t c = ((kt + n - 1) / n + 3) / 4 * 4, m = (kt + c - 1) / c;
        const int64_t cost = rounds(groups * m) * (c + extra) + c / ragged;
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

hipError_t launch_attention_parts(void (*kernel)(AttnParams, int64_t), int waves, int row_tile, const AttnParams& p,
                                  hipStream_t s) {
    return launch_parts(kernel, waves, row_tile, p, s);
}

}  // namespace gcache
