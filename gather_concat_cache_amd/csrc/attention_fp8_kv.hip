// attention_fp8_kv.hip -- attention over a paged cache of e4m3 keys and values
// with a scale for each page, side and head.
//
// Mathematics.  A logit is softmax_scale * kscale * q . code.  The value scales
// differ from page to page, so they ride on the weights: with a row's
// m = max over its keys of s_j + log2 vscale_j (log2 units),
//     P_j = exp2(s_j + log2 vscale_j - m),  o = sum P_j code_j / sum P_j / vscale_j,
// which keeps the weights that meet the codes within binary16 whatever the
// scales are.  The scales are constant over the keys of a page, so this costs
// no operation a weight.  Scores are binary32 sums of exact products of
// binary16 (an e4m3 value is exact there, a query row is scaled by a power of
// two); only the weights are rounded, to 11 bits, shifted up so that they stay
// normal down to 2^-20 of the largest.
#include "attention_tiles.h"

namespace gcache {

template <int DP, bool UNI, bool TREE>
__global__ __launch_bounds__(kTileWaves * kWave, DP <= 128 ? 2 : 1) void k_fp8_rows(AttnParams p, int64_t wg0) {
    __shared__ StepLds<PagedFp8, DP, DP, UNI> lds;
    // heads of a unit 8 apart: the same XCD
    const int64_t wg = wg0 + blockIdx.x, per = 8 * (int64_t)p.hk;
    const int rem = (int)(wg % per), kvh = rem / 8;
    RowTile t;
    if (!find_tile(p, wg / per * 8 + rem % 8, kTileRows, t)) return;
    int v0, v1;
    if (!key_range(t, v0, v1)) return;
    attend_tile<PagedFp8, DP, DP, 1, UNI, TREE>(p, t, kvh, v0, v1, lds);
}

template <int DP>
static hipError_t launch_rows(const AttnParams& p, bool uni, hipStream_t s) {
    return launch_parts(p.mask ? (uni ? k_fp8_rows<DP, true, true> : k_fp8_rows<DP, false, true>)
                               : (uni ? k_fp8_rows<DP, true, false> : k_fp8_rows<DP, false, false>),
                        kTileWaves, kTileRows, p, s);
}

// Pages of whole 16-key groups whose rows are within 32 bits of each other, and
// a head size that is a form's own.
static bool uniform_fp8(const AttnParams& p, int dp) {
    return p.hs == dp && p.div.size % 16 == 0 && p.L.data_token_stride < (int64_t(1) << 26);
}

hipError_t launch_attention_fp8(const AttnParams& p, int row_tiles, hipStream_t s) {
    if (p.hs <= 64) return launch_rows<64>(p, uniform_fp8(p, 64), s);
    if (p.hs <= 128) return launch_rows<128>(p, uniform_fp8(p, 128), s);
    return launch_rows<256>(p, uniform_fp8(p, 256), s);
}

AttnPlan plan_attention_fp8(int64_t total_q, int32_t batch, int32_t hq, int32_t hk, int32_t hs, int64_t max_seq_len,
                            int32_t window, int32_t sinks, int64_t ws_floats_avail) {
    return plan_attention_rows(kTileRows / 16, 256 * (hs <= 128 ? 2 : 1), total_q, batch, hq, hk, hs, max_seq_len, window,
                               sinks, ws_floats_avail);
}

}  // namespace gcache
