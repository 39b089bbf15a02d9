// prompt_attention.hip -- attention of packed prompts: bf16 queries over bf16
// keys and values, both in rows of sequences that follow each other.
//
// Bound by the matrix and vector instructions of two waves a SIMD that do not
// fully overlap.  4 x 4096 tokens, not causal, TFLOP/s: 128 dims 1000, keys of
// 192 and values of 128 1105, 256 dims 905 (one workgroup a CU: its accumulators
// fill the registers), 64 800 (as many exponentials for half the products).
// Head sizes between run in the next larger form with a test a chunk (80: 687
// of its own operations).
#include "attention_tiles.h"

namespace gcache {

template <int DK, int DV, bool EX>
__global__ __launch_bounds__(kTileWaves * kWave, DK <= 192 ? 2 : 1) void k_prompt(PromptParams p, int64_t wg0) {
    __shared__ StepLds<PackedBf16, DK, DV, EX> lds;
    uint32_t kvh, unit;
    if (!head_and_unit(p, (uint32_t)wg0 + blockIdx.x, kvh, unit)) return;
    RowTile t;
    if (!find_tile<true>(p, unit, kTileRows, t)) return;
    int v0, v1;
    if (!key_range(t, v0, v1)) return;
    attend_tile<PackedBf16, DK, DV, EX, false>(p, t, (int)kvh, v0, v1, lds);
}

template <int DK, int DV>
static hipError_t launch_prompt(const PromptParams& p, hipStream_t s) {
    const bool ex = p.dk == DK && p.hs == DV;
    return launch_parts(ex ? k_prompt<DK, DV, true> : k_prompt<DK, DV, false>, kTileWaves, kTileRows, p, s);
}

// The smallest of four forms that holds both head sizes.
hipError_t launch_attention_prompt(const PromptParams& p, hipStream_t s) {
    if (p.dk <= 64 && p.hs <= 64) return launch_prompt<64, 64>(p, s);
    if (p.dk <= 128 && p.hs <= 128) return launch_prompt<128, 128>(p, s);
    if (p.dk <= 192 && p.hs <= 128) return launch_prompt<192, 128>(p, s);
    return launch_prompt<256, 256>(p, s);
}

AttnPlan plan_attention_prompt(int64_t total_q, int32_t batch, int32_t hq, int32_t hk, int32_t dk, int32_t dv,
                               int64_t max_key_len, int32_t window, int32_t sinks, int64_t ws_floats_avail, bool even) {
    const int64_t slots = 256 * (dk <= 192 && dv <= 128 ? 2 : 1);
    return plan_attention_rows(kTileRows / 16, slots, total_q, batch, hq, hk, dv, max_key_len, window, sinks, ws_floats_avail,
                               even);
}

}  // namespace gcache
