// attention_join.h -- the end of a query row, the kernel that joins the key
// splits of a row, and the launch sequence of an attention call.
#pragma once

#include "attention_device.h"

namespace gcache {

// How a row's weighted sum becomes its output: out = scale * sum + keep * what
// out holds (keep 0: that is not read).  A call that accumulates joins the row
// with an earlier part, whose lse the caller's lse holds: parts weigh
// exp(lse - max); a part that saw nothing (lse -infinity) does not count,
// whatever its row holds.
struct RowEnd {
    float scale, keep, lse;
};
__device__ __forceinline__ RowEnd row_end(const AttnParams&, int64_t, int, float m, float l, float gv) {
    return RowEnd{l == 0.0f ? 0.0f : gv / l, 0.0f, row_lse(m, l)};
}
__device__ __forceinline__ RowEnd row_end(const PromptParams& p, int64_t token, int head, float m, float l, float gv) {
    RowEnd e{l == 0.0f ? 0.0f : gv / l, 0.0f, row_lse(m, l)};
    if (p.accumulate) {
        const float was = p.lse[token * p.lse_ts + head];
        const float top = fmaxf(was, e.lse);
        if (was != kNegInf) {
            const float a = e.lse == kNegInf ? 0.0f : __builtin_amdgcn_exp2f((e.lse - top) * kLog2e);
            const float b = __builtin_amdgcn_exp2f((was - top) * kLog2e);
            e.scale *= a / (a + b);
            e.keep = b / (a + b);
            e.lse = top + __builtin_log2f(a + b) * kLn2;
        }
    }
    return e;
}
__device__ __forceinline__ bool accumulates(const AttnParams&) { return false; }
__device__ __forceinline__ bool accumulates(const PromptParams& p) { return p.accumulate; }
// Four dims of a row.
__device__ __forceinline__ void write_dims(const AttnParams&, const RowEnd& e, uint16_t* dst, float a, float b, float c, float d) {
    *reinterpret_cast<u32x2*>(dst) = u32x2{pack_bf16x2(a * e.scale, b * e.scale), pack_bf16x2(c * e.scale, d * e.scale)};
}
__device__ __forceinline__ void write_dims(const PromptParams& p, const RowEnd& e, uint16_t* dst, float a, float b, float c, float d) {
    float x[4] = {a * e.scale, b * e.scale, c * e.scale, d * e.scale};
    if (p.accumulate && e.keep != 0.0f) {
        const u32x2 was = *reinterpret_cast<const u32x2*>(dst);
        x[0] = __builtin_fmaf(bf16_lo(was.x), e.keep, x[0]);
        x[1] = __builtin_fmaf(bf16_hi(was.x), e.keep, x[1]);
        x[2] = __builtin_fmaf(bf16_lo(was.y), e.keep, x[2]);
        x[3] = __builtin_fmaf(bf16_hi(was.y), e.keep, x[3]);
    }
    *reinterpret_cast<u32x2*>(dst) = u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
}

// Join the key splits of a row: a wave, or half of one, per (token, head).  The
// splits' maxima and sums are read by a lane each and reduced across the wave;
// the weighted rows follow with four loads in flight.  Bound by the latency of a
// chain of dependent loads, so by rows in flight: the parts of 761 tokens of 32
// heads of 128, seven each on average, take 14 us, and 22 with a wave a row.
constexpr int kMaxSplits = 256;
// Rows and planned splits (half of the bound p.splits) for a workgroup a row: 1
// token of 16 heads over 65536 latent keys 34 us against 54 with a wave a row, 8
// x 1 over 32768 48 against 54; but 2048 rows of 3 splits 46 against 44.
constexpr int kWideRows = 2048, kWideSplits = 32;
// Dims that half a wave's lanes hold, and the splits that they reduce.
constexpr int kHalfDims = 128, kHalfSplits = 32;

// WIDE: the four waves of a workgroup share a row, each with every fourth
// split, so a single token's many splits are not read in one wave's sequence.
// HALF: a row takes half a wave (the same sums in the same order).
template <bool WIDE, bool HALF, typename P>
__global__ __launch_bounds__(kBlockThreads) void k_attention_join(P p, int64_t wg0) {
    constexpr int LANES = HALF ? kWave / 2 : kWave, SPLITS = HALF ? kHalfSplits : kMaxSplits, PER = kWave / LANES;
    __shared__ float s_w[kWavesPerBlock * PER][SPLITS];
    __shared__ f32x4 s_acc[WIDE ? kWavesPerBlock : 1][WIDE ? kNope / 4 : 1];
    const int lane = lane_id() % LANES, part = wave_id() * PER + lane_id() / LANES;
    const int RT = p.row_tile;
    const int64_t id = WIDE ? wg0 + blockIdx.x : (wg0 + blockIdx.x) * (kWavesPerBlock * PER) + part;
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
    t.keys = key_count(p, t.b);
    tile_range(p, t);
    const int chunk = *p.ws_chunk;
    if (t.total <= chunk) return;                        // written by its only workgroup
    const int n = min((t.total - 1) / chunk + 1, request_splits(request_work(p, t.b), chunk));
    float* wts = s_w[part];                              // this row's own (WIDE: this wave's)
    float mk[SPLITS / LANES], lk[SPLITS / LANES], mm = kNegInf, ll = 0.0f;
#pragma unroll
    for (int i = 0; i < SPLITS / LANES; i++) {
        const int k = i * LANES + lane;
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
    for (int d = 1; d < LANES; d <<= 1) mm = fmaxf(mm, __shfl_xor(mm, d));
#pragma unroll
    for (int i = 0; i < SPLITS / LANES; i++) {
        const float wt = mk[i] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mk[i] - mm);
        ll = __builtin_fmaf(wt, lk[i], ll);
        if (i * LANES + lane < n) wts[i * LANES + lane] = wt;
    }
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) ll += __shfl_xor(ll, d);
    const RowEnd end = row_end(p, token, head, mm, ll, p.gscale[1] ? *p.gscale[1] : 1.0f);
    __builtin_amdgcn_wave_barrier();
    constexpr int STEP = WIDE ? kWavesPerBlock : 1;
    const auto write = [&](int d, const f32x4& x) {
        write_dims(p, end, p.out + (int64_t)token * p.o_ts + (int64_t)head * p.o_hs + d, x[0], x[1], x[2], x[3]);
    };
    for (int d = 4 * lane; d < p.hs; d += 4 * LANES) {
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
    if (lane == 0 && p.lse) p.lse[(int64_t)token * p.lse_ts + head] = end.lse;
}

template <typename P>
hipError_t launch_parts(void (*kernel)(P, int64_t), int waves, int row_tile, const P& in, hipStream_t s) {
    P p = in;
    p.blocks = (int32_t)(p.num_blocks < INT32_MAX ? p.num_blocks : INT32_MAX);
    p.data_offset = (uint32_t)p.L.data_offset;
    p.scale_offset = (uint32_t)p.L.scale_offset;
    p.data_token = (uint32_t)p.L.data_token_stride;
    p.scale_token = (uint32_t)p.L.scale_token_stride;
    p.row_tile = row_tile;
    p.group_shift = p.group > 1 ? 32 - __builtin_clz((unsigned)p.group - 1) : 0;
    p.group_mul = (uint32_t)(((uint64_t(1) << (32 + p.group_shift)) + p.group - 1) / p.group - (uint64_t(1) << 32));
    const int64_t units = p.units;
    const bool join = p.splits > 1;
    const hipError_t e = launch_span(kernel, (units + 7) / 8 * 8 * p.hk, waves * kWave, s, true, !join, p);
    if (e != hipSuccess || !join) return e;
    const int64_t rows = (int64_t)p.total_q * p.hq;
    if (rows <= kWideRows && p.splits >= kWideSplits) return launch_span(k_attention_join<true, false, P>, rows, kBlockThreads, s, false, true, p);
    const bool half = p.hs <= kHalfDims && p.splits <= kHalfSplits;
    const int64_t per = kWavesPerBlock * (half ? 2 : 1);
    return launch_span(half ? k_attention_join<false, true, P> : k_attention_join<false, false, P>, (rows + per - 1) / per,
                       kBlockThreads, s, false, true, p);
}

}  // namespace gcache
