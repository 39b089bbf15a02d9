// qk_norm_rope.hip -- root-mean-square norm of every query and key head with
// the position rotation in the same pass:
//   n_i = x_i * w_i / sqrt(mean(x^2) + eps)
//   pairs (a, b) = (n_i, n_{i + rot/2}) or (n_2i, n_{2i+1}), i < rot/2:
//   (a cos_i - b sin_i, b cos_i + a sin_i); values from rot on only normed.
// All in binary32, one rounding to bf16 at the end.
//
// Memory bound: 4 bytes moved a value.  A wave takes one token and several
// of its heads, 8 values (16 bytes) a lane, so cos, sin and the weights are
// loaded once for up to kHeadSets * 64 / lanes-per-head heads and all data
// loads are in flight before the first is used.  The half-split pairing needs
// the chunk rot/2 values away: the partner lane's raw words come by cross-lane
// reads (4 dwords a head) rather than by a second load.
#include "gcache_operators.h"

namespace gcache {

constexpr int kHeadSets = 4;     // heads a lane works on

// q's lanes hold heads [0, heads[0]), k's the ones behind.
__global__ __launch_bounds__(kBlockThreads) void k_qk_norm_rope(QkNormRopeParams p, int64_t wg0) {
    const int lane = lane_id();
    const int64_t wave = (wg0 + blockIdx.x) * kWavesPerBlock + wave_id();
    const int64_t token = wave / p.waves_per_token;
    if (token >= p.num_tokens) return;
    const int lph = 1 << p.lph_shift;                    // lanes of one head
    const int sub = lane & (lph - 1), dim = 8 * sub;     // the lane's values dim .. dim + 7
    const int head0 = (int)(wave - token * p.waves_per_token) * (kHeadSets << (6 - p.lph_shift)) + (lane >> p.lph_shift);
    const int total = p.heads[0] + p.heads[1];
    const bool in_dim = dim < p.hs;

    uint4 x[kHeadSets];
#pragma unroll
    for (int u = 0; u < kHeadSets; u++) {
        const int h = head0 + (u << (6 - p.lph_shift));
        x[u] = make_uint4(0, 0, 0, 0);
        if (h < total && in_dim) {
            const int kk = h >= p.heads[0];
            x[u] = ld_stream16(p.x[kk] + token * p.x_ts[kk] + (int64_t)(h - (kk ? p.heads[0] : 0)) * p.x_hs[kk] + dim);
        }
    }
    const int64_t pos = p.rot > 0 ? p.positions[token] : 0;
    const bool pos_ok = p.rot == 0 || (pos >= 0 && pos < p.max_pos);
    const bool turn = dim < p.rot && pos_ok;
    const int half = p.rot / 2;
    const int partner = dim < half ? sub + half / 8 : sub - half / 8;   // half-split pairing
    // cos and sin of the lane's values: 8 of each, or 4 for the interleaved pairs
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; i++) cs[i] = 1.0f, sn[i] = 0.0f;
    if (turn) {
        const int at = p.interleaved ? dim / 2 : dim < half ? dim : dim - half;
        const int n = p.interleaved ? 4 : 8;
        if (p.cs_bf16) {
            const uint16_t* row = static_cast<const uint16_t*>(p.cos_sin) + pos * p.cs_stride;
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (i < n) {
                    cs[i] = __uint_as_float((uint32_t)row[at + i] << 16);
                    sn[i] = __uint_as_float((uint32_t)row[half + at + i] << 16);
                }
        } else {
            const float* row = static_cast<const float*>(p.cos_sin) + pos * p.cs_stride;
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (i < n) {
                    cs[i] = row[at + i];
                    sn[i] = row[half + at + i];
                }
        }
    }
#pragma unroll
    for (int u = 0; u < kHeadSets; u++) {
        const int h = head0 + (u << (6 - p.lph_shift));
        const int kk = h >= p.heads[0];
        const uint32_t xw[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        float v[8], ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = bf16_lo(xw[i]);
            v[2 * i + 1] = bf16_hi(xw[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; i++) ss = __builtin_fmaf(v[i], v[i], ss);
        for (int st = 1; st < lph; st <<= 1) ss += __shfl_xor(ss, st);
        const float inv = 1.0f / __builtin_sqrtf(ss / (float)p.hs + p.eps);
        uint32_t pw[4];
#pragma unroll
        for (int i = 0; i < 4; i++) pw[i] = __shfl(xw[i], (lane & ~(lph - 1)) | (partner & (lph - 1)));
        if (h >= total || !in_dim) continue;
        const uint4 wl = *reinterpret_cast<const uint4*>(p.w[kk] + dim);
        const uint32_t ww[4] = {wl.x, wl.y, wl.z, wl.w};
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            y[2 * i] = v[2 * i] * inv * bf16_lo(ww[i]);
            y[2 * i + 1] = v[2 * i + 1] * inv * bf16_hi(ww[i]);
        }
        if (turn) {
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float a = y[2 * i], b = y[2 * i + 1];
                    y[2 * i] = a * cs[i] - b * sn[i];
                    y[2 * i + 1] = b * cs[i] + a * sn[i];
                }
            } else {
                const uint4 wp = *reinterpret_cast<const uint4*>(p.w[kk] + 8 * partner);
                const uint32_t wq[4] = {wp.x, wp.y, wp.z, wp.w};
                const float sign = dim < half ? -1.0f : 1.0f;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float a = bf16_lo(pw[i]) * inv * bf16_lo(wq[i]), b = bf16_hi(pw[i]) * inv * bf16_hi(wq[i]);
                    y[2 * i] = y[2 * i] * cs[2 * i] + sign * a * sn[2 * i];
                    y[2 * i + 1] = y[2 * i + 1] * cs[2 * i + 1] + sign * b * sn[2 * i + 1];
                }
            }
        }
        uint4 o = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                             pack_bf16x2(y[6], y[7]));
        if (!pos_ok) o = make_uint4(0, 0, 0, 0);
        st_stream16(p.y[kk] + token * p.y_ts[kk] + (int64_t)(h - (kk ? p.heads[0] : 0)) * p.y_hs[kk] + dim, o);
    }
}

hipError_t launch_qk_norm_rope(const QkNormRopeParams& in, hipStream_t s) {
    QkNormRopeParams p = in;
    p.lph_shift = 1;                                     // hs >= 16: two lanes at least
    while ((8 << p.lph_shift) < p.hs) p.lph_shift++;
    const int per_wave = kHeadSets << (6 - p.lph_shift);
    p.waves_per_token = (p.heads[0] + p.heads[1] + per_wave - 1) / per_wave;
    const int64_t waves = p.num_tokens * p.waves_per_token;
    return launch_span(k_qk_norm_rope, (waves + kWavesPerBlock - 1) / kWavesPerBlock, kBlockThreads, s, true, true, p);
}

}  // namespace gcache
