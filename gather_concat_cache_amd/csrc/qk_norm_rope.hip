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
// loads are in flight before the first is used.  Sums over a head's lanes come
// by lane permutes inside the vector unit, the partner values of the half-split
// pairing (rot/2 away) by one shuffle.  16384 tokens of 40 heads of 128 values,
// data from HBM: 85 us (4.1 TB/s); the first form, with shuffles through LDS
// for the sums, scalar table loads and IEEE division, 117 us.
#include "gcache_operators.h"

namespace gcache {

// A set is the heads that one load of a wave holds (4 of 128 values).  A token
// takes as few waves as hold its sets at kHeadSets each, and the sets are dealt
// evenly, so that fewer of them than waves stay empty.
// At most 4, 5, 6 and 8 sets, 16384 tokens (us): 28 + 4 heads of 128 70.0,
// 70.1, 70.2, 71.5; 32 + 8 93.0, 85.1, 85.0, 92.1; 64 + 8 156.8, 152.7, 145.0,
// 158.2; 16 + 2 36.6, 32.6, 32.6, 35.5; 16 + 16 of 64 29.1, 29.2, 29.3, 30.4; 4096
// tokens of 16 + 2 of 512 32.1, 31.6, 30.5, 31.6.  (Always 5, uneven: 28 + 4 72.1.)
constexpr int kHeadSets = 6;

typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
// Sum over aligned groups of 2^SH lanes.
template <int SH>
__device__ __forceinline__ float head_sum(float v) {
    if (SH >= 1) v += __uint_as_float(dpp<0xB1>(__float_as_uint(v)));    // lane ^ 1
    if (SH >= 2) v += __uint_as_float(dpp<0x4E>(__float_as_uint(v)));    // lane ^ 2
    if (SH >= 3) v += __uint_as_float(dpp<0x141>(__float_as_uint(v)));   // mirror in 8: the other 4
    if (SH >= 4) v += __uint_as_float(dpp<0x140>(__float_as_uint(v)));   // mirror in 16: the other 8
    if (SH >= 5) v += __shfl_xor(v, 16);
    if (SH >= 6) v += __shfl_xor(v, 32);
    return v;
}

// The norm of heads (out) whose mean square lies outside [kMeanLow,
// kMeanHigh], where single squares are subnormal or overflow, again from
// values times 2^100 (small) or 2^-100.  Small values stay scaled, exactly, in
// xw and v; inv fits what is there.  Asking costs every call 0.2 to 0.4 us (of
// 85 for 16384 tokens of 40 heads of 128).
constexpr float kMeanLow = 0x1p-96f, kMeanHigh = 0x1p+120f, kUp = 0x1p+100f, kDown = 0x1p-100f;
template <int SH>
__device__ __forceinline__ void wide_range(bool out, bool small, float inv_hs, float eps, uint32_t* xw, float* v, float& inv) {
    const float by = small ? kUp : kDown;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) ss = __builtin_fmaf(v[i] * by, v[i] * by, ss);
    ss = head_sum<SH>(ss);
    const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, inv_hs, eps * by * by));
    if (!out) return;
    inv = small ? r : r * kDown;
    if (!small) return;
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] *= kUp;
#pragma unroll
    for (int i = 0; i < 4; i++) xw[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
}

// N consecutive table values as floats.
template <int N, bool BF16>
__device__ __forceinline__ void table_values(const void* row, int at, float* out) {
    if (BF16) {
        const uint16_t* r = static_cast<const uint16_t*>(row) + at;
        uint32_t w[4] = {0, 0, 0, 0};
        if (N == 8) {
            const u32x4 x = *reinterpret_cast<const u32x4_a2*>(r);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else {
            const u32x2 x = *reinterpret_cast<const u32x2_a2*>(r);
            w[0] = x.x, w[1] = x.y;
        }
#pragma unroll
        for (int i = 0; i < N / 2; i++) {
            out[2 * i] = bf16_lo(w[i]);
            out[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
        const float* r = static_cast<const float*>(row) + at;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u32x4 x = *reinterpret_cast<const u32x4_a4*>(r + i);
            out[i] = __uint_as_float(x.x);
            out[i + 1] = __uint_as_float(x.y);
            out[i + 2] = __uint_as_float(x.z);
            out[i + 3] = __uint_as_float(x.w);
        }
    }
}

// SH: log2 of the lanes of a head.  q's heads come first, k's behind.
template <int SH, bool INTER, bool BF16>
__global__ __launch_bounds__(kBlockThreads) void k_qk_norm_rope(QkNormRopeParams p, int64_t wg0) {
    constexpr int LPH = 1 << SH, HPW = 64 >> SH;         // lanes of a head, heads a wave's load holds
    const int lane = lane_id();
    const int64_t wave = (wg0 + blockIdx.x) * kWavesPerBlock + wave_id();
    const int64_t token = wave / p.waves_per_token;
    if (token >= p.num_tokens) return;
    const int sub = lane & (LPH - 1), dim = 8 * sub;     // the lane's values dim .. dim + 7
    const int first = (int)(wave - token * p.waves_per_token) * (p.sets * HPW), head0 = first + (lane >> SH);
    const int end = min(p.heads[0] + p.heads[1], first + p.sets * HPW);  // behind the wave's heads
    const bool in_dim = dim < p.hs;
    const int64_t pos = p.rot > 0 ? p.positions[token] : 0;

    uint4 x[kHeadSets];
#pragma unroll
    for (int u = 0; u < kHeadSets; u++) {
        const int h = head0 + u * HPW;
        x[u] = make_uint4(0, 0, 0, 0);
        if (h < end && in_dim) {
            const int kk = h >= p.heads[0];
            x[u] = *reinterpret_cast<const uint4*>(p.x[kk] + token * p.x_ts[kk] +
                                                  (int64_t)(h - (kk ? p.heads[0] : 0)) * p.x_hs[kk] + dim);
        }
    }
    const bool pos_ok = p.rot == 0 || (pos >= 0 && pos < p.max_pos);
    const bool turn = dim < p.rot && pos_ok;
    const int half = p.rot / 2;
    const bool low = dim < half;
    const int partner = low ? sub + half / 8 : sub - half / 8;          // half-split pairing
    // cos and sin of the lane's values (of its four pairs when interleaved), the weights of both sides
    constexpr int N = INTER ? 4 : 8;
    float cs[N], sn[N];
#pragma unroll
    for (int i = 0; i < N; i++) cs[i] = 1.0f, sn[i] = 0.0f;
    if (turn) {
        const int at = INTER ? dim / 2 : low ? dim : dim - half;
        const void* row = static_cast<const uint8_t*>(p.cos_sin) + pos * p.cs_stride * (BF16 ? 2 : 4);
        table_values<N, BF16>(row, at, cs);
        table_values<N, BF16>(row, half + at, sn);
        if (!INTER)
#pragma unroll
            for (int i = 0; i < N; i++) sn[i] = low ? -sn[i] : sn[i];
    }
    float w[2][8], wp[2][8];                             // of the lane's values, of the partner's
#pragma unroll
    for (int kk = 0; kk < 2; kk++) {
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (p.heads[kk] > 0 && in_dim) {
            a = *reinterpret_cast<const uint4*>(p.w[kk] + dim);
            if (!INTER && turn) b = *reinterpret_cast<const uint4*>(p.w[kk] + 8 * partner);
        }
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            w[kk][2 * i] = bf16_lo(aw[i]);
            w[kk][2 * i + 1] = bf16_hi(aw[i]);
            wp[kk][2 * i] = bf16_lo(bw[i]);
            wp[kk][2 * i + 1] = bf16_hi(bw[i]);
        }
    }
#pragma unroll
    for (int u = 0; u < kHeadSets; u++) {
        if (u >= p.sets) break;
        const int h = head0 + u * HPW;
        const int kk = h >= p.heads[0];
        uint32_t xw[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        float v[8], ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = bf16_lo(xw[i]);
            v[2 * i + 1] = bf16_hi(xw[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; i++) ss = __builtin_fmaf(v[i], v[i], ss);
        ss = head_sum<SH>(ss);
        const float mean = __builtin_fmaf(ss, p.inv_hs, p.eps);
        // v_rsq_f32: one ulp, against the bf16 rounding at the end
        float inv = __builtin_amdgcn_rsqf(mean);
        // squares that leave binary32, and means that v_rsq_f32 takes as 0 (the same for all lanes of a head; rare, so the
        // wave decides)
        const bool out = !(mean >= kMeanLow && mean <= kMeanHigh);
        if (__builtin_expect(__any(out), 0)) wide_range<SH>(out, mean < kMeanLow, p.inv_hs, p.eps, xw, v, inv);
        uint32_t pw[4];
        if (!INTER)
#pragma unroll
            for (int i = 0; i < 4; i++)
                pw[i] = (uint32_t)__shfl((int)xw[i], (lane & ~(LPH - 1)) | (partner & (LPH - 1)));
        if (h >= end || !in_dim) continue;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = v[i] * inv * (kk ? w[1][i] : w[0][i]);
        if (turn) {
            if (INTER) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float a = y[2 * i], b = y[2 * i + 1];
                    y[2 * i] = a * cs[i] - b * sn[i];
                    y[2 * i + 1] = b * cs[i] + a * sn[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float b = (i & 1 ? bf16_hi(pw[i / 2]) : bf16_lo(pw[i / 2])) * inv * (kk ? wp[1][i] : wp[0][i]);
                    y[i] = y[i] * cs[i % N] + b * sn[i % N];
                }
            }
        }
        uint4 o = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                             pack_bf16x2(y[6], y[7]));
        if (!pos_ok) o = make_uint4(0, 0, 0, 0);
        st_stream16(p.y[kk] + token * p.y_ts[kk] + (int64_t)(h - (kk ? p.heads[0] : 0)) * p.y_hs[kk] + dim, o);
    }
}

template <int SH>
static hipError_t launch_lanes(const QkNormRopeParams& in, hipStream_t s) {
    QkNormRopeParams p = in;
    // as few waves as hold the token's heads, each with as many sets as the others
    const int sets = (p.heads[0] + p.heads[1] + (64 >> SH) - 1) / (64 >> SH);
    p.waves_per_token = (sets + kHeadSets - 1) / kHeadSets;
    p.sets = (sets + p.waves_per_token - 1) / p.waves_per_token;
    p.inv_hs = 1.0f / (float)p.hs;
    const int64_t wgs = (p.num_tokens * p.waves_per_token + kWavesPerBlock - 1) / kWavesPerBlock;
    auto k = p.interleaved ? (p.cs_bf16 ? k_qk_norm_rope<SH, true, true> : k_qk_norm_rope<SH, true, false>)
                           : (p.cs_bf16 ? k_qk_norm_rope<SH, false, true> : k_qk_norm_rope<SH, false, false>);
    return launch_span(k, wgs, kBlockThreads, s, true, true, p);
}

hipError_t launch_qk_norm_rope(const QkNormRopeParams& p, hipStream_t s) {
    return p.hs <= 16 ? launch_lanes<1>(p, s) : p.hs <= 32 ? launch_lanes<2>(p, s) : p.hs <= 64 ? launch_lanes<3>(p, s)
           : p.hs <= 128 ? launch_lanes<4>(p, s) : p.hs <= 256 ? launch_lanes<5>(p, s) : launch_lanes<6>(p, s);
}

}  // namespace gcache
