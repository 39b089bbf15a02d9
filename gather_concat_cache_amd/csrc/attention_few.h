// attention_few.h -- attention of few query rows (one token to a few drafted
// ones): the four waves of a workgroup share 16 * R query rows, take every
// fourth 32-key tile of the workgroup's key range straight into registers and
// join through LDS.  Long contexts are bound by memory: each wave has a tile's
// bytes in flight while it works on another, but reads them in pieces of 64
// bytes a key and one byte a scale (64 x 1 token over 8192 keys, 8 kv heads of
// 128: 172 us, 3.5 TB/s; a plain stream of reads reaches 7).  Short ones are
// bound by the chain of dependent loads and the launches (8 tokens over 1029
// keys, split: 11 us, and 4 for the join).
#pragma once

#include <type_traits>

#include "attention_device.h"

namespace gcache {

constexpr int kFewWaves = 4;

// Cache bytes of one 32-key tile as a lane needs them: its quarter of K rows
// lane % 16 and 16 + lane % 16; its DP / 16 dims of eight V rows.
template <int DP>
struct RawK {
    static constexpr int W = DP / 32;                    // data words of a quarter row
    uint32_t k[2][W], s[2];                              // and a word with its DP / 64 scales
};
template <int DP>
struct RawV {
    static constexpr int W = DP > 128 ? DP / 128 : 1;
    uint32_t v[8][W], s[8];
};

// The lane's offsets into a page of its parts of rows, the head's and the
// side's distance among them: 32 bits where uniform_pages() says that they fit,
// else 64 (K and V planes, or head planes, of a whole cache may lie apart).
template <bool UNI>
struct LaneParts {
    typedef std::conditional_t<UNI, uint32_t, uint64_t> offset;
    offset kd, ks, vd[4], vs[4];
    __device__ __forceinline__ void renew() {
        if constexpr (UNI) {
            gcache::renew(kd);
            gcache::renew(ks);
            gcache::renew(vd);
            gcache::renew(vs);
        }
    }
};
// UNI kernels take head sizes of exactly DP and pages of whole 16-key groups,
// so that a group's address is wave-uniform; the others take any head size up
// to DP (dims behind head_size read the row's first bytes with a zero scale)
// and look up every key's page.  The general form on a UNI call: 64 x 1 token
// over 8192 keys 219 us against 172, 16 x 8 74 against 48, prefill 4 x 2048
// 1050 against 510.
template <int DP, bool UNI>
__device__ __forceinline__ LaneParts<UNI> lane_parts(const AttnParams& p, int kvh, int lane) {
    const int c = lane & 15, g = lane >> 4;
    typedef typename LaneParts<UNI>::offset offset;
    const offset hd = (offset)(kvh * p.L.data_head_stride), hs = (offset)(kvh * p.L.scale_head_stride);
    const offset side = (offset)p.L.side_stride;
    const bool in = UNI || (DP / 16) * c < p.hs;
    LaneParts<UNI> o;
    o.kd = hd + data_part<UNI>(p, c, (DP / 8) * g);
    o.ks = hs + scale_part<UNI>(p, c, (DP / 64) * g);
#pragma unroll
    for (int j = 0; j < 4; j++) {
        o.vd[j] = side + hd + data_part<UNI>(p, 4 * g + j, in ? (DP / 32) * c : 0);
        o.vs[j] = side + hs + scale_part<UNI>(p, 4 * g + j, in ? (DP * c) / 256 : 0);
    }
    return o;
}

// One key's quarter row: DP / 32 data words and the DP / 64 scales.
template <int DP, bool UNI>
__device__ __forceinline__ void load_k_row(const AttnParams& p, const RowBytes& b, const LaneParts<UNI>& lo, int g,
                                           uint32_t* k, uint32_t* sc) {
    constexpr int KB = DP / 8;                           // data bytes
    const uint8_t *kd = b.d + lo.kd, *sd = b.s + lo.ks;
    if (UNI) {
        if (KB == 8) {
            const u32x2 w = *reinterpret_cast<const u32x2_a8*>(kd);
            k[0] = w.x;
            k[1] = w.y;
        } else {
#pragma unroll
            for (int u = 0; u < KB / 16; u++) {
                const u32x4 w = *reinterpret_cast<const u32x4_a8*>(kd + 16 * u);
#pragma unroll
                for (int i = 0; i < 4; i++) k[(4 * u + i) % (DP / 32)] = w[i];
            }
        }
        if (DP == 64) sc[0] = *sd;
        if (DP == 128) sc[0] = *reinterpret_cast<const u16_a1*>(sd);
        if (DP == 256) sc[0] = *reinterpret_cast<const u32_a1*>(sd);
    } else {                                             // units of 16 dims
        uint32_t x = 0;
#pragma unroll
        for (int u = 0; u < KB / 8; u++) {
            const bool in = (DP / 4) * g + 16 * u < p.hs;
            const u32x2 w = *reinterpret_cast<const u32x2_a8*>(in ? kd + 8 * u : b.d + lo.kd - KB * g);
            const uint32_t y = in ? sd[u] : 0u;
            x |= y << (8 * u);
            k[2 * u] = w.x;
            k[2 * u + 1] = w.y;
        }
        sc[0] = x;
    }
}

template <int DP, bool UNI>
__device__ __forceinline__ void load_k(const AttnParams& p, const KeyPages& pg, const RowBytes* gb, const LaneParts<UNI>& lo,
                                       int lane, RawK<DP>& r) {
#pragma unroll
    for (int t = 0; t < 2; t++) {
        const RowBytes b = UNI ? gb[t] : row_bytes<UNI>(p, pg, t, lane & 15);
        load_k_row<DP, UNI>(p, b, lo, lane >> 4, r.k[t], &r.s[t]);
    }
}

template <int DP, bool UNI>
__device__ __forceinline__ void load_v(const AttnParams& p, const KeyPages& pg, const RowBytes* gb, const LaneParts<UNI>& lo,
                                       int lane, RawV<DP>& r) {
    const int c = lane & 15, g = lane >> 4;
    const bool in = UNI || (DP / 16) * c < p.hs;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const RowBytes b = UNI ? gb[j >> 2] : row_bytes<UNI>(p, pg, j >> 2, 4 * g + (j & 3));
        const uint8_t *vd = b.d + lo.vd[j & 3], *sd = b.s + lo.vs[j & 3];
        if (DP == 64) r.v[j][0] = *reinterpret_cast<const uint16_t*>(vd);
        if (DP == 128) r.v[j][0] = *reinterpret_cast<const uint32_t*>(vd);
        if (DP == 256) {
            const u32x2 w = *reinterpret_cast<const u32x2_a8*>(vd);
            r.v[j][0] = w.x;
            r.v[j][RawV<DP>::W > 1 ? 1 : 0] = w.y;
        }
        r.s[j] = in ? *sd : 0u;
    }
}

template <int DP, int R, bool UNI, bool TREE>
__global__ __launch_bounds__(kFewWaves * kWave, R * DP <= 128 ? 3 : R * DP <= 256 ? 2 : 1)
void k_attention_few(AttnParams p, int64_t wg0) {
    constexpr int KS = DP / 32;                          // head-dim steps of the first product
    constexpr int DT = DP / 16;                          // 16-dim tiles of the output
    constexpr int DW = DT < 8 ? DT : 8;                  // dims of a V word
    constexpr int RT = 16 * R;
    __shared__ float s_o[kFewWaves][16][16 * DW + 4];
    __shared__ float s_m[kFewWaves][16], s_l[kFewWaves][16];

    // The heads of a (row tile, split) unit read neighbouring bytes of the
    // same tokens: they get workgroup numbers 8 apart, i.e. the same XCD's L2.
    const int64_t wg = wg0 + blockIdx.x;
    const int64_t per = 8 * (int64_t)p.hk;
    const int rem = (int)(wg % per);
    const int64_t unit = wg / per * 8 + rem % 8;
    const int kvh = rem / 8;
    RowTile t;
    if (!find_tile(p, unit, RT, t)) return;
    int v0, v1;                                    // 32-key tiles; an even number but for the last split
    if (!key_range(t, v0, v1)) return;

    const int lane = lane_id(), w = wave_id();
    const int c = lane & 15, g = lane >> 4;
    const int32_t* bt_row = p.block_table + (int64_t)t.b * p.bt_stride;
    const auto tile_key = [&](int v) { return (v < t.sink_tiles ? v : v - t.sink_tiles + t.win_tile0) * kTileKeys; };
    const auto look_up = [&](int v) { return find_pages<UNI, kTileKeys>(p, bt_row, tile_key(v < v1 ? v : v0), lane); };
    LaneParts<UNI> lo = lane_parts<DP, UNI>(p, kvh, lane);

    // Loads return in order: page ids are asked for before the bytes of the
    // tile ahead, so waiting for ids leaves bytes in flight.
    RawK<DP> rk;
    RawV<DP> rv;
    KeyPages pg, pg_next;
    int v = v0 + w;
    if (v < v1) {
        pg = look_up(v);
        pg_next = look_up(v + kFewWaves);
        const RowBytes gb[2] = {group_bytes<UNI>(p, pg, 0), group_bytes<UNI>(p, pg, 1)};
        load_k<DP, UNI>(p, pg, gb, lo, lane, rk);
        load_v<DP, UNI>(p, pg, gb, lo, lane, rv);
    }

    f16x8 q[R][KS];
    float fac[R];
    int pos[R], tok[R];
#pragma unroll
    for (int r = 0; r < R; r++) load_query<DP, false>(p, t, kvh, 16 * r, lane, q[r], fac[r], pos[r], tok[r]);
    const int pos_lo = t.ctx + t.row0 / p.group, pos_hi = t.ctx + (t.row0 + t.rows - 1) / p.group;

    f32x4 o[R][DT];
    float m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        m[r] = kNegInf;
        l[r] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; d++) o[r][d] = f32x4{0, 0, 0, 0};
    }

    for (; v < v1; v += kFewWaves) {
        const bool more = v + kFewWaves < v1;
        lo.renew();
        const int key0 = tile_key(v);
        const uint32_t live = live_keys<UNI, kTileKeys>(p, pg, lane);
        // ---- S^T = K Q^T
        f32x4 s[R][2];
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
#pragma unroll
            for (int r = 0; r < R; r++) s[r][kk] = f32x4{0, 0, 0, 0};
            const uint32_t x = drop_nan_e4m3x4(rk.s[kk]);
            const f16x2 x0 = e4m3x2_f16<false>(x), x1 = e4m3x2_f16<true>(x);
            const f16x2 sc[4] = {{x0.x, x0.x}, {x0.y, x0.y}, {x1.x, x1.x}, {x1.y, x1.y}};
#pragma unroll
            for (int st = 0; st < KS; st++) {
                const f16x8 a = k_operand(rk.k[kk][st], sc[st / 2]);
#pragma unroll
                for (int r = 0; r < R; r++) s[r][kk] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[r][st], s[r][kk], 0, 0, 0);
            }
        }
        // ---- the next tile's K takes the registers just used
        RowBytes gb[2];
        if (more) {
            pg = pg_next;
            pg_next = look_up(v + 2 * kFewWaves);
            gb[0] = group_bytes<UNI>(p, pg, 0);
            gb[1] = group_bytes<UNI>(p, pg, 1);
            load_k<DP, UNI>(p, pg, gb, lo, lane, rk);
        }
        // ---- logits, mask
        const bool all = live == 0xFFu && all_seen<TREE>(p, t, pos_lo, pos_hi, key0, kTileKeys);
#pragma unroll
        for (int r = 0; r < R; r++) {
            s[r][0] *= fac[r];
            s[r][1] *= fac[r];
        }
        if (!__all(all)) {
#pragma unroll
            for (int r = 0; r < R; r++) hide<TREE, 2>(p, t, pos[r], tok[r], key0 + 4 * g, live, s[r]);
        }
        // ---- running maximum; the accumulators follow it with a lag
        float top[R];
        bool late = false;
#pragma unroll
        for (int r = 0; r < R; r++) {
            top[r] = group_max(max8(s[r][0], s[r][1]));
            late = late || top[r] > m[r] + kLag;
        }
        if (__builtin_expect(__any(late), 0)) {          // wave-uniform, rare after the first tiles
#pragma unroll
            for (int r = 0; r < R; r++) {
                const float mn = fmaxf(m[r], top[r]);
                const float al = mn == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m[r] - mn);
                m[r] = mn;
                l[r] *= al;
#pragma unroll
                for (int d = 0; d < DT; d++) o[r][d] *= al;
            }
        }
        f16x8 pw[R];
#pragma unroll
        for (int r = 0; r < R; r++) {
            const float sub = m[r] == kNegInf ? 0.0f : kShift - m[r];
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float e = __builtin_amdgcn_exp2f(s[r][j >> 2][j & 3] + sub);
                sum += e;
                pw[r][j] = (_Float16)e;
            }
            l[r] += sum;
        }
        // ---- O^T += V^T P^T
        f16x2 vsc[4];
        v_scales(rv.s, vsc);
#pragma unroll
        for (int vw = 0; vw < RawV<DP>::W; vw++) {
            uint32_t word[8];
#pragma unroll
            for (int j = 0; j < 8; j++) word[j] = rv.v[j][vw];
            const PairedCodes x = pair_codes(word);
            const auto mul = [&](int d, const f16x8& a) {
#pragma unroll
                for (int r = 0; r < R; r++)
                    o[r][8 * vw + d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pw[r], o[r][8 * vw + d], 0, 0, 0);
            };
            mul(0, v_operand<0>(x, vsc));
            mul(1, v_operand<1>(x, vsc));
            mul(2, v_operand<2>(x, vsc));
            mul(3, v_operand<3>(x, vsc));
            if (DW > 4) {
                mul(4 % DT, v_operand<4>(x, vsc));
                mul(5 % DT, v_operand<5>(x, vsc));
                mul(6 % DT, v_operand<6>(x, vsc));
                mul(7 % DT, v_operand<7>(x, vsc));
            }
        }
        if (more) load_v<DP, UNI>(p, pg, gb, lo, lane, rv);
    }

    // ---- join the four waves, 16 rows and 16 * DW dims at a time
    const bool partial = p.splits > 1 && t.total > t.chunk;
    const float gv = *p.gscale[1];
    const int jr = threadIdx.x >> 4, jc = threadIdx.x & 15;   // the row and dim column this thread writes
#pragma unroll
    for (int r = 0; r < R; r++) {
        const float lw = group_sum(l[r]);
        __syncthreads();
        if (g == 0) {
            s_m[w][c] = m[r];
            s_l[w][c] = lw;
        }
        const bool in = 16 * r + jr < t.rows;
        const int row = in ? t.row0 + 16 * r + jr : t.row0;
        const int tl = row / p.group;
        const int head = kvh * p.group + row - tl * p.group;
        const int64_t token = t.q0 + tl, id = token * p.hq + head;
        float scale = 0.0f, wt[kFewWaves];
#pragma unroll
        for (int ch = 0; ch < DT / DW; ch++) {
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int d = 0; d < DW; d += 4)
                    *reinterpret_cast<f32x4*>(&s_o[w][c][(4 * g + i) * DW + d]) =
                        f32x4{o[r][ch * DW + d][i], o[r][ch * DW + d + 1][i], o[r][ch * DW + d + 2][i],
                              o[r][ch * DW + d + 3][i]};
            __syncthreads();
            if (ch == 0) {
                float mm = kNegInf;
#pragma unroll
                for (int k = 0; k < kFewWaves; k++) mm = fmaxf(mm, s_m[k][jr]);
                float ll = 0.0f;
#pragma unroll
                for (int k = 0; k < kFewWaves; k++) {
                    wt[k] = s_m[k][jr] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(s_m[k][jr] - mm);
                    ll = __builtin_fmaf(wt[k], s_l[k][jr], ll);
                }
                scale = partial ? 1.0f : ll == 0.0f ? 0.0f : gv / ll;
                if (in && jc == 0) {
                    if (partial) {
                        float* ml = p.ws_ml + 2 * ((int64_t)t.split * p.total_q * p.hq + id);
                        ml[0] = mm;
                        ml[1] = ll;
                    } else if (p.lse) {
                        p.lse[token * p.lse_ts + head] = row_lse(mm, ll);
                    }
                }
            }
            float acc[DW];
#pragma unroll
            for (int d = 0; d < DW; d++) acc[d] = 0.0f;
#pragma unroll
            for (int k = 0; k < kFewWaves; k++)
#pragma unroll
                for (int d = 0; d < DW; d++) acc[d] = __builtin_fmaf(wt[k], s_o[k][jr][jc * DW + d], acc[d]);
            const int dim = jc * DT + ch * DW;
            if (in && dim < p.hs) {
                if (partial) {
                    float* dst = p.ws_o + ((int64_t)t.split * p.total_q * p.hq + id) * p.hs + dim;
#pragma unroll
                    for (int d = 0; d < DW; d += 4)
                        *reinterpret_cast<f32x4*>(dst + d) = f32x4{acc[d], acc[d + 1], acc[d + 2], acc[d + 3]};
                } else {
                    uint16_t* dst = p.out + token * p.o_ts + (int64_t)head * p.o_hs + dim;
                    uint32_t pk[DW / 2];
#pragma unroll
                    for (int d = 0; d < DW / 2; d++) pk[d] = pack_bf16x2(acc[2 * d] * scale, acc[2 * d + 1] * scale);
                    if (DW == 8) *reinterpret_cast<u32x4*>(dst) = u32x4{pk[0], pk[1], pk[2 % (DW / 2)], pk[3 % (DW / 2)]};
                    else *reinterpret_cast<u32x2*>(dst) = u32x2{pk[0], pk[1]};
                }
            }
            __syncthreads();
        }
    }
}

template <int DP, int R>
hipError_t launch_few(const AttnParams& p, hipStream_t s) {
    const bool uni = uniform_pages(p) && p.hs == DP;
    return launch_attention_parts(
        p.mask ? (uni ? k_attention_few<DP, R, true, true> : k_attention_few<DP, R, false, true>)
               : (uni ? k_attention_few<DP, R, true, false> : k_attention_few<DP, R, false, false>),
        kFewWaves, 16 * R, p, s);
}

}  // namespace gcache
