// attention_kv.hip -- attention over the per-head NVFP4 K/V cache: the
// few-rows kernel for its head sizes, and the kernel for many query rows.
// Which one runs is plan_attention's choice.
#include "attention_few.h"

namespace gcache {

// ---------------------------------------------------------------------------
// Many query rows: four waves with 32 rows each and one stream of keys.  A
// 64-key step's operands are dequantized once, a quarter by each wave, into
// LDS in the exact register order of the matrix instruction (1 KiB a
// fragment, lane l at 16 l: conflict-free 16-byte reads and writes), double
// buffered: step i is multiplied while step i + 1 is converted and step
// i + 2's bytes are in flight.  (With every wave dequantizing for itself the
// converters were more than half of the vector instructions.)
// Bound by instruction issue: a wave's step is about 300 vector instructions
// beside 32 or 64 matrix ones, and 32 exponentials at a quarter of the rate.
// Causal prefill of 4 x 2048 tokens over 4096 keys, 32 heads of 128, group 4:
// 510 us, 809 TFLOP/s of the 1377 that a large f16 product reaches.
// ---------------------------------------------------------------------------
constexpr int kStepKeys = 64, kRowsWaves = 4, kRowsTile = 128;

template <int DP>
struct Share {
    static constexpr int KS = DP / 32, DT = DP / 16;
    static constexpr int KF = 4 * KS;                    // K fragments of a step
    static constexpr int VF = 2 * DT;                    // V fragments of a step
    static constexpr int HT = DT / 2;                    // V dim tiles a wave converts
    uint32_t k[DP / 32];                                 // raw: one key of 16
    uint32_t ks;
    uint32_t v[8];                                       // raw: HT codes of eight keys
    uint32_t vs[8];
};

template <int DP, bool UNI>
__device__ __forceinline__ void load_share(const AttnParams& p, const KeyPages& pg, const LaneParts<UNI>& lo, int lane, int w,
                                           Share<DP>& r) {
    const int c = lane & 15, g = lane >> 4;
    // wave w: the K rows of keys 16 w .. 16 w + 15; V of keys 32 (w / 2) .. + 31, half w % 2 of the lane's dims
    const int vh = w & 2;                                // V's first group
    const RowBytes gb[2] = {group_bytes<UNI>(p, pg, vh), group_bytes<UNI>(p, pg, vh + 1)};
    const RowBytes kb = UNI ? RowBytes{w & 1 ? gb[1].d : gb[0].d, w & 1 ? gb[1].s : gb[0].s} : row_bytes<UNI>(p, pg, w, c);
    load_k_row<DP, UNI>(p, kb, lo, g, r.k, &r.ks);
    const bool in = UNI || (DP / 16) * c < p.hs;
    const uint32_t half = (w & 1) * (DP / 64);           // bytes: half of the lane's DP / 32
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const RowBytes b = UNI ? gb[j >> 2] : row_bytes<UNI>(p, pg, vh + (j >> 2), 4 * g + (j & 3));
        const uint8_t *vd = b.d + (half + lo.vd[j & 3]), *sv = b.s + lo.vs[j & 3];
        if (DP == 64) r.v[j] = *vd;
        if (DP == 128) r.v[j] = *reinterpret_cast<const uint16_t*>(vd);
        if (DP == 256) r.v[j] = *reinterpret_cast<const uint32_t*>(vd);
        const uint32_t x = *sv;
        r.vs[j] = in ? x : 0u;
    }
}

template <int DP>
__device__ __forceinline__ void convert_share(const Share<DP>& r, int lane, int w, f16x8* lds) {
    typedef Share<DP> S;
    const uint32_t x = drop_nan_e4m3x4(r.ks);
    const f16x2 a = e4m3x2_f16<false>(x), b = e4m3x2_f16<true>(x);
    const f16x2 sc[4] = {{a.x, a.x}, {a.y, a.y}, {b.x, b.x}, {b.y, b.y}};
#pragma unroll
    for (int st = 0; st < S::KS; st++) lds[(w * S::KS + st) * kWave + lane] = k_operand(r.k[st], sc[st / 2]);
    f16x2 vsc[4];
    v_scales(r.vs, vsc);
    const PairedCodes pc = pair_codes(r.v);
    f16x8* dst = lds + (S::KF + (w >> 1) * S::DT + (w & 1) * S::HT) * kWave + lane;
    dst[0] = v_operand<0>(pc, vsc);
    dst[kWave] = v_operand<1>(pc, vsc);
    if (S::HT > 2) {
        dst[2 * kWave] = v_operand<2>(pc, vsc);
        dst[3 * kWave] = v_operand<3>(pc, vsc);
    }
    if (S::HT > 4) {
        dst[4 * kWave] = v_operand<4>(pc, vsc);
        dst[5 * kWave] = v_operand<5>(pc, vsc);
        dst[6 * kWave] = v_operand<6>(pc, vsc);
        dst[7 * kWave] = v_operand<7>(pc, vsc);
    }
}

// One tile of up to 64 R rows: wave w takes 16 R of them.
template <int DP, int R, bool UNI, bool TREE>
__device__ __forceinline__ void attend_rows(const AttnParams& p, const RowTile& t, int kvh, int v0, int v1,
                                            f16x8 (*s_frag)[(Share<DP>::KF + Share<DP>::VF) * kWave]) {
    typedef Share<DP> S;
    constexpr int KS = S::KS, DT = S::DT;
    constexpr int kDepth = 4;                            // fragments in flight from LDS

    const int lane = lane_id(), w = wave_id();
    const int c = lane & 15, g = lane >> 4;
    const int32_t* bt_row = p.block_table + (int64_t)t.b * p.bt_stride;
    f16x8 q[R][KS];
    float fac[R];
    int pos[R], tok[R];
#pragma unroll
    for (int r = 0; r < R; r++)
        load_query<DP, false>(p, t, kvh, 16 * (R * w + r), lane, q[r], fac[r], pos[r], tok[r]);
    const bool busy = 16 * R * w < t.rows;               // the other waves of a partly filled tile only convert
    const int row_a = min(t.row0 + 16 * R * w, t.row0 + t.rows - 1);
    const int row_b = min(t.row0 + 16 * R * w + 16 * R - 1, t.row0 + t.rows - 1);
    const int pos_lo = t.ctx + row_a / p.group, pos_hi = t.ctx + row_b / p.group;   // of the wave's rows

    f32x4 o[R][DT];
    // weights are exp2(s + sub), sub = kShift - m (0 before the first visible key); a tile whose largest
    // exponent passes lim moves m
    float m[R], l[R], sub[R], lim[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        m[r] = lim[r] = kNegInf;
        l[r] = sub[r] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; d++) o[r][d] = f32x4{0, 0, 0, 0};
    }
    const LaneParts<UNI> lo = lane_parts<DP, UNI>(p, kvh, lane);
    // Steps of 64 keys: the tiles [v0, v1) are runs of sink tiles and window
    // tiles; a step covers two consecutive tile numbers of one run, or the run's
    // last one alone: then its upper 32 keys are hidden as if their pages did not
    // exist (the mask lv), for the next run may hold them, or another split.
    const auto step_key = [&](int v) { return (v < t.sink_tiles ? v : v - t.sink_tiles + t.win_tile0) * kTileKeys; };
    const auto run_end = [&](int v) { return v < t.sink_tiles ? min(t.sink_tiles, v1) : v1; };
    Share<DP> raw;
    KeyPages pg, pg_n, pg_nn;                            // of this step, the converted one, the loading one
    const auto after = [&](int x) { return min(x + 2, run_end(x)); };
    const auto look_up = [&](int x) { return find_pages<UNI, kStepKeys>(p, bt_row, step_key(x < v1 ? x : v0), lane); };
    int v = v0, vn = v1, vnn = v1;
    if (v < v1) {
        pg = look_up(v);
        vn = after(v);
        pg_n = look_up(vn);
        vnn = vn < v1 ? after(vn) : v1;
        pg_nn = look_up(vnn);
        load_share<DP, UNI>(p, pg, lo, lane, w, raw);
        convert_share<DP>(raw, lane, w, s_frag[0]);
        if (vn < v1) load_share<DP, UNI>(p, pg_n, lo, lane, w, raw);
    }
    __syncthreads();
    for (int buf = 0; v < v1; buf ^= 1) {                // workgroup-uniform
        const int key0 = step_key(v), tiles = after(v) - v;   // one or two tiles
        uint32_t lv = live_keys<UNI, kStepKeys>(p, pg, lane);
        if (tiles == 1) lv &= 0xFF;
        const int vp = vnn < v1 ? after(vnn) : v1;
        if (vn < v1) {
            convert_share<DP>(raw, lane, w, s_frag[buf ^ 1]);
            pg = pg_n;
            pg_n = pg_nn;
            if (vnn < v1) {
                pg_nn = look_up(vp);
                load_share<DP, UNI>(p, pg_n, lo, lane, w, raw);
            }
        }
        const f16x8* fr = s_frag[buf] + lane;
        if (busy) {                                      // wave-uniform
            const bool all = lv == 0xFFFFu && all_seen<TREE>(p, t, pos_lo, pos_hi, key0, kStepKeys);
            f32x4 s[R][4];
#pragma unroll
            for (int r = 0; r < R; r++)
#pragma unroll
                for (int kt = 0; kt < 4; kt++) s[r][kt] = f32x4{0, 0, 0, 0};
            stream_fragments<S::KF, kDepth>(fr, [&](int i, const f16x8& a) {
#pragma unroll
                for (int r = 0; r < R; r++)
                    s[r][i / KS] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[r][i % KS], s[r][i / KS], 0, 0, 0);
            });
#pragma unroll
            for (int r = 0; r < R; r++)
#pragma unroll
                for (int kt = 0; kt < 4; kt++)
#pragma unroll
                    for (int i = 0; i < 4; i++) s[r][kt][i] = __builtin_fmaf(s[r][kt][i], fac[r], sub[r]);
            if (!__all(all)) {
#pragma unroll
                for (int r = 0; r < R; r++) hide<TREE, 4>(p, t, pos[r], tok[r], key0 + 4 * g, lv, s[r]);
            }
            float top[R];
            bool late = false;
#pragma unroll
            for (int r = 0; r < R; r++) {
                top[r] = group_max(fmaxf(max8(s[r][0], s[r][1]), max8(s[r][2], s[r][3])));
                late = late || top[r] > lim[r];
            }
            if (__builtin_expect(__any(late), 0)) {          // wave-uniform, rare after the first tiles
#pragma unroll
                for (int r = 0; r < R; r++) {
                    const float mn = fmaxf(m[r], top[r] - sub[r]);
                    const bool any = mn != kNegInf;
                    const float al = any ? __builtin_amdgcn_exp2f(m[r] - mn) : 1.0f;
                    const float to = any ? kShift - mn : 0.0f, by = to - sub[r];
                    m[r] = mn;
                    sub[r] = to;
                    lim[r] = any ? kShift + kLag : kNegInf;
                    l[r] *= al;
#pragma unroll
                    for (int kt = 0; kt < 4; kt++) s[r][kt] += by;
#pragma unroll
                    for (int d = 0; d < DT; d++) o[r][d] *= al;
                }
            }
            f16x8 pw[R][2];
#pragma unroll
            for (int r = 0; r < R; r++) {
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 16; j++) {
                    const float e = __builtin_amdgcn_exp2f(s[r][j >> 2][j & 3]);
                    sum += e;
                    pw[r][j >> 3][j & 7] = (_Float16)e;
                }
                l[r] += sum;
            }
            stream_fragments<S::VF, kDepth>(fr + S::KF * kWave, [&](int i, const f16x8& a) {
#pragma unroll
                for (int r = 0; r < R; r++)
                    o[r][i % DT] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pw[r][i / DT], o[r][i % DT], 0, 0, 0);
            });
        }
        v = vn;
        vn = vnn;
        vnn = vp;
        if (v >= v1) break;
        __syncthreads();
    }

    // ---- each lane holds 4 runs of DT dims of its row
    const bool partial = p.splits > 1 && t.total > t.chunk;
    const float gv = *p.gscale[1];
#pragma unroll
    for (int r = 0; r < R; r++) {
        const float ll = group_sum(l[r]);
        const int off = 16 * (R * w + r) + c;
        if (off >= t.rows) continue;
        const int row = t.row0 + off, tl = row / p.group, head = kvh * p.group + row - tl * p.group;
        const int64_t id = (int64_t)(t.q0 + tl) * p.hq + head;
        const float scale = partial ? 1.0f : ll == 0.0f ? 0.0f : gv / ll;
        if (g == 0) {
            if (partial) {
                float* ml = p.ws_ml + 2 * ((int64_t)t.split * p.total_q * p.hq + id);
                ml[0] = m[r];
                ml[1] = ll;
            } else if (p.lse) {
                p.lse[(int64_t)(t.q0 + tl) * p.lse_ts + head] =
                    row_lse(m[r], ll);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int dim = (4 * g + i) * DT;
            if (dim >= p.hs) continue;
            if (partial) {
                float* dst = p.ws_o + ((int64_t)t.split * p.total_q * p.hq + id) * p.hs + dim;
#pragma unroll
                for (int d = 0; d < DT; d += 4)
                    *reinterpret_cast<f32x4*>(dst + d) = f32x4{o[r][d][i], o[r][d + 1][i], o[r][d + 2][i], o[r][d + 3][i]};
            } else {
                uint16_t* dst = p.out + (int64_t)(t.q0 + tl) * p.o_ts + (int64_t)head * p.o_hs + dim;
#pragma unroll
                for (int d = 0; d < DT; d += 4)
                    *reinterpret_cast<u32x2*>(dst + d) = u32x2{pack_bf16x2(o[r][d][i] * scale, o[r][d + 1][i] * scale),
                                                               pack_bf16x2(o[r][d + 2][i] * scale, o[r][d + 3][i] * scale)};
            }
        }
    }
}

// Tiles of up to 64 rows (a short request, or a request's last rows) give each
// wave one 16-row tile; the longer ones two, which share each K and V fragment.
// 32 x 16 tokens (64 rows) over 8192 keys: 185 us, against 203 with two row
// tiles for half of the waves, at equal splits; head size 256: 188 against 234.
template <int DP, bool UNI, bool TREE>
__global__ __launch_bounds__(kRowsWaves * kWave, DP <= 128 ? 2 : 1) void k_attention_rows(AttnParams p, int64_t wg0) {
    __shared__ f16x8 s_frag[2][(Share<DP>::KF + Share<DP>::VF) * kWave];
    const int64_t wg = wg0 + blockIdx.x;
    const int64_t per = 8 * (int64_t)p.hk;
    const int rem = (int)(wg % per);
    const int64_t unit = wg / per * 8 + rem % 8;
    const int kvh = rem / 8;
    RowTile t;
    if (!find_tile(p, unit, kRowsTile, t)) return;
    int v0, v1;                                          // 32-key tiles; an even number but for the last split
    if (!key_range(t, v0, v1)) return;
    if (t.rows <= kRowsTile / 2) attend_rows<DP, 1, UNI, TREE>(p, t, kvh, v0, v1, s_frag);
    else attend_rows<DP, 2, UNI, TREE>(p, t, kvh, v0, v1, s_frag);
}

template <int DP>
static hipError_t launch_rows(const AttnParams& p, hipStream_t s) {
    const bool uni = uniform_pages(p) && p.hs == DP;
    return launch_attention_parts(
        p.mask ? (uni ? k_attention_rows<DP, true, true> : k_attention_rows<DP, false, true>)
               : (uni ? k_attention_rows<DP, true, false> : k_attention_rows<DP, false, false>),
        kRowsWaves, kRowsTile, p, s);
}

hipError_t launch_attention_kv(const AttnParams& p, int row_tiles, hipStream_t s) {
    if (p.hs <= 64) return row_tiles == 1 ? launch_few<64, 1>(p, s) : row_tiles == 2 ? launch_few<64, 2>(p, s) : launch_rows<64>(p, s);
    if (p.hs <= 128)
        return row_tiles == 1 ? launch_few<128, 1>(p, s) : row_tiles == 2 ? launch_few<128, 2>(p, s) : launch_rows<128>(p, s);
    return row_tiles == 1 ? launch_few<256, 1>(p, s) : launch_rows<256>(p, s);
}

}  // namespace gcache
