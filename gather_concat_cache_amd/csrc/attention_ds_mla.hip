// attention_ds_mla.hip -- tree attention over the nvfp4_ds_mla cache in
// absorbed form (scores over 576 values of an entry, values are its first
// 512): the kernel for few query rows, and the one for many.
#include "attention_device.h"

namespace gcache {

// ---------------------------------------------------------------------------
// Many query rows over the latent cache: eight waves and 64 rows.  A row's
// output alone is 512 values, so the two products are split differently.
//   Scores: wave (rt, kt) multiplies row tile rt with key tile kt of a 32-key
//   step; the step's 36 K fragments are dequantized once into LDS (36 KiB,
//   double buffered).
//   Weights: written to LDS as the second product's operand.
//   Values: wave w multiplies all 64 rows' weights with dims 64 w .. 64 w + 63,
//   whose codes only it dequantizes, in registers.
// One barrier a step: K(n + 1) and the weights of step n are written before it,
// the values of step n and the scores of step n + 1 come after it.  All waves
// hold every row's running maximum; a wave that finds a score kLag above it
// raises a flag before the barrier, and the workgroup then agrees on the new
// maxima and writes the weights again (two more barriers, rare).
// Bound by instruction issue around the two products, about 230 registers a lane
// (Q 72, O 64, raw bytes and operands) allowing one workgroup a CU: 32 x 32
// tokens of 16 heads over 8192 keys 433 us, 675 TFLOP/s.  (Running the values of
// a step between the scores of the next took 5 per cent longer.)
// ---------------------------------------------------------------------------
constexpr int kLatentWaves = 8, kLatentRows = 64;
constexpr int kLatentFrags = 36;                         // K fragments of a step: 2 key tiles x 18

struct LatentK {                                         // raw K of wave w: tile w % 2, steps 4 (w / 2) .. + 3
    u32x4 k;
    uint32_t ks;
    u32x2 rope;                                          // waves 0..3: RoPE step w / 2
};
struct LatentV {
    uint32_t v[8], s[8];
};

template <bool UNI>
__device__ __forceinline__ void load_latent_k(const AttnParams& p, const KeyPages& pg, uint32_t kd, uint32_t ks, uint32_t rope,
                                              int lane, int w, LatentK& r) {
    const RowBytes b = row_bytes<UNI>(p, pg, w & 1, lane & 15);
    r.k = *reinterpret_cast<const u32x4*>(b.d + kd);
    r.ks = *reinterpret_cast<const uint16_t*>(b.s + ks);
    if (w < 4) r.rope = *reinterpret_cast<const u32x2*>(b.d + rope);
}
template <bool UNI>
__device__ __forceinline__ void load_latent_v(const AttnParams& p, const KeyPages& pg, const uint32_t* vd, const uint32_t* vs,
                                              int lane, LatentV& r) {
    const RowBytes gb[2] = {group_bytes<UNI>(p, pg, 0), group_bytes<UNI>(p, pg, 1)};
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const RowBytes b = UNI ? gb[j >> 2] : row_bytes<UNI>(p, pg, j >> 2, 4 * (lane >> 4) + (j & 3));
        r.v[j] = *reinterpret_cast<const uint16_t*>(b.d + vd[j & 3]);
        r.s[j] = b.s[vs[j & 3]];
    }
}
__device__ __forceinline__ void convert_latent_k(const LatentK& r, int lane, int w, f16x8* lds) {
    const f16x2 s2 = e4m3x2_f16<false>(drop_nan_e4m3x4(r.ks));
    const f16x2 sc[2] = {{s2.x, s2.x}, {s2.y, s2.y}};
    f16x8* dst = lds + ((w & 1) * 18 + 4 * (w >> 1)) * kWave + lane;
#pragma unroll
    for (int i = 0; i < 4; i++) dst[i * kWave] = k_operand(r.k[i], sc[i / 2]);
    if (w < 4) lds[((w & 1) * 18 + 16 + (w >> 1)) * kWave + lane] = rope_operand(r.rope.x, r.rope.y);
}

template <bool UNI, bool TREE>
__global__ __launch_bounds__(kLatentWaves * kWave, 2) void k_attention_latent(AttnParams p, int64_t wg0) {
    constexpr int KF = 18;                               // K fragments of a key tile
    __shared__ f16x8 s_k[2][kLatentFrags * kWave];
    __shared__ f16x4 s_p[2][4][kWave][2];                // weights: row tile, lane, key tile
    __shared__ float s_top[2][4][16], s_l[2][4][16];
    __shared__ int s_flag[3];

    const int64_t unit = wg0 + blockIdx.x;
    RowTile t;
    if (!find_tile(p, unit, kLatentRows, t)) return;
    int v0, v1;
    if (!key_range(t, v0, v1)) return;

    const int lane = lane_id(), w = wave_id();
    const int c = lane & 15, g = lane >> 4;
    const int kt = w & 1, rt = w >> 1;
    const int32_t* bt_row = p.block_table + (int64_t)t.b * p.bt_stride;
    f16x8 q[KF];
    float fac;
    int pos, tok;
    load_query<512, true>(p, t, 0, 16 * rt, lane, q, fac, pos, tok);
    const int row_a = min(t.row0 + 16 * rt, t.row0 + t.rows - 1), row_b = min(t.row0 + 16 * rt + 15, t.row0 + t.rows - 1);
    const int pos_lo = t.ctx + row_a / p.group, pos_hi = t.ctx + row_b / p.group;

    f32x4 o[4][4];
    float m[4], own = kNegInf, l = 0.0f;                 // own: m[rt]
#pragma unroll
    for (int i = 0; i < 4; i++) {
        m[i] = kNegInf;
#pragma unroll
        for (int d = 0; d < 4; d++) o[i][d] = f32x4{0, 0, 0, 0};
    }
    if (threadIdx.x < 3) s_flag[threadIdx.x] = 0;
    const auto look_up = [&](int x) { return find_pages<UNI, kTileKeys>(p, bt_row, (x < v1 ? x : v0) * kTileKeys, lane); };
    // the lane's parts of its K row, and of its V rows
    uint32_t kd = data_part<UNI>(p, c, 64 * g + 16 * (w >> 1)), ks = scale_part<UNI>(p, c, 8 * g + 2 * (w >> 1));
    uint32_t rope = data_part<UNI>(p, c, kNvRopeOff + 16 * g + 8 * (w >> 1));
    uint32_t vd[4], vs[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        vd[j] = data_part<UNI>(p, 4 * g + j, 32 * w + 2 * c);
        vs[j] = scale_part<UNI>(p, 4 * g + j, 4 * w + (c >> 2));
    }
    LatentK rk;
    LatentV rv;
    KeyPages pg0, pg1, pg2;                              // of steps v, v + 1, v + 2
    if (v0 < v1) {
        pg0 = look_up(v0);
        pg1 = look_up(v0 + 1);
        pg2 = look_up(v0 + 2);
        load_latent_k<UNI>(p, pg0, kd, ks, rope, lane, w, rk);
        convert_latent_k(rk, lane, w, s_k[0]);
        load_latent_k<UNI>(p, pg1, kd, ks, rope, lane, w, rk);
        load_latent_v<UNI>(p, pg0, vd, vs, lane, rv);
    }
    __syncthreads();
    for (int v = v0, n = 0, f = 0; v < v1; v++, n ^= 1, f = f == 2 ? 0 : f + 1) {
        if (UNI) {
            renew(kd);
            renew(ks);
            renew(rope);
            renew(vd);
            renew(vs);
        }
        // ---- scores of step v, K of step v + 1
        const uint32_t live = live_keys<UNI, kTileKeys>(p, pg0, lane) >> (4 * kt) & 0xF;
        f32x4 s = {0, 0, 0, 0};
        stream_fragments<KF, 4>(s_k[n] + kt * KF * kWave + lane,
                                [&](int i, const f16x8& a) { s = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[i], s, 0, 0, 0); });
        convert_latent_k(rk, lane, w, s_k[n ^ 1]);       // (behind the last step: page 0 of the row again, unused)
        pg0 = pg1;
        pg1 = pg2;
        pg2 = look_up(v + 3);
        load_latent_k<UNI>(p, pg1, kd, ks, rope, lane, w, rk);
        const int key0 = v * kTileKeys + 16 * kt;
        s *= fac;
        if (!(live == 0xF && all_seen<TREE>(p, t, pos_lo, pos_hi, key0, 16)) || !UNI)
            hide<TREE, 1>(p, t, pos, tok, key0 + 4 * g, live, &s);
        float top = group_max(fmaxf(max3(s[0], s[1], s[2]), s[3]));
        if (__any(top > own + kLag) && lane == 0) s_flag[f] = 1;
        f32x4 e;
        const auto weigh = [&]() {
            const float sub = own == kNegInf ? 0.0f : kShift - own;
#pragma unroll
            for (int i = 0; i < 4; i++) e[i] = __builtin_amdgcn_exp2f(s[i] + sub);
            s_p[n][rt][lane][kt] = f16x4{(_Float16)e[0], (_Float16)e[1], (_Float16)e[2], (_Float16)e[3]};
        };
        weigh();
        __syncthreads();
        if (__builtin_expect(s_flag[f] != 0, 0)) {       // workgroup-uniform
            if (g == 0) s_top[kt][rt][c] = top;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float mn = fmaxf(m[i], fmaxf(s_top[0][i][c], s_top[1][i][c]));
                const float al = mn == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m[i] - mn);
                m[i] = mn;
                if (i == rt) {
                    l *= al;
                    own = mn;
                }
#pragma unroll
                for (int d = 0; d < 4; d++) o[i][d] *= al;
            }
            weigh();
            __syncthreads();
        }
        // step v + 2 uses this flag's place; nobody has passed the barrier before that yet
        if (threadIdx.x == 0) s_flag[f == 0 ? 2 : f - 1] = 0;
        l += (e[0] + e[1]) + (e[2] + e[3]);

        // ---- values of step v
        f16x2 vsc[4];
        v_scales(rv.s, vsc);
        const PairedCodes x = pair_codes(rv.v);
        load_latent_v<UNI>(p, pg0, vd, vs, lane, rv);         // of step v + 1
        f16x8 pw[4];
#pragma unroll
        for (int i = 0; i < 4; i++) pw[i] = *reinterpret_cast<const f16x8*>(&s_p[n][i][lane][0]);
        const auto mul = [&](int d, const f16x8& a) {
#pragma unroll
            for (int i = 0; i < 4; i++) o[i][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pw[i], o[i][d], 0, 0, 0);
        };
        mul(0, v_operand<0>(x, vsc));
        mul(1, v_operand<1>(x, vsc));
        mul(2, v_operand<2>(x, vsc));
        mul(3, v_operand<3>(x, vsc));
    }

    // ---- sums of the key tiles' waves, then each wave writes its 64 dims of every row
    l = group_sum(l);
    if (g == 0) s_l[kt][rt][c] = l;
    __syncthreads();
    const bool partial = p.splits > 1 && t.total > t.chunk;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int off = 16 * i + c;
        if (off >= t.rows) continue;
        const float ll = s_l[0][i][c] + s_l[1][i][c];
        const int row = t.row0 + off, tl = row / p.group, head = row - tl * p.group;
        const int64_t id = (int64_t)(t.q0 + tl) * p.hq + head;
        const float scale = partial ? 1.0f : ll == 0.0f ? 0.0f : 1.0f / ll;
        if (g == 0 && w == i) {
            if (partial) {
                float* ml = p.ws_ml + 2 * ((int64_t)t.split * p.total_q * p.hq + id);
                ml[0] = m[i];
                ml[1] = ll;
            } else if (p.lse) {
                p.lse[(int64_t)(t.q0 + tl) * p.lse_ts + head] =
                    row_lse(m[i], ll);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int dim = 64 * w + 4 * (4 * g + j);
            const f32x4 x = {o[i][0][j], o[i][1][j], o[i][2][j], o[i][3][j]};
            if (partial) {
                *reinterpret_cast<f32x4*>(p.ws_o + ((int64_t)t.split * p.total_q * p.hq + id) * kNope + dim) = x;
            } else {
                *reinterpret_cast<u32x2*>(p.out + (int64_t)(t.q0 + tl) * p.o_ts + (int64_t)head * p.o_hs + dim) =
                    u32x2{pack_bf16x2(x[0] * scale, x[1] * scale), pack_bf16x2(x[2] * scale, x[3] * scale)};
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Few query rows over the latent cache: four waves and 16 rows.  In a step of
// 64 keys wave w multiplies the rows with keys 16 w .. 16 w + 15; the four
// waves agree on the rows' maxima and leave the weights in LDS; wave w then
// adds dims 128 w .. 128 w + 127 of all 64 keys.  A wave so holds 32
// accumulator registers instead of 128, and two workgroups fit a CU: one's
// loads and barriers pass under the other's conversions.  128 x 1 token of 16
// heads over 8192 keys: 116 us, 3.2 TB/s of the 7 that a plain stream of reads
// reaches; beside the loads, in pieces of 16 bytes down to one, the conversions
// of 1088 values for 352 bytes.  (Waves with 32 keys each for themselves, as in
// the per-head form, took 11 per cent longer.)  The query is converted once,
// a quarter of its fragments by each wave: 2 us less for a single short call.
// ---------------------------------------------------------------------------
constexpr int kTokenWaves = 4, kTokenKeys = 16 * kTokenWaves;

template <bool UNI, bool TREE>
__global__ __launch_bounds__(kTokenWaves * kWave, 2) void k_attention_latent_token(AttnParams p, int64_t wg0) {
    constexpr int KF = 18;                               // K fragments of a key tile
    __shared__ f16x4 s_p[kTokenKeys / kTileKeys][kWave][2];   // weights: tile, lane, half
    __shared__ float s_top[kTokenWaves][16], s_l[kTokenWaves][16];
    __shared__ f16x8 s_q[KF * kWave];

    const int64_t unit = wg0 + blockIdx.x;
    RowTile t;
    if (!find_tile(p, unit, 16, t)) return;
    int t0, t1;                                    // 32-key tiles; an even number but for the last split
    if (!key_range(t, t0, t1)) return;
    const int v0 = t0 / 2, v1 = t1 / 2 + (t1 & 1);       // (keys behind an odd last tile are hidden from every row)

    const int lane = lane_id(), w = wave_id();
    const int c = lane & 15, g = lane >> 4;
    const int32_t* bt_row = p.block_table + (int64_t)t.b * p.bt_stride;
    const auto look_up = [&](int x) { return find_pages<UNI, kTokenKeys>(p, bt_row, (x < v1 ? x : v0) * kTokenKeys, lane); };
    // the lane's parts of its K row, and of its V rows: dims 128 w + 8 c .. + 7
    uint32_t kd = data_part<UNI>(p, c, 64 * g), ks = scale_part<UNI>(p, c, 8 * g);
    uint32_t rope = data_part<UNI>(p, c, kNvRopeOff + 16 * g);
    uint32_t vd[4], vs[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        vd[j] = data_part<UNI>(p, 4 * g + j, 64 * w + 4 * c);
        vs[j] = scale_part<UNI>(p, 4 * g + j, 8 * w + (c >> 1));
    }
    u32x4 rk[5];                                         // raw K: data, RoPE
    u32x2 rs;
    uint32_t rv[2][8], vsb[2][8];                        // raw V, scale bytes
    const auto load_k = [&](const KeyPages& pg) {
        const RowBytes b = row_bytes<UNI>(p, pg, w, c);
#pragma unroll
        for (int i = 0; i < 4; i++) rk[i] = *reinterpret_cast<const u32x4*>(b.d + kd + 16 * i);
        rs = *reinterpret_cast<const u32x2*>(b.s + ks);
        rk[4] = *reinterpret_cast<const u32x4*>(b.d + rope);
    };
    const auto load_v = [&](const KeyPages& pg) {
#pragma unroll
        for (int x = 0; x < 2; x++) {
            const RowBytes gb[2] = {group_bytes<UNI>(p, pg, 2 * x), group_bytes<UNI>(p, pg, 2 * x + 1)};
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const RowBytes b = UNI ? gb[j >> 2] : row_bytes<UNI>(p, pg, 2 * x + (j >> 2), 4 * g + (j & 3));
                rv[x][j] = *reinterpret_cast<const uint32_t*>(b.d + vd[j & 3]);
                vsb[x][j] = b.s[vs[j & 3]];
            }
        }
    };
    KeyPages pg, pg_next;
    if (v0 < v1) {
        pg = look_up(v0);
        pg_next = look_up(v0 + 1);
        load_k(pg);
        load_v(pg);
    }
    // every wave converts some of the query's fragments, all read them back
    f16x8 q[KF];
    float fac;
    int pos, tok;
    {
        constexpr int OWN = (KF + kTokenWaves - 1) / kTokenWaves;
        u32x4 raw[OWN];
        const uint16_t* src = query_row(p, t, 0, 0, lane, pos, tok);
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < OWN; i++) {
            const int st = min(w + kTokenWaves * i, KF - 1);
            raw[i] = u32x4{0, 0, 0, 0};
            if (pos_in(t, 0, lane)) raw[i] = *reinterpret_cast<const u32x4*>(src + query_dim<512>(st, g));
        }
#pragma unroll
        for (int i = 0; i < OWN; i++) amax = row_amax(raw[i], amax);
        amax = group_max(amax);
        if (g == 0) s_top[w][c] = amax;
        __syncthreads();
        amax = fmaxf(fmaxf(s_top[0][c], s_top[1][c]), fmaxf(s_top[2][c], s_top[3][c]));
        const float mul = query_scale(p, amax, 1.0f, fac);
#pragma unroll
        for (int i = 0; i < OWN; i++) s_q[min(w + kTokenWaves * i, KF - 1) * kWave + lane] = query_operand(raw[i], mul);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KF; i++) q[i] = s_q[i * kWave + lane];
    }
    const int pos_lo = t.ctx + t.row0 / p.group, pos_hi = t.ctx + (t.row0 + t.rows - 1) / p.group;

    f32x4 o[8];
    float m = kNegInf, l = 0.0f;
#pragma unroll
    for (int d = 0; d < 8; d++) o[d] = f32x4{0, 0, 0, 0};

    for (int v = v0; v < v1; v++) {
        if (UNI) {
            renew(kd);
            renew(ks);
            renew(rope);
            renew(vd);
            renew(vs);
        }
        // ---- S^T = K Q^T, two chains
        const uint32_t live = live_keys<UNI, kTokenKeys>(p, pg, lane) >> (4 * w) & 0xF;
        f32x4 s = {0, 0, 0, 0}, s2 = {0, 0, 0, 0};
        f16x2 sc[8];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t x = drop_nan_e4m3x4(rs[i]);
            const f16x2 a = e4m3x2_f16<false>(x), b = e4m3x2_f16<true>(x);
            sc[4 * i] = f16x2{a.x, a.x};
            sc[4 * i + 1] = f16x2{a.y, a.y};
            sc[4 * i + 2] = f16x2{b.x, b.x};
            sc[4 * i + 3] = f16x2{b.y, b.y};
        }
#pragma unroll
        for (int i = 0; i < KF; i++) {
            const f16x8 a = i < 16 ? k_operand(rk[i / 4][i % 4], sc[i / 2 % 8]) : rope_operand(rk[4][2 * (i % 2)], rk[4][2 * (i % 2) + 1]);
            f32x4& acc = i & 1 ? s2 : s;
            acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[i], acc, 0, 0, 0);
        }
        // ---- the next step's K takes the registers just used.  (Behind the last: the first step's page, unused.)
        pg = pg_next;
        pg_next = look_up(v + 2);
        load_k(pg);
        const int key0 = v * kTokenKeys + 16 * w;
        s = (s + s2) * fac;
        if (!__all(live == 0xF && all_seen<TREE>(p, t, pos_lo, pos_hi, key0, 16)))
            hide<TREE, 1>(p, t, pos, tok, key0 + 4 * g, live, &s);
        // ---- the waves' common maximum; the accumulators follow it with a lag
        const float top = group_max(fmaxf(max3(s[0], s[1], s[2]), s[3]));
        if (g == 0) s_top[w][c] = top;
        __syncthreads();
        const float mn = fmaxf(fmaxf(fmaxf(m, s_top[0][c]), fmaxf(s_top[1][c], s_top[2][c])), s_top[3][c]);
        if (__builtin_expect(__any(mn > m + kLag), 0)) { // workgroup-uniform
            const float al = mn == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= al;
#pragma unroll
            for (int d = 0; d < 8; d++) o[d] *= al;
        }
        const float sub = m == kNegInf ? 0.0f : kShift - m;
        f32x4 e;
#pragma unroll
        for (int i = 0; i < 4; i++) e[i] = __builtin_amdgcn_exp2f(s[i] + sub);
        s_p[w >> 1][lane][w & 1] = f16x4{(_Float16)e[0], (_Float16)e[1], (_Float16)e[2], (_Float16)e[3]};
        l += (e[0] + e[1]) + (e[2] + e[3]);
        __syncthreads();
        // ---- O^T += V^T P^T
#pragma unroll
        for (int x = 0; x < 2; x++) {
            const f16x8 pw = *reinterpret_cast<const f16x8*>(&s_p[x][lane][0]);
            f16x2 vsc[4];
            v_scales(vsb[x], vsc);
            const PairedCodes y = pair_codes(rv[x]);
            const auto mul = [&](int d, const f16x8& a) { o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pw, o[d], 0, 0, 0); };
            mul(0, v_operand<0>(y, vsc));
            mul(1, v_operand<1>(y, vsc));
            mul(2, v_operand<2>(y, vsc));
            mul(3, v_operand<3>(y, vsc));
            mul(4, v_operand<4>(y, vsc));
            mul(5, v_operand<5>(y, vsc));
            mul(6, v_operand<6>(y, vsc));
            mul(7, v_operand<7>(y, vsc));
        }
        load_v(pg);
    }

    // ---- sums of the waves' keys, then each wave writes its 128 dims of every row
    l = group_sum(l);
    if (g == 0) s_l[w][c] = l;
    __syncthreads();
    if (c >= t.rows) return;
    const bool partial = p.splits > 1 && t.total > t.chunk;
    const float ll = (s_l[0][c] + s_l[1][c]) + (s_l[2][c] + s_l[3][c]);
    const int row = t.row0 + c, tl = row / p.group, head = row - tl * p.group;
    const int64_t id = (int64_t)(t.q0 + tl) * p.hq + head;
    const float scale = partial ? 1.0f : ll == 0.0f ? 0.0f : 1.0f / ll;
    if (g == 0 && w == 0) {
        if (partial) {
            float* ml = p.ws_ml + 2 * ((int64_t)t.split * p.total_q * p.hq + id);
            ml[0] = m;
            ml[1] = ll;
        } else if (p.lse) {
            p.lse[(int64_t)(t.q0 + tl) * p.lse_ts + head] = row_lse(m, ll);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int dim = 128 * w + 8 * (4 * g + j);
        if (partial) {
            float* dst = p.ws_o + ((int64_t)t.split * p.total_q * p.hq + id) * kNope + dim;
            *reinterpret_cast<f32x4*>(dst) = f32x4{o[0][j], o[1][j], o[2][j], o[3][j]};
            *reinterpret_cast<f32x4*>(dst + 4) = f32x4{o[4][j], o[5][j], o[6][j], o[7][j]};
        } else {
            uint32_t pk[4];
#pragma unroll
            for (int d = 0; d < 4; d++) pk[d] = pack_bf16x2(o[2 * d][j] * scale, o[2 * d + 1][j] * scale);
            *reinterpret_cast<u32x4*>(p.out + (int64_t)(t.q0 + tl) * p.o_ts + (int64_t)head * p.o_hs + dim) =
                u32x4{pk[0], pk[1], pk[2], pk[3]};
        }
    }
}

hipError_t launch_attention_ds_mla(const AttnParams& p, int row_tiles, hipStream_t s) {
    const bool uni = uniform_pages(p);
    if (row_tiles == 1)
        return launch_attention_parts(
            p.mask ? (uni ? k_attention_latent_token<true, true> : k_attention_latent_token<false, true>)
                   : (uni ? k_attention_latent_token<true, false> : k_attention_latent_token<false, false>),
            kTokenWaves, 16, p, s);
    return launch_attention_parts(p.mask ? (uni ? k_attention_latent<true, true> : k_attention_latent<false, true>)
                                         : (uni ? k_attention_latent<true, false> : k_attention_latent<false, false>),
                                  kLatentWaves, kLatentRows, p, s);
}

}  // namespace gcache
