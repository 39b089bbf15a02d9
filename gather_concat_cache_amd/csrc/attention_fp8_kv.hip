// attention_fp8_kv.hip -- attention over a paged cache of e4m3 keys and values
// with a scale for each page, side and head.
//
// Mathematics.  A logit is softmax_scale * kscale * q . code.  The value scales
// differ from page to page, so they ride on the weights: with a row's
// m = max over its keys of s_j + log2 vscale_j (log2 units),
//     P_j = exp2(s_j + log2 vscale_j - m),  o = sum P_j code_j / sum P_j / vscale_j,
// which keeps the weights that meet the codes within binary16 whatever the
// scales are.  The scales are constant over the keys of a page, so this costs
// no operation a weight.  Where value scales are so far apart that sum P_j /
// vscale_j would leave binary32 (far_scale()), the row's sum goes on apart, as
// sum exp2(s_j - M) with the maximum M of the logits alone, and
//     o = sum P_j code_j 2^(m - M) / sum exp2(s_j - M).
// Scores are binary32 sums of exact products of binary16 (an e4m3 value is exact
// there, a query row is scaled by a power of two); only the weights are rounded,
// to 11 bits, shifted up so that they stay normal down to 2^-20 of the largest.
#include "attention_tiles.h"

namespace gcache {

// Many query rows.  Bound by instruction issue: e4m3's conversions and the
// exponentials beside the products.  4 x 2048 tokens over 4096 keys, 32 / 8 heads
// of 128: 497 us, 830 TFLOP/s; with 256 dims (a workgroup a CU: registers) 895.
// Other pages than whole 16-key groups look up a page and a scale a key: 620.
template <int DP, bool UNI, bool TREE>
__global__ __launch_bounds__(kTileWaves * kWave, DP <= 128 ? 2 : 1) void k_fp8_rows(AttnParams p, int64_t wg0) {
    __shared__ StepLds<PagedFp8, DP, DP, UNI> lds;
    uint32_t kvh, unit;
    if (!head_and_unit(p, (uint32_t)wg0 + blockIdx.x, kvh, unit)) return;
    RowTile t;
    if (!find_tile<true>(p, unit, kTileRows, t)) return;
    int v0, v1;
    if (!key_range(t, v0, v1)) return;
    attend_tile<PagedFp8, DP, DP, UNI, TREE>(p, t, (int)kvh, v0, v1, lds);
}

template <int DP>
static hipError_t launch_rows(const AttnParams& p, bool uni, hipStream_t s) {
    return launch_parts(p.mask ? (uni ? k_fp8_rows<DP, true, true> : k_fp8_rows<DP, false, true>)
                               : (uni ? k_fp8_rows<DP, true, false> : k_fp8_rows<DP, false, false>),
                        kTileWaves, kTileRows, p, s);
}

// ---------------------------------------------------------------------------
// Few query rows (one token to a few drafted ones): the four waves of a
// workgroup share 16 R rows, take every fourth 32-key tile of the workgroup's
// key range and join through LDS.  Each wave has LDS of its own for two tiles,
// filled straight from memory: the tile ahead is in flight while one is
// multiplied, and a tile's K place is refilled as soon as its scores are done,
// so that nothing waits for another wave and no register holds bytes in flight.
// 16x16x32 products as in attention_device.h; lane group g = l / 16 takes 16
// contiguous dims of a 64-dim piece of a key, two steps of the first product;
// for the second the LDS transpose read gives a lane one dim of the eight keys
// 4 g + i and 16 + 4 g + i, which are its weights'.
// Bound by memory for one token: 64 x 1 over 32768 keys, 8 kv heads of 128,
// 5.65 TB/s (over 8192 keys 4.75, and 5.3 where a page's heads are outermost, so
// that a head's 16 rows are one piece).  Two row tiles a wave (R = 2) read the
// keys once for up to 32 rows, where 128-row tiles would be mostly empty.
// ---------------------------------------------------------------------------
constexpr int kFew = 4;                                  // waves

// V rows: the transpose read of two lane groups takes a chunk of the rows 8 n + i
// and 16 + 8 n + i, i < 8.
template <int NC>
__device__ __forceinline__ int few_value_swizzle(int r) {
    constexpr int W = kWindow<NC>;
    return W == 16 ? (r & 7) | (r >> 1 & 8) : W == 8 ? (r >> 1 & 3) | (r >> 2 & 4) : (r >> 2 & 1) | (r >> 3 & 2);
}
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
// What a wave read from LDS has arrived: its place may be refilled.
__device__ __forceinline__ void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

template <int DP, int R, bool UNI, bool TREE>
__global__ __launch_bounds__(kFew * kWave, DP <= 128 ? 2 : 1) void k_fp8_few(AttnParams p, int64_t wg0) {
    constexpr int KS = DP / 32, DT = DP / 16;            // steps of the first product, 16-dim tiles of the output
    constexpr int NC = DP / 16, LR = kWave / NC, N = kTileKeys / LR;    // chunks of a row, rows of a load, loads of a side
    constexpr int SIDE = kTileKeys * DP;                 // bytes
    constexpr int OROW = DP + 4;
    // Far pages are looked for in every 32-key tile (64 x 1 over 8192 keys 229 us
    // against 235 with a look before the first, 32 requests of 2 to 8 tokens behind
    // a window 70 against 74).  Two row tiles over other pages than whole 16-key
    // groups have no registers for that and look first, with a loop for either
    // answer (16 x 8 tokens, pages of 24, 108 against 117).
    constexpr bool kLook = R > 1 && !UNI;
    static_assert(kFew * 16 * OROW * 4 <= kFew * 4 * SIDE, "the join fits the ring");
    __shared__ __attribute__((aligned(256))) uint8_t s_ring[kFew][4][SIDE];      // K, V of two tiles
    __shared__ float s_m[kFew][16], s_l[kFew][16];
    __shared__ FarSum s_far[kFew][R][kWave];             // in LDS, because few rows ever use it

    // heads of a unit 8 apart: the same XCD
    const uint32_t wg = (uint32_t)wg0 + blockIdx.x, per = 8 * (uint32_t)p.hk, set = wg / per, rem = wg - set * per;
    const int kvh = (int)(rem / 8);
    RowTile t;
    if (!find_tile(p, set * 8 + rem % 8, 16 * R, t)) return;
    int v0, v1;
    if (!key_range(t, v0, v1)) return;

    const int lane = lane_id(), w = wave_id(), c = lane & 15, g = lane >> 4;
    const int32_t* bt_row = p.block_table + (int64_t)t.b * p.bt_stride;
    const auto tile_key = [&](int v) { return (v < t.sink_tiles ? v : v - t.sink_tiles + t.win_tile0) * kTileKeys; };
    const uint32_t ring = lds_address(s_ring[w][0]);

    // Pages of a tile: of its two 16-key groups (UNI), or of the rows of the
    // lane's loads, and of key lane % 32.
    constexpr int IDS = UNI ? 2 : N + 1;
    struct Pages {
        PageAt at[IDS];
    };
    const auto find = [&](int v) {
        const int key0 = tile_key(v < v1 ? v : v0);
        Pages x;
#pragma unroll
        for (int n = 0; n < IDS; n++)
            x.at[n] = find_page<UNI>(p, bt_row, key0 + (UNI ? 16 * n : n < N ? n * LR + lane / NC : lane & 31));
        return x;
    };
    const auto issue = [&](const Pages& x, int slot, int side) {
        const int64_t far = kvh * p.L.data_head_stride + side * p.L.side_stride;
        const uint32_t to = ring + (2 * slot + side) * SIDE;
#pragma unroll
        for (int n = 0; n < N; n++) {
            const int row = n * LR + lane / NC, place = lane % NC;
            const int chunk = place ^ (side ? few_value_swizzle<NC>(row) : key_swizzle<NC>(row));
            if constexpr (UNI) {
                const int half = n * LR / 16;            // loads do not cross groups
                load_lds(to + n * 1024, page_row(p, x.at[half]) + far, (uint32_t)(row - 16 * half) * p.data_token + 16 * chunk);
            } else {
                const uint8_t* zero = reinterpret_cast<const uint8_t*>(&g_zero_chunk);
                load_lds(to + n * 1024, 16 * chunk < p.hs ? page_row(p, x.at[n]) + far + 16 * chunk : zero);
            }
        }
    };
    // the tile's scales: of its groups, or of key lane % 32
    constexpr int SC = UNI ? 2 : 1;
    struct Scales {
        RawScale raw[SC];
        bool live[SC];
    };
    const auto scales = [&](const Pages& x) {
        Scales s;
#pragma unroll
        for (int n = 0; n < SC; n++) {
            const PageAt& at = x.at[UNI ? n : N];
            s.raw[n] = raw_scale<UNI>(p, at, kvh);
            s.live[n] = page_exists(p, at);
        }
        return s;
    };

    int v = v0 + w;
    Pages next;                                          // of the tile two ahead
    Scales sc, sc_next;
    FarLook look;
    if constexpr (kLook) look.find(p, t, kvh, v0, v1);
    if (v < v1) {
        Pages x = find(v);
        next = find(v + kFew);
        sc = scales(x);
        if constexpr (kLook) look.load(p);
        issue(x, 0, 0);
        issue(x, 0, 1);
        if (v + kFew < v1) {
            x = next;
            next = find(v + 2 * kFew);
            sc_next = scales(x);
            issue(x, 1, 0);
            issue(x, 1, 1);
        }
    } else if constexpr (kLook) look.load(p);

    // The rows see a far page: s_far holds their sums then, l does not.
    bool far = false;

    // ---- query rows, the dims as the K reads hold them
    f16x8 q[R][KS];
    float fac[R];
    int pos[R], tok[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        const uint16_t* src = query_row(p, t, kvh, 16 * r, lane, pos[r], tok[r]);
        u32x4 raw[KS];
        float amax = 0.0f;
#pragma unroll
        for (int st = 0; st < KS; st++) {
            const int dim = 64 * (st >> 1) + 16 * g + 8 * (st & 1);
            raw[st] = u32x4{0, 0, 0, 0};
            if (pos_in(t, 16 * r, lane) && dim < p.hs) raw[st] = *reinterpret_cast<const u32x4*>(src + dim);
        }
#pragma unroll
        for (int st = 0; st < KS; st++) amax = row_amax(raw[st], amax);
        const float mul = query_scale(p, group_max(amax), 1.0f, fac[r]);
#pragma unroll
        for (int st = 0; st < KS; st++) q[r][st] = query_operand(raw[st], mul);
    }
    const int pos_lo = t.ctx + t.row0 / p.group, pos_hi = t.ctx + (t.row0 + t.rows - 1) / p.group;

    const uint32_t k_lane = c * DP + ((g ^ key_swizzle<NC>(c)) << 4);
    const int v_row = 4 * g + (c >> 1 & 3) + 16 * (c >> 3);
    const uint32_t v_lane = v_row * DP + (few_value_swizzle<NC>(v_row) << 4) + 8 * (c & 1);

    f32x4 o[R][DT];
    float m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        m[r] = kNegInf;
        l[r] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; d++) o[r][d] = f32x4{0, 0, 0, 0};
    }

    // apart: whether a far page is there, or (without a look) may be
    const auto loop = [&](auto apart) {
        for (int slot = 0; v < v1; v += kFew, slot ^= 1) {
            const bool one = v + kFew < v1, two = v + 2 * kFew < v1;
            const int key0 = tile_key(v);
            const uint32_t k_at = ring + 2 * slot * SIDE + k_lane, v_at = ring + (2 * slot + 1) * SIDE + v_lane;
            if (one) wait_loads<2 * N>();                    // the tile ahead stays in flight
            else wait_loads<0>();
            // ---- S^T = K Q^T
            f32x4 s[R][2];
            u32x4 raw[2][KS / 2];
#pragma unroll
            for (int kt = 0; kt < 2; kt++)
#pragma unroll
                for (int j = 0; j < KS / 2; j++)
                    raw[kt][j] = read_lds<u32x4>(chunk_at<NC>(k_at, 4 * j) + kt * 16 * DP);
#pragma unroll
            for (int kt = 0; kt < 2; kt++) {
#pragma unroll
                for (int r = 0; r < R; r++) s[r][kt] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < KS / 2; j++) {
                    const f16x8 a = fp8_operand(raw[kt][j].x, raw[kt][j].y), b = fp8_operand(raw[kt][j].z, raw[kt][j].w);
#pragma unroll
                    for (int r = 0; r < R; r++) {
                        s[r][kt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[r][2 * j], s[r][kt], 0, 0, 0);
                        s[r][kt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, q[r][2 * j + 1], s[r][kt], 0, 0, 0);
                    }
                }
            }
            // ---- K's place takes the tile two ahead
            Pages x = next;
            Scales sc_two;
            if (two) {
                next = find(v + 3 * kFew);
                sc_two = scales(x);
                reads_done();
                issue(x, slot, 0);
            }
            // ---- logits with the scales of their pages
            uint32_t live;
            float inv[UNI ? 2 : 8];
            bool odd = false;                                // a page of the tile is far
            if constexpr (UNI) {
                live = 0;
#pragma unroll
                for (int kt = 0; kt < 2; kt++) {
                    const PageScale ps = scale_of(sc.raw[kt], sc.live[kt]);
                    odd = odd || (!kLook && far_page(t, sc.raw[kt], sc.live[kt], key0 + 16 * kt));
                    live |= sc.live[kt] ? 0xFu << (4 * kt) : 0u;
                    inv[kt] = ps.inv_v;
#pragma unroll
                    for (int r = 0; r < R; r++) {
                        const float f = fac[r] * ps.k;
#pragma unroll
                        for (int i = 0; i < 4; i++) s[r][kt][i] = __builtin_fmaf(s[r][kt][i], f, ps.log2_v);
                    }
                }
            } else {
                const PageScale ps = scale_of(sc.raw[0], sc.live[0]);
                odd = !kLook && far_page(t, sc.raw[0], sc.live[0], key0 + (lane & 31));
                const uint64_t bits = __ballot(sc.live[0]);
                live = (uint32_t)(bits >> (4 * g) & 0xF) | (uint32_t)(bits >> (16 + 4 * g) & 0xF) << 4;
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const int from = 16 * (j >> 2) + 4 * g + (j & 3);
                    const float ks = __shfl(ps.k, from), lv = __shfl(ps.log2_v, from);
                    inv[j] = __shfl(ps.inv_v, from);
#pragma unroll
                    for (int r = 0; r < R; r++) s[r][j >> 2][j & 3] = __builtin_fmaf(s[r][j >> 2][j & 3], fac[r] * ks, lv);
                }
            }
            const bool all = __all(live == 0xFFu && all_seen<TREE>(p, t, pos_lo, pos_hi, key0, kTileKeys));
            if (!all) {
#pragma unroll
                for (int r = 0; r < R; r++) hide<TREE, 2>(p, t, pos[r], tok[r], key0 + 4 * g, live, s[r]);
            }
            // ---- running maximum; the accumulators follow it with a lag
            float top[R];
            bool late = apart.value && (far || odd);
#pragma unroll
            for (int r = 0; r < R; r++) {
                top[r] = group_max(max8(s[r][0], s[r][1]));
                late = late || top[r] > m[r] + kLag;
            }
            if (__builtin_expect(__any(late), 0)) {          // wave-uniform, rare after the first tiles
                const bool now = apart.value && (far || __any(odd));
#pragma unroll
                for (int r = 0; r < R; r++) {
                    FarSum fs{m[r], l[r]};               // (before a large scale's m flushes l; l holds the tiles before)
                    const float mn = fmaxf(m[r], top[r]);
                    const float al = mn == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m[r] - mn);
                    m[r] = mn;
                    l[r] *= al;
#pragma unroll
                    for (int d = 0; d < DT; d++) o[r][d] *= al;
                    if (now) {
                        if (far) fs = s_far[w][r][lane];
                        const auto logit = [&](int j) { return s[r][j >> 2][j & 3] + __builtin_log2f(inv[UNI ? j >> 2 : j]); };
                        float most = kNegInf;
#pragma unroll
                        for (int j = 0; j < 8; j++) most = fmaxf(most, logit(j));
                        far_add<8>(fs, group_max(most), kShift, logit);
                        s_far[w][r][lane] = fs;
                    }
                }
                far = now;
            }
            f16x8 pw[R];
#pragma unroll
            for (int r = 0; r < R; r++) {
                const float sub = m[r] == kNegInf ? 0.0f : kShift - m[r];
#pragma unroll
                for (int kt = 0; kt < 2; kt++) {
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const float e = __builtin_amdgcn_exp2f(s[r][kt][i] + sub);
                        if constexpr (UNI) sum += e;
                        else sum = __builtin_fmaf(e, inv[4 * kt + i], sum);
                        pw[r][4 * kt + i] = (_Float16)e;
                    }
                    l[r] = UNI ? __builtin_fmaf(sum, inv[UNI ? kt : 0], l[r]) : l[r] + sum;
                }
            }
            // ---- O^T += V^T P^T
            const auto multiply = [&](auto fix) {
                u32x2 vr[DT];
#pragma unroll
                for (int d = 0; d < DT; d++)
                    vr[d] = __builtin_bit_cast(u32x2, read_transposed8(chunk_at<NC>(v_at, d)));
#pragma unroll
                for (int d = 0; d < DT; d++) {
                    const f16x8 a = fp8_operand(fix(vr[d].x), fix(vr[d].y));
#pragma unroll
                    for (int r = 0; r < R; r++) o[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pw[r], o[r][d], 0, 0, 0);
                }
            };
            if (all) multiply([](uint32_t x) { return x; });
            else multiply([](uint32_t x) { return drop_nan_e4m3x4(x); });    // hidden codes may be NaN
            if (two) {
                reads_done();
                issue(x, slot, 1);
            }
            sc = sc_next;
            if (two) sc_next = sc_two;
        }
    };
    if constexpr (kLook) {
        far = __syncthreads_or(look.far(p));
        if (far) {
#pragma unroll
            for (int r = 0; r < R; r++) s_far[w][r][lane] = FarSum{kNegInf, 0.0f};
        }
    }
    if (!kLook || far) loop(std::true_type{});
    else loop(std::false_type{});

    // ---- join the four waves, 16 rows at a time
    float* s_o = reinterpret_cast<float*>(&s_ring[0][0][0]);
    const bool partial = p.splits > 1 && t.total > t.chunk;
    const int jr = threadIdx.x >> 4, jc = threadIdx.x & 15;   // the row and dim column this thread writes
#pragma unroll
    for (int r = 0; r < R; r++) {
        float lw = group_sum(l[r]);
        if (__builtin_expect(far, 0)) {
            const FarSum fs = s_far[w][r][lane];
            lw = group_sum(fs.l);
            const float mean = far_end(fs, m[r], lw);
#pragma unroll
            for (int d = 0; d < DT; d++) o[r][d] *= mean;
        }
        __syncthreads();                                 // the other waves' reads of the ring, or of the last rows
        if (g == 0) {
            s_m[w][c] = m[r];
            s_l[w][c] = lw;
        }
#pragma unroll
        for (int d = 0; d < DT; d++) *reinterpret_cast<f32x4*>(s_o + (w * 16 + c) * OROW + 16 * d + 4 * g) = o[r][d];
        __syncthreads();
        const bool in = 16 * r + jr < t.rows;
        const int row = in ? t.row0 + 16 * r + jr : t.row0;
        const int tl = row / p.group, head = kvh * p.group + row - tl * p.group;
        const int64_t token = t.q0 + tl, id = token * p.hq + head;
        float mm = kNegInf, ll = 0.0f, wt[kFew];
#pragma unroll
        for (int k = 0; k < kFew; k++) mm = fmaxf(mm, s_m[k][jr]);
#pragma unroll
        for (int k = 0; k < kFew; k++) {
            wt[k] = s_m[k][jr] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(s_m[k][jr] - mm);
            ll = __builtin_fmaf(wt[k], s_l[k][jr], ll);
        }
        const RowEnd end = row_end(p, token, head, mm, ll, 1.0f);
        if (in && jc == 0) {
            if (partial) {
                float* ml = p.ws_ml + 2 * ((int64_t)t.split * p.total_q * p.hq + id);
                ml[0] = mm;
                ml[1] = ll;
            } else if (p.lse) p.lse[token * p.lse_ts + head] = end.lse;
        }
#pragma unroll
        for (int d = 0; d < DP / 64; d++) {
            const int dim = 64 * d + 4 * jc;
            f32x4 acc = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < kFew; k++) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(s_o + (k * 16 + jr) * OROW + dim);
#pragma unroll
                for (int i = 0; i < 4; i++) acc[i] = __builtin_fmaf(wt[k], x[i], acc[i]);
            }
            if (!in || dim >= p.hs) continue;
            if (partial) *reinterpret_cast<f32x4*>(p.ws_o + ((int64_t)t.split * p.total_q * p.hq + id) * p.hs + dim) = acc;
            else write_dims(p, end, p.out + token * p.o_ts + (int64_t)head * p.o_hs + dim, acc[0], acc[1], acc[2], acc[3]);
        }
    }
}

template <int DP, int R>
static hipError_t launch_few(const AttnParams& p, bool uni, hipStream_t s) {
    return launch_parts(p.mask ? (uni ? k_fp8_few<DP, R, true, true> : k_fp8_few<DP, R, false, true>)
                               : (uni ? k_fp8_few<DP, R, true, false> : k_fp8_few<DP, R, false, false>),
                        kFew, 16 * R, p, s);
}

// Pages of whole 16-key groups whose rows are within 32 bits of each other, and
// a head size that is a form's own.
static bool uniform_fp8(const AttnParams& p, int dp) {
    return p.hs == dp && p.div.size % 16 == 0 && p.L.data_token_stride < (int64_t(1) << 26);
}

hipError_t launch_attention_fp8(const AttnParams& p, int row_tiles, hipStream_t s) {
    const int dp = p.hs <= 64 ? 64 : p.hs <= 128 ? 128 : 256;
    const bool uni = uniform_fp8(p, dp);
    if (dp == 64) return row_tiles == 1 ? launch_few<64, 1>(p, uni, s) : row_tiles == 2 ? launch_few<64, 2>(p, uni, s) : launch_rows<64>(p, uni, s);
    if (dp == 128)
        return row_tiles == 1 ? launch_few<128, 1>(p, uni, s) : row_tiles == 2 ? launch_few<128, 2>(p, uni, s) : launch_rows<128>(p, uni, s);
    return row_tiles == 1 ? launch_few<256, 1>(p, uni, s) : launch_rows<256>(p, uni, s);
}

AttnPlan plan_attention_fp8(int64_t total_q, int32_t batch, int32_t hq, int32_t hk, int32_t hs, int64_t max_seq_len,
                            int32_t window, int32_t sinks, int64_t ws_floats_avail) {
    const int64_t mean = (total_q * (hq / hk) + batch - 1) / batch;      // rows of a request and kv head
    const int row_tiles = mean <= 16 || (hs > 128 && mean <= 32) ? 1 : mean <= 32 ? 2 : kTileRows / 16;
    const int64_t slots = 256 * (hs <= 128 ? 2 : 1);
    return plan_attention_rows(row_tiles, slots, total_q, batch, hq, hk, hs, max_seq_len, window, sinks, ws_floats_avail);
}

}  // namespace gcache
