// attention_kernels.hip -- attention over the quantized paged caches, read in
// place: the per-head NVFP4 K/V cache (any byte layout) and the 352-byte
// nvfp4_ds_mla entry in absorbed form (all heads share the latent; scores
// over 576 values, values over 512).
//
// Mathematics.  For a query row with logits s_j = scale * q . k_j over its
// visible keys, o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m) for any m.
// One pass over the keys keeps a running m, l = sum exp2(s - m) and
// o = sum exp2(s - m) v in binary32, in units of log2; partial triples
// (m, l, o) of disjoint key sets join by rescaling to the larger m.
//
// Rounding.  An NVFP4 value e2m1 * e4m3 has at most 6 significant bits and a
// magnitude of 2^-10 .. 2688, so it is exact in binary16; the per-tensor
// scales stay outside (in the logit factor and in the output).  A query row
// is scaled by the power of two that puts its largest magnitude in
// [2^10, 2^11) and is then exact in binary16 down to 2^-24 of that maximum.
// So scores are binary32 sums of exact products; only the weights
// exp2(s - m) are rounded, to binary16 (11 bits against bf16's 8, at the same
// matrix rate), shifted up by kShift so that they stay normal numbers down to
// 2^-20 of the largest.  A block scale that holds the e4m3 NaN code (no write
// makes one) counts as 0, so pages that no row sees cannot reach an output.
//
// Mapping.  One wave works on 16 * R query rows (query token x head of the
// group) and 32 keys a step, all in registers:
//   S^T = K Q^T     matrix rows are keys, columns are query rows;
//   O^T = V^T P^T   matrix rows are value dims, columns are query rows.
// The 16x16 result layout (lane: column l % 16, rows 4 (l / 16) + i) makes
// the scores of two 16-key tiles exactly the k-operand of the second product
// when its 8 k-slots of lane group g are taken as keys 4g..4g+3 and
// 16+4g..16+4g+3, so weights never leave their lane, and the row statistics
// are per column, i.e. lane local.  Contraction order over the head dim is
// free, so lane group g takes the contiguous quarter g of a key's row (one
// 16-byte load for 128 dims).  For V, lane column c takes the contiguous
// dims c * DT .. c * DT + DT - 1 of its 8 keys and pairs the codes of two keys
// in one byte with masks and shifts before the converter, which then returns
// exactly the operand's register order.
// The four waves of a workgroup share the query rows, take every fourth
// 32-key tile of the workgroup's key range and join through LDS.
#include "gcache_operators.h"

namespace gcache {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a8 __attribute__((aligned(8)));
typedef u32x2 u32x2_a8 __attribute__((aligned(8)));
typedef uint64_t u64_a1 __attribute__((aligned(1)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef uint16_t u16_a1 __attribute__((aligned(1)));

constexpr int kTileKeys = 32;
constexpr int kAttnWaves = 4;
// log2 units: weights are 2^kShift * exp2(s - m), m trails the true maximum
// by at most kLag before the accumulators are rescaled, so weights stay
// below 2^(kShift + kLag) = 2^14.
constexpr float kShift = 6.0f, kLag = 8.0f;
constexpr float kNegInf = -__builtin_inff();

// Zero every byte of x that holds the e4m3 NaN code (0x7F or 0xFF).
__device__ __forceinline__ uint32_t drop_nan_e4m3x4(uint32_t x) {
    const uint32_t m = ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    return x & ~(m | (m - (m >> 7)));
}
template <bool HI>
__device__ __forceinline__ f16x2 e4m3x2_f16(uint32_t w) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI);
}
template <int SEL>
__device__ __forceinline__ f16x2 e2m1x2_f16(uint32_t w) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, SEL);
}
// Over the four lanes l % 16 + 16 k of a column: the two swap instructions
// exchange rows of 16 (then halves of 32) between two copies of v, so each
// lane holds its own value and its partner's without an LDS round trip.
__device__ __forceinline__ float group_max(float v) {
    const u32x2 a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
    const u32x2 b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b.x), __uint_as_float(b.y));
}
// Largest of 8 (16) logits: three at a time.  The operands come out of
// multiplies, so the plain instruction needs none of the quieting that fmaxf
// adds to each operand; the last step is fmaxf again.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float max8(const f32x4& a, const f32x4& b) {
    return fmaxf(max3(max3(a[0], a[1], a[2]), a[3], b[0]), max3(b[1], b[2], b[3]));
}
__device__ __forceinline__ float group_sum(float v) {
    const u32x2 a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a.x) + __uint_as_float(a.y);
    const u32x2 b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b.x) + __uint_as_float(b.y);
}

// What a workgroup works on, from the device metadata.
struct RowTile {
    int b;                       // request
    int row0, rows;              // first row of the tile in the request, rows in it (<= 16 R)
    int q0;                      // first packed query token of the request
    int qlen, ctx, kv_len;       // ctx = position of the request's first query
    int sink_tiles, win_tile0, total;   // 32-key tiles: [0, sink_tiles) then from win_tile0
};

__device__ __forceinline__ int query_start(const AttnParams& p, int b) {
    const int v = p.qs[b];
    return min(max(v, 0), p.total_q);
}

// Visible 32-key tiles of rows [row0, row0 + rows) of request b.
__device__ __forceinline__ void tile_range(const AttnParams& p, RowTile& t) {
    // key numbers stay clear of int32's end, so key0 + 32 cannot wrap
    const int64_t table_keys =
        p.num_blocks > 0 ? min(p.bt_stride * p.div.size, (int64_t)INT32_MAX - 2 * kTileKeys) : 0;
    const int seq = max(p.seq_lens[t.b], 0);
    t.ctx = seq - t.qlen;        // may be negative: those rows see nothing
    t.kv_len = (int)min((int64_t)seq, table_keys);
    const int p0 = t.ctx + t.row0 / p.group;
    const int p1 = t.ctx + (t.row0 + t.rows - 1) / p.group;
    const int hi = p.mask ? t.kv_len : min(p1 + 1, t.kv_len);
    int lo = 0, sk = 0;
    if (p.window > 0) {
        lo = (int)max((int64_t)0, (int64_t)p0 - p.window + 1);
        sk = min(p.sinks, hi);
    }
    t.win_tile0 = lo / kTileKeys;
    const int end = hi > 0 ? (hi - 1) / kTileKeys + 1 : 0;
    t.sink_tiles = sk > 0 ? min((sk - 1) / kTileKeys + 1, min(t.win_tile0, end)) : 0;
    t.total = p1 < 0 ? 0 : t.sink_tiles + max(0, end - t.win_tile0);
}

// Row tile `tile` of the call: request b owns the tile numbers from
// qs[b] * group / RT + b on, which leaves it at least ceil(rows / RT).
__device__ __forceinline__ bool find_tile(const AttnParams& p, int tile, int RT, RowTile& t) {
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)query_start(p, mid) * p.group / RT + mid <= tile) lo = mid;
        else hi = mid;
    }
    t.b = lo;
    t.q0 = query_start(p, lo);
    t.qlen = query_start(p, lo + 1) - t.q0;
    const int64_t row0 = (tile - ((int64_t)t.q0 * p.group / RT + lo)) * RT;
    const int64_t rows = (int64_t)t.qlen * p.group;
    if (t.qlen <= 0 || row0 < 0 || row0 >= rows) return false;
    t.row0 = (int)row0;
    t.rows = (int)min((int64_t)RT, rows - row0);
    tile_range(p, t);
    return true;
}

// Block and offset of a position; positions are below 2^31.
__device__ __forceinline__ void split_position(const AttnParams& p, int pos, int& blk, int& off) {
    const int size = (int)p.div.size;
    if (p.div.shift >= 0) {
        blk = pos >> p.div.shift;
        off = pos & (size - 1);
    } else {
        blk = (int)((uint32_t)pos / (uint32_t)size);
        off = pos - blk * size;
    }
}

// The block-table entries of KEYS consecutive keys, spread over the lanes.
// UNI: block_size is a multiple of 16, so every 16 keys lie in one page: lane
// i holds the page of keys 16 i .. 16 i + 15, and their bytes are at wave-uniform
// addresses to which a lane adds loop-invariant 32-bit offsets.  Otherwise lane
// i holds key i's page.  The entry is only looked at when it is used (a step
// later), so its load stays in flight.
struct KeyPages {
    int blk;                     // as in the table
    int off;                     // token in the page, -1: behind the table's row
};
template <bool UNI, int KEYS>
__device__ __forceinline__ KeyPages find_pages(const AttnParams& p, const int32_t* __restrict__ bt_row, int key0, int lane) {
    int bi;
    KeyPages g;
    split_position(p, key0 + (UNI ? 16 * (lane & (KEYS / 16 - 1)) : lane & (KEYS - 1)), bi, g.off);
    const bool in = bi < p.bt_stride;
    g.blk = bt_row[in ? bi : 0];
    if (!in) g.off = -1;
    return g;
}
// The page of 16-key group h (UNI) or of key i: block (0 when there is none,
// which is then masked) and token.
template <bool UNI>
__device__ __forceinline__ bool take_page(const AttnParams& p, const KeyPages& g, int h, int i, int& blk, int& off) {
    blk = UNI ? __builtin_amdgcn_readlane(g.blk, h) : __shfl(g.blk, i);
    off = UNI ? __builtin_amdgcn_readlane(g.off, h) : __shfl(g.off, i);
    const bool ok = off >= 0 && (uint32_t)blk < (uint64_t)p.num_blocks;
    blk = ok ? blk : 0;
    off = ok ? off : 0;
    return ok;
}
// Bit 4 h + i: the page of the lane's key 16 h + 4 (lane / 16) + i exists.
template <bool UNI, int KEYS>
__device__ __forceinline__ uint32_t live_keys(const AttnParams& p, const KeyPages& g, int lane) {
    const bool ok = g.off >= 0 && (uint32_t)g.blk < (uint64_t)p.num_blocks;
    const uint64_t bits = __ballot(ok);
    uint32_t live = 0;
#pragma unroll
    for (int h = 0; h < KEYS / 16; h++)
        live |= UNI ? (bits >> h & 1 ? 0xFu << (4 * h) : 0u) : (uint32_t)(bits >> (16 * h + 4 * (lane >> 4)) & 0xF) << (4 * h);
    return live;
}

// A lane's offsets from the first key of a half: its K key (lane % 16) and
// its four V keys (4 (lane / 16) + j), each to the lane's part of the row.
// UNI takes calls whose 16-key span fits 32 bits (the launcher checks).
struct LaneOffsets {
    uint32_t kd, ks, vd[4], vs[4];
};
template <int DP, bool MLA>
__device__ __forceinline__ LaneOffsets lane_offsets(const AttnParams& p, int kvh, int lane) {
    const int c = lane & 15, g = lane >> 4;
    LaneOffsets o;
    const uint32_t tok_d = (uint32_t)p.L.data_token_stride, tok_s = (uint32_t)p.L.scale_token_stride;
    const uint32_t hd = MLA ? 0 : (uint32_t)(kvh * p.L.data_head_stride), hsc = MLA ? 0 : (uint32_t)(kvh * p.L.scale_head_stride);
    const uint32_t side = MLA ? 0 : (uint32_t)p.L.side_stride;
    o.kd = c * tok_d + hd + (DP / 8) * g;
    o.ks = c * tok_s + hsc + (DP / 64) * g;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        o.vd[j] = (4 * g + j) * tok_d + hd + (DP / 32) * c + side;
        o.vs[j] = (4 * g + j) * tok_s + hsc + (DP * c) / 256 + side;
    }
    return o;
}

// First bytes of 16-key group h at wave-uniform addresses (UNI).
struct GroupBytes {
    const uint8_t *d, *s;
};
template <bool UNI, bool MLA>
__device__ __forceinline__ GroupBytes group_bytes(const AttnParams& p, const KeyPages& g, int h) {
    GroupBytes b = {nullptr, nullptr};
    if (UNI) {
        int blk, off;
        take_page<true>(p, g, h, 0, blk, off);
        const uint8_t* page = p.cache + (int64_t)blk * p.L.block_stride;
        b.d = page + (int64_t)off * p.L.data_token_stride + (MLA ? 0 : p.L.data_offset);
        if (!MLA) b.s = page + (int64_t)off * p.L.scale_token_stride + p.L.scale_offset;
    }
    return b;
}
// Where the lane's K key of group h (value == false) or its V key j of it
// reads: the lane's data bytes and scale bytes.
template <int DP, bool MLA, bool UNI>
__device__ __forceinline__ void key_bytes(const AttnParams& p, const KeyPages& g, const GroupBytes& b, const LaneOffsets& o,
                                          int h, bool value, int j, int kvh, int lane, const uint8_t*& d,
                                          const uint8_t*& s) {
    const int c = lane & 15, gr = lane >> 4;
    if (UNI) {
        d = b.d + (value ? o.vd[j] : o.kd);
        s = b.s + (value ? o.vs[j] : o.ks);
    } else {
        int blk, off;
        take_page<false>(p, g, h, 16 * h + (value ? 4 * gr + j : c), blk, off);
        const uint8_t* page = p.cache + (int64_t)blk * p.L.block_stride + (value ? p.L.side_stride : 0);
        d = page + p.L.data_offset + (int64_t)off * p.L.data_token_stride + (int64_t)kvh * p.L.data_head_stride +
            (value ? (DP / 32) * c : (DP / 8) * gr);
        s = page + p.L.scale_offset + (int64_t)off * p.L.scale_token_stride + (int64_t)kvh * p.L.scale_head_stride +
            (value ? (DP * c) / 256 : (DP / 64) * gr);
    }
}

// Raw cache bytes of one 32-key tile as a lane needs them.
template <int DP, bool MLA>
struct Raw {
    static constexpr int KW = DP / 32;                   // data words of the lane's quarter row
    static constexpr int KSW = DP / 256 > 0 ? DP / 256 : 1;  // words holding its DP / 64 scales
    static constexpr int VW = DP / 128 > 0 ? DP / 128 : 1;   // data words of its DP / 16 dims
    uint32_t k[2][KW];
    uint32_t ks[2][KSW];
    uint32_t rope[MLA ? 2 : 1][4];
    uint32_t v[8][VW];
    uint32_t vs[8];
    uint32_t live;               // live_keys()
};

template <int DP, bool MLA, bool UNI>
__device__ __forceinline__ void load_tile(const AttnParams& p, const KeyPages& pg, const LaneOffsets& lo, int kvh, int lane,
                                          Raw<DP, MLA>& r) {
    constexpr int KB = DP / 8;                           // K data bytes per lane and key
    const int c = lane & 15, g = lane >> 4;
    const bool full = MLA || p.hs == DP;
    const GroupBytes gb[2] = {group_bytes<UNI, MLA>(p, pg, 0), group_bytes<UNI, MLA>(p, pg, 1)};
#pragma unroll
    for (int t = 0; t < 2; t++) {
        const uint8_t *kd, *sd;
        key_bytes<DP, MLA, UNI>(p, pg, gb[t], lo, t, false, 0, kvh, lane, kd, sd);
        if (MLA) {
            const uint8_t* e = kd - KB * g;
#pragma unroll
            for (int u = 0; u < KB / 16; u++) {
                const u32x4 w = *reinterpret_cast<const u32x4*>(kd + 16 * u);
#pragma unroll
                for (int i = 0; i < 4; i++) r.k[t][4 * u + i] = w[i];
            }
            const u32x4 w = *reinterpret_cast<const u32x4*>(e + kNvRopeOff + 16 * g);
#pragma unroll
            for (int i = 0; i < 4; i++) r.rope[t][i] = w[i];
            const u32x2 s = *reinterpret_cast<const u32x2*>(e + kNvScaleOff + 8 * g);
            r.ks[t][0] = s.x;
            r.ks[t][1 % Raw<DP, MLA>::KSW] = s.y;
        } else {
            if (full) {
                if (KB == 8) {
                    const u32x2 w = *reinterpret_cast<const u32x2_a8*>(kd);
                    r.k[t][0] = w.x;
                    r.k[t][1] = w.y;
                } else {
#pragma unroll
                    for (int u = 0; u < KB / 16; u++) {
                        const u32x4 w = *reinterpret_cast<const u32x4_a8*>(kd + 16 * u);
#pragma unroll
                        for (int i = 0; i < 4; i++) r.k[t][(4 * u + i) % Raw<DP, MLA>::KW] = w[i];
                    }
                }
                if (DP == 64) r.ks[t][0] = *sd;
                if (DP == 128) r.ks[t][0] = *reinterpret_cast<const u16_a1*>(sd);
                if (DP == 256) r.ks[t][0] = *reinterpret_cast<const u32_a1*>(sd);
            } else {                                     // head_size below DP: units of 16 dims
                r.ks[t][0] = 0;
#pragma unroll
                for (int u = 0; u < KB / 8; u++) {
                    const bool in = (DP / 4) * g + 16 * u < p.hs;
                    u32x2 w = {0, 0};
                    if (in) {
                        w = *reinterpret_cast<const u32x2_a8*>(kd + 8 * u);
                        r.ks[t][0] |= (uint32_t)sd[u] << (8 * u);
                    }
                    r.k[t][2 * u] = w.x;
                    r.k[t][2 * u + 1] = w.y;
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const uint8_t *vd, *sd;
        key_bytes<DP, MLA, UNI>(p, pg, gb[j >> 2], lo, j >> 2, true, j & 3, kvh, lane, vd, sd);
        if (MLA) {
            const uint8_t* e = vd - 16 * c;
            const u32x4 w = *reinterpret_cast<const u32x4*>(vd);
#pragma unroll
            for (int i = 0; i < 4; i++) r.v[j][i % Raw<DP, MLA>::VW] = w[i];
            r.vs[j] = *reinterpret_cast<const uint16_t*>(e + kNvScaleOff + 2 * c);
        } else {
            if (full || (DP / 16) * c < p.hs) {
                if (DP == 64) r.v[j][0] = *reinterpret_cast<const uint16_t*>(vd);
                if (DP == 128) r.v[j][0] = *reinterpret_cast<const uint32_t*>(vd);
                if (DP == 256) {
                    const u32x2 w = *reinterpret_cast<const u32x2_a8*>(vd);
                    r.v[j][0] = w.x;
                    r.v[j][1 % Raw<DP, MLA>::VW] = w.y;
                }
                r.vs[j] = *sd;
            } else {
#pragma unroll
                for (int i = 0; i < Raw<DP, MLA>::VW; i++) r.v[j][i] = 0;
                r.vs[j] = 0;
            }
        }
    }
    r.live = live_keys<UNI, kTileKeys>(p, pg, lane);
}

// One row of queries a column: lane l takes row t.row0 + row_off + l % 16, its
// values as the second operand of S^T = K Q^T, and the factor from scores to
// logits in log2 units.  Rows behind the tile are zeros at position -1.
template <int DP, bool MLA>
__device__ __forceinline__ void load_query(const AttnParams& p, const RowTile& t, int kvh, int row_off, int lane,
                                           f16x8* q, float& fac, int& pos, int& tok) {
    constexpr int KS = DP / 32, RS = MLA ? 2 : 0;
    const int c = lane & 15, g = lane >> 4;
    const bool in = row_off + c < t.rows;
    const int row = in ? t.row0 + row_off + c : t.row0;
    const int tl = row / p.group;
    const int head = kvh * p.group + row - tl * p.group;
    tok = t.q0 + tl;
    pos = in ? t.ctx + tl : -1;
    const uint16_t* src = p.q + (int64_t)tok * p.q_ts + (int64_t)head * p.q_hs;
    u32x4 raw[KS + RS];
    float amax = 0.0f;
#pragma unroll
    for (int s = 0; s < KS + RS; s++) {
        const int dim = s < KS ? (DP / 4) * g + 8 * s : kNope + 16 * g + 8 * (s - KS);
        raw[s] = u32x4{0, 0, 0, 0};
        if (in && (MLA || dim < p.hs)) raw[s] = *reinterpret_cast<const u32x4*>(src + dim);
    }
#pragma unroll
    for (int s = 0; s < KS + RS; s++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(raw[s][i])), fabsf(bf16_hi(raw[s][i]))));
    amax = group_max(amax);
    const int e = (int)(__float_as_uint(amax) >> 23);
    const int up = min(max(264 - e, 1), 253);            // biased exponent of the row's scaling
    const float mul = __uint_as_float((uint32_t)up << 23);
    fac = p.scale_log2 * (MLA ? 1.0f : *p.gscale[0]) * __uint_as_float((uint32_t)(254 - up) << 23);
#pragma unroll
    for (int s = 0; s < KS + RS; s++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            q[s][2 * i] = (_Float16)(bf16_lo(raw[s][i]) * mul);
            q[s][2 * i + 1] = (_Float16)(bf16_hi(raw[s][i]) * mul);
        }
}

// A row at position pos sees the keys <= hi that are > lo or sinks, and of a
// tree's drafted tokens those that its mask names.
template <bool TREE>
__device__ __forceinline__ int sight_hi(const AttnParams& p, const RowTile& t, int pos) {
    return pos < 0 ? -1 : TREE ? t.kv_len - 1 : min(pos, t.kv_len - 1);
}
__device__ __forceinline__ int sight_lo(const AttnParams& p, int pos) {
    return p.window > 0 && pos >= p.window ? pos - p.window : -1;
}
// Bit 4 h + i: the lane's key key0 + 16 h + i (h < H, i < 4) is <= last.
template <int H>
__device__ __forceinline__ uint32_t keys_upto(int last, int key0) {
    uint32_t bits = 0;
#pragma unroll
    for (int h = 0; h < H; h++) bits |= ((1u << min(max(last - key0 + 1 - 16 * h, 0), 4)) - 1) << (4 * h);
    return bits;
}
// Hidden keys' logits of one row become -infinity; key0 counts the lane group,
// live as from live_keys.
template <bool TREE, int H>
__device__ __forceinline__ void hide(const AttnParams& p, const RowTile& t, int pos, int tok, int key0, uint32_t live,
                                     f32x4* x) {
    uint32_t see = live & keys_upto<H>(sight_hi<TREE>(p, t, pos), key0);
    if (TREE) {
        // drafted keys: their byte in the row's mask, four loads at a time
        const uint8_t* row = p.mask + (int64_t)tok * p.mask_ts;
        uint32_t named = 0;
#pragma unroll 1
        for (int h = 0; h < H; h++) {
            const int d0 = key0 + 16 * h - t.ctx;
            uint32_t byte[4];
#pragma unroll
            for (int i = 0; i < 4; i++)
                byte[i] = (see >> (4 * h + i) & 1) && d0 + i >= 0 && d0 + i < p.mask_cols ? row[d0 + i] : 0;
#pragma unroll
            for (int i = 0; i < 4; i++) named |= (uint32_t)(byte[i] != 0) << (4 * h + i);
        }
        see &= keys_upto<H>(t.ctx - 1, key0) | named;
    } else if (p.window > 0) {
        see &= ~keys_upto<H>(sight_lo(p, pos), key0) | keys_upto<H>(p.sinks - 1, key0);
    }
#pragma unroll
    for (int h = 0; h < H; h++)
#pragma unroll
        for (int i = 0; i < 4; i++) x[h][i] = see >> (4 * h + i) & 1 ? x[h][i] : kNegInf;
}
// No row of the tile needs a mask for keys [key0, key0 + n) of existing pages.
template <bool TREE>
__device__ __forceinline__ bool all_seen(const AttnParams& p, const RowTile& t, int pos_lo, int pos_hi, int key0, int n) {
    if (key0 + n > t.kv_len) return false;
    if (TREE) return key0 + n <= t.ctx;
    return key0 + n - 1 <= pos_lo && (p.window <= 0 || key0 + n <= p.sinks || key0 > pos_hi - p.window);
}

template <int DP, bool MLA, int R, bool UNI, bool TREE>
__global__ __launch_bounds__(kAttnWaves * kWave, R * DP <= 128 ? 3 : R * DP <= 256 ? 2 : 1)
void k_attention(AttnParams p, int64_t wg0) {
    constexpr int KS = DP / 32;                          // head-dim steps of the first product
    constexpr int RS = MLA ? 2 : 0;                      // RoPE steps
    constexpr int DT = DP / 16;                          // 16-dim tiles of the output
    constexpr int RT = 16 * R;
    constexpr int TC = DT < 8 ? DT : 8;                  // dim tiles joined at a time
    constexpr int kRowFloats = 16 * TC + 4;
    __shared__ float s_o[kAttnWaves][16][kRowFloats];
    __shared__ float s_m[kAttnWaves][16], s_l[kAttnWaves][16];

    // The heads of a (row tile, split) unit read neighbouring bytes of the
    // same tokens: they get workgroup numbers 8 apart, i.e. the same XCD's L2.
    const int64_t wg = wg0 + blockIdx.x;
    const int64_t per = 8 * (int64_t)p.hk;
    const int rem = (int)(wg % per);
    const int64_t unit = wg / per * 8 + rem % 8;
    const int kvh = rem / 8;
    if (unit >= (int64_t)p.tiles * p.splits) return;
    const int tile = (int)(unit / p.splits), split = (int)(unit % p.splits);
    RowTile t;
    if (!find_tile(p, tile, RT, t)) return;
    const int v0 = split * p.chunk;                      // chunk * splits fits int32 (host)
    if (split > 0 && v0 >= t.total) return;
    // a sequence longer than the planned bound: the last split takes the rest
    const int v1 = split == p.splits - 1 ? t.total : min(t.total, v0 + p.chunk);

    const int lane = lane_id(), w = wave_id();
    const int c = lane & 15, g = lane >> 4;
    const int32_t* bt_row = p.block_table + (int64_t)t.b * p.bt_stride;

    f16x8 q[R][KS + RS];
    float fac[R];
    int pos[R], tok[R];
#pragma unroll
    for (int r = 0; r < R; r++) load_query<DP, MLA>(p, t, kvh, 16 * r, lane, q[r], fac[r], pos[r], tok[r]);
    const int pos_lo = t.ctx + t.row0 / p.group;         // of the tile's rows
    const int pos_hi = t.ctx + (t.row0 + t.rows - 1) / p.group;

    f32x4 o[R][DT];
    float m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        m[r] = kNegInf;
        l[r] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; d++) o[r][d] = f32x4{0, 0, 0, 0};
    }

    // The next tile's bytes and the page ids of the one behind it are in
    // flight while a tile is worked on.
    const auto tile_key = [&](int v) { return (v < t.sink_tiles ? v : v - t.sink_tiles + t.win_tile0) * kTileKeys; };
    const LaneOffsets lo = lane_offsets<DP, MLA>(p, kvh, lane);
    // (The page ids are asked for before the bytes: loads return in order, so
    // waiting for the ids leaves the bytes in flight.)
    Raw<DP, MLA> next;
    KeyPages pg, pg_next;
    if (v0 + w < v1) {
        pg = find_pages<UNI, kTileKeys>(p, bt_row, tile_key(v0 + w), lane);
        pg_next = pg;
        if (v0 + w + kAttnWaves < v1) pg_next = find_pages<UNI, kTileKeys>(p, bt_row, tile_key(v0 + w + kAttnWaves), lane);
        load_tile<DP, MLA, UNI>(p, pg, lo, kvh, lane, next);
    }
    for (int v = v0 + w; v < v1; v += kAttnWaves) {
        const int key0 = tile_key(v);
        const Raw<DP, MLA> raw = next;
        if (v + kAttnWaves < v1) {
            pg = pg_next;
            if (v + 2 * kAttnWaves < v1) pg_next = find_pages<UNI, kTileKeys>(p, bt_row, tile_key(v + 2 * kAttnWaves), lane);
            load_tile<DP, MLA, UNI>(p, pg, lo, kvh, lane, next);
        }

        // ---- S^T = K Q^T
        f32x4 s[R][2];
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
#pragma unroll
            for (int r = 0; r < R; r++) s[r][kk] = f32x4{0, 0, 0, 0};
            f16x2 sc[DP / 64 > 1 ? DP / 64 : 2];
#pragma unroll
            for (int i = 0; i < Raw<DP, MLA>::KSW; i++) {
                const uint32_t x = drop_nan_e4m3x4(raw.ks[kk][i]);
                const f16x2 a = e4m3x2_f16<false>(x), b = e4m3x2_f16<true>(x);
                sc[4 * i] = f16x2{a.x, a.x};
                if (DP >= 128) sc[4 * i + 1] = f16x2{a.y, a.y};
                if (DP >= 256) {
                    sc[4 * i + 2] = f16x2{b.x, b.x};
                    sc[4 * i + 3] = f16x2{b.y, b.y};
                }
            }
#pragma unroll
            for (int st = 0; st < KS; st++) {
                const uint32_t wd = raw.k[kk][st];
                const f16x2 a0 = e2m1x2_f16<0>(wd) * sc[st / 2], a1 = e2m1x2_f16<1>(wd) * sc[st / 2];
                const f16x2 a2 = e2m1x2_f16<2>(wd) * sc[st / 2], a3 = e2m1x2_f16<3>(wd) * sc[st / 2];
                const f16x8 a = {a0.x, a0.y, a1.x, a1.y, a2.x, a2.y, a3.x, a3.y};
#pragma unroll
                for (int r = 0; r < R; r++) s[r][kk] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[r][st], s[r][kk], 0, 0, 0);
            }
            if (MLA) {
#pragma unroll
                for (int st = 0; st < 2; st++) {
                    const uint32_t x = raw.rope[kk % (MLA ? 2 : 1)][2 * st], y = raw.rope[kk % (MLA ? 2 : 1)][2 * st + 1];
                    const f16x2 a0 = e4m3x2_f16<false>(x), a1 = e4m3x2_f16<true>(x);
                    const f16x2 a2 = e4m3x2_f16<false>(y), a3 = e4m3x2_f16<true>(y);
                    const f16x8 a = {a0.x, a0.y, a1.x, a1.y, a2.x, a2.y, a3.x, a3.y};
#pragma unroll
                    for (int r = 0; r < R; r++)
                        s[r][kk] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[r][KS + st % (RS ? RS : 1)], s[r][kk], 0, 0, 0);
                }
            }
        }

        // ---- logits, mask
        const bool all = all_seen<TREE>(p, t, pos_lo, pos_hi, key0, kTileKeys) && __all(raw.live == 0xFFu);
#pragma unroll
        for (int r = 0; r < R; r++) {
            s[r][0] *= fac[r];
            s[r][1] *= fac[r];
        }
        if (!all) {
#pragma unroll
            for (int r = 0; r < R; r++) hide<TREE, 2>(p, t, pos[r], tok[r], key0 + 4 * g, raw.live, s[r]);
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
        // scales of key pairs (2i, 2i+1), per 16-dim block of the lane's dims
        f16x2 vsc[DP == 512 ? 2 : 1][4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (DP == 512) {
                const uint32_t x = drop_nan_e4m3x4(__builtin_amdgcn_perm(raw.vs[2 * i + 1], raw.vs[2 * i], 0x05010400u));
                vsc[0][i] = e4m3x2_f16<false>(x);        // bytes: block 0 of both keys, then block 1
                vsc[DP == 512 ? 1 : 0][i] = e4m3x2_f16<true>(x);
                if (DP == 512) vsc[0][i] = e4m3x2_f16<false>(x);
            } else {
                vsc[0][i] = e4m3x2_f16<false>(drop_nan_e4m3x4(raw.vs[2 * i] | raw.vs[2 * i + 1] << 8));
            }
        }
        constexpr int VW = Raw<DP, MLA>::VW;
        constexpr int DW = DT < 8 ? DT : 8;              // dims per data word
#pragma unroll
        for (int vw = 0; vw < VW; vw++) {
            uint32_t ev[4], od[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t a = raw.v[2 * i][vw], b = raw.v[2 * i + 1][vw];
                ev[i] = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
                od[i] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
            }
            const int blk = DP == 512 ? vw / 2 : 0;
#pragma unroll
            for (int d = 0; d < DW; d++) {
                f16x8 a;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t x = d & 1 ? od[i] : ev[i];
                    const f16x2 h = (d / 2 == 0 ? e2m1x2_f16<0>(x) : d / 2 == 1 ? e2m1x2_f16<1>(x)
                                     : d / 2 == 2 ? e2m1x2_f16<2>(x) : e2m1x2_f16<3>(x)) * vsc[blk][i];
                    a[2 * i] = h.x;
                    a[2 * i + 1] = h.y;
                }
#pragma unroll
                for (int r = 0; r < R; r++)
                    o[r][8 * vw + d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pw[r], o[r][8 * vw + d], 0, 0, 0);
            }
        }
    }

    // ---- join the four waves, 16 rows and 16 * TC dims at a time
    const bool partial = p.splits > 1 && t.total > p.chunk;
    const float gv = MLA ? 1.0f : *p.gscale[1];
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
        const int row = t.row0 + 16 * r + jr;
        const int tl = in ? row / p.group : 0;
        const int head = kvh * p.group + (in ? row - tl * p.group : 0);
        const int64_t token = t.q0 + tl;
        float scale = 0.0f, wt[kAttnWaves];
#pragma unroll
        for (int ch = 0; ch < DT / TC; ch++) {
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int d = 0; d < TC; d += 4)
                    *reinterpret_cast<f32x4*>(&s_o[w][c][(4 * g + i) * TC + d]) =
                        f32x4{o[r][ch * TC + d][i], o[r][ch * TC + d + 1][i], o[r][ch * TC + d + 2][i],
                              o[r][ch * TC + d + 3][i]};
            __syncthreads();
            if (ch == 0) {
                float mm = kNegInf;
#pragma unroll
                for (int k = 0; k < kAttnWaves; k++) mm = fmaxf(mm, s_m[k][jr]);
                float ll = 0.0f;
#pragma unroll
                for (int k = 0; k < kAttnWaves; k++) {
                    wt[k] = s_m[k][jr] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(s_m[k][jr] - mm);
                    ll = __builtin_fmaf(wt[k], s_l[k][jr], ll);
                }
                if (partial) {
                    scale = 1.0f;
                    if (in && jc == 0) {
                        float* ml = p.ws_ml + 2 * ((int64_t)split * p.total_q * p.hq + token * p.hq + head);
                        ml[0] = mm;
                        ml[1] = ll;
                    }
                } else {
                    scale = ll == 0.0f ? 0.0f : gv / ll;
                    if (in && jc == 0 && p.lse)
                        p.lse[token * p.lse_ts + head] =
                            ll == 0.0f ? kNegInf : (mm - kShift + __builtin_log2f(ll)) * 0.6931471805599453f;
                }
            }
            float acc[TC];
#pragma unroll
            for (int d = 0; d < TC; d++) acc[d] = 0.0f;
#pragma unroll
            for (int k = 0; k < kAttnWaves; k++)
#pragma unroll
                for (int d = 0; d < TC; d++) acc[d] = __builtin_fmaf(wt[k], s_o[k][jr][jc * TC + d], acc[d]);
            const int dim = jc * DT + ch * TC;
            if (in && (MLA || dim < p.hs)) {
                if (partial) {
                    float* dst = p.ws_o + ((int64_t)split * p.total_q * p.hq + token * p.hq + head) * p.hs + dim;
#pragma unroll
                    for (int d = 0; d < TC; d += 4)
                        *reinterpret_cast<f32x4*>(dst + d) = f32x4{acc[d], acc[d + 1], acc[d + 2], acc[d + 3]};
                } else {
                    uint16_t* dst = p.out + token * p.o_ts + (int64_t)head * p.o_hs + dim;
                    uint32_t pk[TC / 2];
#pragma unroll
                    for (int d = 0; d < TC / 2; d++) pk[d] = pack_bf16x2(acc[2 * d] * scale, acc[2 * d + 1] * scale);
                    if (TC == 8) *reinterpret_cast<u32x4*>(dst) = u32x4{pk[0], pk[1], pk[2 % (TC / 2)], pk[3 % (TC / 2)]};
                    else *reinterpret_cast<u32x2*>(dst) = u32x2{pk[0], pk[1]};
                }
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------------------
// Many query rows: four waves with 32 rows each and one stream of keys.  A
// 64-key step's operands are dequantized once, a quarter by each wave, into
// LDS in the exact register order of the matrix instruction (1 KiB a
// fragment, lane l at 16 l: conflict-free 16-byte reads and writes), double
// buffered: step i is multiplied while step i + 1 is converted and step
// i + 2's bytes are in flight.  Against dequantizing in every wave this takes
// the converters' share of the vector instructions from 58 to 25 per cent.
// ---------------------------------------------------------------------------
constexpr int kStepKeys = 64;

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
__device__ __forceinline__ void load_share(const AttnParams& p, const KeyPages& pg, const LaneOffsets& lo, int kvh,
                                           int lane, int w, Share<DP>& r, uint32_t& live) {
    constexpr int KB = DP / 8;
    const int c = lane & 15, g = lane >> 4;
    const bool full = p.hs == DP;
    // wave w: the K rows of keys 16 w .. 16 w + 15; V of keys 32 (w / 2) .. + 31, half w % 2 of the lane's dims
    live = live_keys<UNI, kStepKeys>(p, pg, lane);
    const uint8_t *kd, *sd;
    const int vh = w & 2;                                // V's first group
    const GroupBytes gb[2] = {group_bytes<UNI, false>(p, pg, vh), group_bytes<UNI, false>(p, pg, vh + 1)};
    const GroupBytes kb = {w & 1 ? gb[1].d : gb[0].d, w & 1 ? gb[1].s : gb[0].s};
    key_bytes<DP, false, UNI>(p, pg, kb, lo, w, false, 0, kvh, lane, kd, sd);
    if (full) {
        if (KB == 8) {
            const u32x2 x = *reinterpret_cast<const u32x2_a8*>(kd);
            r.k[0] = x.x;
            r.k[1] = x.y;
        } else {
#pragma unroll
            for (int u = 0; u < KB / 16; u++) {
                const u32x4 x = *reinterpret_cast<const u32x4_a8*>(kd + 16 * u);
#pragma unroll
                for (int i = 0; i < 4; i++) r.k[(4 * u + i) % (DP / 32)] = x[i];
            }
        }
        if (DP == 64) r.ks = *sd;
        if (DP == 128) r.ks = *reinterpret_cast<const u16_a1*>(sd);
        if (DP == 256) r.ks = *reinterpret_cast<const u32_a1*>(sd);
    } else {
        r.ks = 0;
#pragma unroll
        for (int u = 0; u < KB / 8; u++) {
            u32x2 x = {0, 0};
            if ((DP / 4) * g + 16 * u < p.hs) {
                x = *reinterpret_cast<const u32x2_a8*>(kd + 8 * u);
                r.ks |= (uint32_t)sd[u] << (8 * u);
            }
            r.k[2 * u] = x.x;
            r.k[2 * u + 1] = x.y;
        }
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const uint8_t *vd, *sv;
        key_bytes<DP, false, UNI>(p, pg, gb[j >> 2], lo, vh + (j >> 2), true, j & 3, kvh, lane, vd, sv);
        r.v[j] = 0;
        r.vs[j] = 0;
        if (full || (DP / 16) * c < p.hs) {
            if (DP == 64) r.v[j] = vd[w & 1];
            if (DP == 128) r.v[j] = reinterpret_cast<const uint16_t*>(vd)[w & 1];
            if (DP == 256) r.v[j] = reinterpret_cast<const uint32_t*>(vd)[w & 1];
            r.vs[j] = *sv;
        }
    }
}

template <int DP>
__device__ __forceinline__ void convert_share(const Share<DP>& r, int lane, int w, f16x8* lds) {
    typedef Share<DP> S;
    const uint32_t x = drop_nan_e4m3x4(r.ks);
    const f16x2 a = e4m3x2_f16<false>(x), b = e4m3x2_f16<true>(x);
    const f16x2 sc[4] = {{a.x, a.x}, {a.y, a.y}, {b.x, b.x}, {b.y, b.y}};
#pragma unroll
    for (int st = 0; st < S::KS; st++) {
        const uint32_t wd = r.k[st];
        const f16x2 a0 = e2m1x2_f16<0>(wd) * sc[st / 2], a1 = e2m1x2_f16<1>(wd) * sc[st / 2];
        const f16x2 a2 = e2m1x2_f16<2>(wd) * sc[st / 2], a3 = e2m1x2_f16<3>(wd) * sc[st / 2];
        lds[(w * S::KS + st) * kWave + lane] = f16x8{a0.x, a0.y, a1.x, a1.y, a2.x, a2.y, a3.x, a3.y};
    }
    f16x2 vsc[4];
    uint32_t ev[4], od[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        vsc[i] = e4m3x2_f16<false>(drop_nan_e4m3x4(r.vs[2 * i] | r.vs[2 * i + 1] << 8));
        const uint32_t lo = r.v[2 * i], hi = r.v[2 * i + 1];
        ev[i] = (lo & 0x0F0F0F0Fu) | ((hi << 4) & 0xF0F0F0F0u);
        od[i] = ((lo >> 4) & 0x0F0F0F0Fu) | (hi & 0xF0F0F0F0u);
    }
    f16x8* dst = lds + (S::KF + (w >> 1) * S::DT + (w & 1) * S::HT) * kWave + lane;
#pragma unroll
    for (int d = 0; d < S::HT; d++) {
        f16x8 f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t y = d & 1 ? od[i] : ev[i];
            const f16x2 h = (d / 2 == 0 ? e2m1x2_f16<0>(y) : d / 2 == 1 ? e2m1x2_f16<1>(y)
                             : d / 2 == 2 ? e2m1x2_f16<2>(y) : e2m1x2_f16<3>(y)) * vsc[i];
            f[2 * i] = h.x;
            f[2 * i + 1] = h.y;
        }
        dst[d * kWave] = f;
    }
}

template <int DP, int R, bool UNI, bool TREE>
__global__ __launch_bounds__(kAttnWaves * kWave, DP <= 128 ? 2 : 1) void k_attention_rows(AttnParams p, int64_t wg0) {
    typedef Share<DP> S;
    constexpr int KS = S::KS, DT = S::DT;
    constexpr int RT = kAttnWaves * 16 * R;
    __shared__ f16x8 s_frag[2][(S::KF + S::VF) * kWave];

    const int64_t wg = wg0 + blockIdx.x;
    const int64_t per = 8 * (int64_t)p.hk;
    const int rem = (int)(wg % per);
    const int64_t unit = wg / per * 8 + rem % 8;
    const int kvh = rem / 8;
    if (unit >= (int64_t)p.tiles * p.splits) return;
    const int tile = (int)(unit / p.splits), split = (int)(unit % p.splits);
    RowTile t;
    if (!find_tile(p, tile, RT, t)) return;
    const int v0 = split * p.chunk;                      // 32-key tiles, as in k_attention; chunk is even
    if (split > 0 && v0 >= t.total) return;
    const int v1 = split == p.splits - 1 ? t.total : min(t.total, v0 + p.chunk);

    const int lane = lane_id(), w = wave_id();
    const int c = lane & 15, g = lane >> 4;
    const int32_t* bt_row = p.block_table + (int64_t)t.b * p.bt_stride;
    f16x8 q[R][KS];
    float fac[R];
    int pos[R], tok[R];
#pragma unroll
    for (int r = 0; r < R; r++)
        load_query<DP, false>(p, t, kvh, 16 * (R * w + r), lane, q[r], fac[r], pos[r], tok[r]);
    const int row_a = min(t.row0 + 16 * R * w, t.row0 + t.rows - 1);
    const int row_b = min(t.row0 + 16 * R * w + 16 * R - 1, t.row0 + t.rows - 1);
    const int pos_lo = t.ctx + row_a / p.group, pos_hi = t.ctx + row_b / p.group;   // of the wave's rows

    f32x4 o[R][DT];
    float m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        m[r] = kNegInf;
        l[r] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; d++) o[r][d] = f32x4{0, 0, 0, 0};
    }
    const LaneOffsets lo = lane_offsets<DP, false>(p, kvh, lane);
    // Steps of 64 keys: the tiles [v0, v1) are runs of sink tiles and window
    // tiles; a step covers two consecutive tile numbers of one run.  Keys of a
    // step behind its run (or behind v1) are hidden by `end`.
    const auto step_key = [&](int v) { return (v < t.sink_tiles ? v : v - t.sink_tiles + t.win_tile0) * kTileKeys; };
    const auto run_end = [&](int v) { return v < t.sink_tiles ? min(t.sink_tiles, v1) : v1; };
    Share<DP> raw;
    KeyPages pg, pg_next;
    uint32_t live, live_n = 0, live_nn = 0;
    const auto after = [&](int x) { return min(x + 2, run_end(x)); };
    const auto look_up = [&](int x) { return find_pages<UNI, kStepKeys>(p, bt_row, step_key(x < v1 ? x : v0), lane); };
    int v = v0, vn = v1, vnn = v1, vp = v1;              // this step, the converted, the loading, the looked-up one
    if (v < v1) {
        pg = look_up(v);
        vn = after(v);
        pg_next = look_up(vn);
        load_share<DP, UNI>(p, pg, lo, kvh, lane, w, raw, live);
        convert_share<DP>(raw, lane, w, s_frag[0]);
        if (vn < v1) {
            vnn = after(vn);
            pg = pg_next;
            pg_next = look_up(vnn);
            load_share<DP, UNI>(p, pg, lo, kvh, lane, w, raw, live_n);
        }
    }
    __syncthreads();
    for (int buf = 0; v < v1; buf ^= 1) {                // workgroup-uniform
        if (vn < v1) {
            convert_share<DP>(raw, lane, w, s_frag[buf ^ 1]);
            if (vnn < v1) {
                vp = after(vnn);
                pg = pg_next;
                pg_next = look_up(vp);
                load_share<DP, UNI>(p, pg, lo, kvh, lane, w, raw, live_nn);
            }
        }
        const int key0 = step_key(v), tiles = after(v) - v;   // one or two tiles
        const f16x8* fr = s_frag[buf] + lane;
        const uint32_t lv = tiles == 2 ? live : live & 0xFFu;
        const bool all = lv == 0xFFFFu && all_seen<TREE>(p, t, pos_lo, pos_hi, key0, kStepKeys);

        f32x4 s[R][4];
#pragma unroll
        for (int kt = 0; kt < 4; kt++) {
#pragma unroll
            for (int r = 0; r < R; r++) s[r][kt] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int st = 0; st < KS; st++) {
                const f16x8 a = fr[(kt * KS + st) * kWave];
#pragma unroll
                for (int r = 0; r < R; r++) s[r][kt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[r][st], s[r][kt], 0, 0, 0);
            }
        }
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int kt = 0; kt < 4; kt++) s[r][kt] *= fac[r];
        if (!__all(all)) {
#pragma unroll
            for (int r = 0; r < R; r++) hide<TREE, 4>(p, t, pos[r], tok[r], key0 + 4 * g, lv, s[r]);
        }
        float top[R];
        bool late = false;
#pragma unroll
        for (int r = 0; r < R; r++) {
            top[r] = group_max(fmaxf(max8(s[r][0], s[r][1]), max8(s[r][2], s[r][3])));
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
        f16x8 pw[R][2];
#pragma unroll
        for (int r = 0; r < R; r++) {
            const float sub = m[r] == kNegInf ? 0.0f : kShift - m[r];
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 16; j++) {
                const float e = __builtin_amdgcn_exp2f(s[r][j >> 2][j & 3] + sub);
                sum += e;
                pw[r][j >> 3][j & 7] = (_Float16)e;
            }
            l[r] += sum;
        }
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int d = 0; d < DT; d++) {
                const f16x8 a = fr[(S::KF + h * DT + d) * kWave];
#pragma unroll
                for (int r = 0; r < R; r++) o[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pw[r][h], o[r][d], 0, 0, 0);
            }
        v = vn;
        vn = vnn;
        vnn = vp;
        live = live_n;
        live_n = live_nn;
        if (v >= v1) break;
        __syncthreads();
    }

    // ---- each lane holds 4 runs of DT dims of its row
    const bool partial = p.splits > 1 && t.total > p.chunk;
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
                float* ml = p.ws_ml + 2 * ((int64_t)split * p.total_q * p.hq + id);
                ml[0] = m[r];
                ml[1] = ll;
            } else if (p.lse) {
                p.lse[(int64_t)(t.q0 + tl) * p.lse_ts + head] =
                    ll == 0.0f ? kNegInf : (m[r] - kShift + __builtin_log2f(ll)) * 0.6931471805599453f;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int dim = (4 * g + i) * DT;
            if (dim >= p.hs) continue;
            if (partial) {
                float* dst = p.ws_o + ((int64_t)split * p.total_q * p.hq + id) * p.hs + dim;
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
__device__ __forceinline__ const uint8_t* latent_entry(const AttnParams& p, const KeyPages& pg, int h, int i) {
    int blk, off;
    take_page<UNI>(p, pg, h, 16 * h + i, blk, off);
    const uint8_t* e = p.cache + (int64_t)blk * p.L.block_stride + (int64_t)off * p.L.data_token_stride;
    return UNI ? e + (uint32_t)i * (uint32_t)p.L.data_token_stride : e;
}
template <bool UNI>
__device__ __forceinline__ void load_latent_k(const AttnParams& p, const KeyPages& pg, int lane, int w, LatentK& r) {
    const int c = lane & 15, g = lane >> 4;
    const uint8_t* e = latent_entry<UNI>(p, pg, w & 1, c);
    r.k = *reinterpret_cast<const u32x4*>(e + 64 * g + 16 * (w >> 1));
    r.ks = *reinterpret_cast<const uint16_t*>(e + kNvScaleOff + 8 * g + 2 * (w >> 1));
    if (w < 4) r.rope = *reinterpret_cast<const u32x2*>(e + kNvRopeOff + 16 * g + 8 * (w >> 1));
}
template <bool UNI>
__device__ __forceinline__ void load_latent_v(const AttnParams& p, const KeyPages& pg, int lane, int w, LatentV& r) {
    const int c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const uint8_t* e = latent_entry<UNI>(p, pg, j >> 2, 4 * g + (j & 3));
        r.v[j] = *reinterpret_cast<const uint16_t*>(e + 32 * w + 2 * c);
        r.s[j] = e[kNvScaleOff + 4 * w + (c >> 2)];
    }
}
__device__ __forceinline__ void convert_latent_k(const LatentK& r, int lane, int w, f16x8* lds) {
    const uint32_t x = drop_nan_e4m3x4(r.ks);
    const f16x2 s2 = e4m3x2_f16<false>(x);
    const f16x2 sc[2] = {{s2.x, s2.x}, {s2.y, s2.y}};
    f16x8* dst = lds + ((w & 1) * 18 + 4 * (w >> 1)) * kWave + lane;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const f16x2 a0 = e2m1x2_f16<0>(r.k[i]) * sc[i / 2], a1 = e2m1x2_f16<1>(r.k[i]) * sc[i / 2];
        const f16x2 a2 = e2m1x2_f16<2>(r.k[i]) * sc[i / 2], a3 = e2m1x2_f16<3>(r.k[i]) * sc[i / 2];
        dst[i * kWave] = f16x8{a0.x, a0.y, a1.x, a1.y, a2.x, a2.y, a3.x, a3.y};
    }
    if (w < 4) {
        const f16x2 a0 = e4m3x2_f16<false>(r.rope.x), a1 = e4m3x2_f16<true>(r.rope.x);
        const f16x2 a2 = e4m3x2_f16<false>(r.rope.y), a3 = e4m3x2_f16<true>(r.rope.y);
        lds[((w & 1) * 18 + 16 + (w >> 1)) * kWave + lane] = f16x8{a0.x, a0.y, a1.x, a1.y, a2.x, a2.y, a3.x, a3.y};
    }
}

template <bool UNI, bool TREE>
__global__ __launch_bounds__(kLatentWaves * kWave, 2) void k_attention_latent(AttnParams p, int64_t wg0) {
    constexpr int KF = 18;                               // K fragments of a key tile
    __shared__ f16x8 s_k[2][kLatentFrags * kWave];
    __shared__ f16x4 s_p[2][4][kWave][2];                // weights: row tile, lane, key tile
    __shared__ float s_top[2][4][16], s_l[2][4][16];
    __shared__ int s_flag[3];

    const int64_t unit = wg0 + blockIdx.x;
    if (unit >= (int64_t)p.tiles * p.splits) return;
    const int tile = (int)(unit / p.splits), split = (int)(unit % p.splits);
    RowTile t;
    if (!find_tile(p, tile, kLatentRows, t)) return;
    const int v0 = split * p.chunk;
    if (split > 0 && v0 >= t.total) return;
    const int v1 = split == p.splits - 1 ? t.total : min(t.total, v0 + p.chunk);

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
    float m[4], l = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        m[i] = kNegInf;
#pragma unroll
        for (int d = 0; d < 4; d++) o[i][d] = f32x4{0, 0, 0, 0};
    }
    if (threadIdx.x < 3) s_flag[threadIdx.x] = 0;
    const auto look_up = [&](int x) { return find_pages<UNI, kTileKeys>(p, bt_row, (x < v1 ? x : v0) * kTileKeys, lane); };
    LatentK rk;
    LatentV rv;
    KeyPages pg0, pg1, pg2;                              // of steps v, v + 1, v + 2
    if (v0 < v1) {
        pg0 = look_up(v0);
        pg1 = look_up(v0 + 1);
        pg2 = look_up(v0 + 2);
        load_latent_k<UNI>(p, pg0, lane, w, rk);
        convert_latent_k(rk, lane, w, s_k[0]);
        load_latent_k<UNI>(p, pg1, lane, w, rk);
        load_latent_v<UNI>(p, pg0, lane, w, rv);
    }
    __syncthreads();
    for (int v = v0, n = 0, f = 0; v < v1; v++, n ^= 1, f = f == 2 ? 0 : f + 1) {
        // ---- scores of step v, K of step v + 1
        const uint32_t live = live_keys<UNI, kTileKeys>(p, pg0, lane) >> (4 * kt) & 0xF;
        f32x4 s = {0, 0, 0, 0};
        {
            const f16x8* fr = s_k[n] + kt * KF * kWave + lane;
#pragma unroll
            for (int i = 0; i < KF; i++) s = __builtin_amdgcn_mfma_f32_16x16x32_f16(fr[i * kWave], q[i], s, 0, 0, 0);
        }
        convert_latent_k(rk, lane, w, s_k[n ^ 1]);       // (behind the last step: page 0 of the row again, unused)
        pg0 = pg1;
        pg1 = pg2;
        pg2 = look_up(v + 3);
        load_latent_k<UNI>(p, pg1, lane, w, rk);
        const int key0 = v * kTileKeys + 16 * kt;
        s *= fac;
        if (!(live == 0xF && all_seen<TREE>(p, t, pos_lo, pos_hi, key0, 16)) || !UNI)
            hide<TREE, 1>(p, t, pos, tok, key0 + 4 * g, live, &s);
        float top = group_max(fmaxf(max3(s[0], s[1], s[2]), s[3]));
        float own = rt == 0 ? m[0] : rt == 1 ? m[1] : rt == 2 ? m[2] : m[3];
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
        uint32_t ev[4], od[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            vsc[i] = e4m3x2_f16<false>(drop_nan_e4m3x4(rv.s[2 * i] | rv.s[2 * i + 1] << 8));
            ev[i] = (rv.v[2 * i] & 0x0F0F0F0Fu) | ((rv.v[2 * i + 1] << 4) & 0xF0F0F0F0u);
            od[i] = ((rv.v[2 * i] >> 4) & 0x0F0F0F0Fu) | (rv.v[2 * i + 1] & 0xF0F0F0F0u);
        }
        load_latent_v<UNI>(p, pg0, lane, w, rv);         // of step v + 1
        f16x8 pw[4];
#pragma unroll
        for (int i = 0; i < 4; i++) pw[i] = *reinterpret_cast<const f16x8*>(&s_p[n][i][lane][0]);
#pragma unroll
        for (int d = 0; d < 4; d++) {
            f16x8 a;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t y = d & 1 ? od[i] : ev[i];
                const f16x2 h = (d / 2 == 0 ? e2m1x2_f16<0>(y) : e2m1x2_f16<1>(y)) * vsc[i];
                a[2 * i] = h.x;
                a[2 * i + 1] = h.y;
            }
#pragma unroll
            for (int i = 0; i < 4; i++) o[i][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pw[i], o[i][d], 0, 0, 0);
        }
    }

    // ---- sums of the key tiles' waves, then each wave writes its 64 dims of every row
    l = group_sum(l);
    if (g == 0) s_l[kt][rt][c] = l;
    __syncthreads();
    const bool partial = p.splits > 1 && t.total > p.chunk;
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
                float* ml = p.ws_ml + 2 * ((int64_t)split * p.total_q * p.hq + id);
                ml[0] = m[i];
                ml[1] = ll;
            } else if (p.lse) {
                p.lse[(int64_t)(t.q0 + tl) * p.lse_ts + head] =
                    ll == 0.0f ? kNegInf : (m[i] - kShift + __builtin_log2f(ll)) * 0.6931471805599453f;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int dim = 64 * w + 4 * (4 * g + j);
            const f32x4 x = {o[i][0][j], o[i][1][j], o[i][2][j], o[i][3][j]};
            if (partial) {
                *reinterpret_cast<f32x4*>(p.ws_o + ((int64_t)split * p.total_q * p.hq + id) * kNope + dim) = x;
            } else {
                *reinterpret_cast<u32x2*>(p.out + (int64_t)(t.q0 + tl) * p.o_ts + (int64_t)head * p.o_hs + dim) =
                    u32x2{pack_bf16x2(x[0] * scale, x[1] * scale), pack_bf16x2(x[2] * scale, x[3] * scale)};
            }
        }
    }
}

// Join the key splits of a row: one wave per (token, head).
__global__ __launch_bounds__(kBlockThreads) void k_attention_join(AttnParams p, int64_t wg0) {
    const int lane = lane_id();
    const int RT = p.row_tile;
    const int64_t id = (wg0 + blockIdx.x) * kWavesPerBlock + wave_id();
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
    tile_range(p, t);
    if (t.total <= p.chunk) return;                      // written by its only workgroup
    const int n = min((t.total - 1) / p.chunk + 1, p.splits);
    float mm = kNegInf;
    for (int k = 0; k < n; k++) mm = fmaxf(mm, p.ws_ml[2 * (k * rows + id)]);
    float ll = 0.0f;
    for (int k = 0; k < n; k++) {
        const float mk = p.ws_ml[2 * (k * rows + id)];
        const float wt = mk == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mk - mm);
        ll = __builtin_fmaf(wt, p.ws_ml[2 * (k * rows + id) + 1], ll);
    }
    const float scale = ll == 0.0f ? 0.0f : (p.gscale[1] ? *p.gscale[1] : 1.0f) / ll;
    for (int d = 4 * lane; d < p.hs; d += 4 * kWave) {
        f32x4 acc = {0, 0, 0, 0};
        for (int k = 0; k < n; k++) {
            const float mk = p.ws_ml[2 * (k * rows + id)];
            const float wt = mk == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mk - mm);
            const f32x4 x = *reinterpret_cast<const f32x4*>(p.ws_o + (k * rows + id) * p.hs + d);
#pragma unroll
            for (int i = 0; i < 4; i++) acc[i] = __builtin_fmaf(wt, x[i], acc[i]);
        }
        *reinterpret_cast<u32x2*>(p.out + (int64_t)token * p.o_ts + (int64_t)head * p.o_hs + d) =
            u32x2{pack_bf16x2(acc[0] * scale, acc[1] * scale), pack_bf16x2(acc[2] * scale, acc[3] * scale)};
    }
    if (lane == 0 && p.lse)
        p.lse[(int64_t)token * p.lse_ts + head] =
            ll == 0.0f ? kNegInf : (mm - kShift + __builtin_log2f(ll)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
AttnPlan plan_attention(int64_t total_q, int32_t batch, int32_t hq, int32_t hk, int32_t dp, int32_t dv,
                        int64_t max_seq_len, int32_t window, int32_t sinks, int64_t ws_floats_avail) {
    AttnPlan a;
    const int64_t group = hq / hk, rows = total_q * group;
    const int64_t mean = (rows + batch - 1) / batch;     // rows of a request and kv head
    a.row_tiles = mean <= 16 || (dp >= 256 && mean <= 32) ? 1 : mean <= 32 ? 2 : dp > 256 ? kLatentRows / 16 : 8;
    const int64_t rt = 16 * a.row_tiles;
    a.tiles = (int32_t)(rows / rt + batch);
    // 32-key tiles that a row tile can see (a bound; only the split depends on it)
    int64_t keys = max_seq_len;
    if (window > 0) {
        const int64_t seen = (int64_t)window + rt / group + 1 + sinks + 2 * kTileKeys;
        if (seen < keys) keys = seen;
    }
    const int64_t kt = (keys + kTileKeys - 1) / kTileKeys + 1;
    const int64_t groups = (int64_t)a.tiles * hk;
    const int64_t want = 1024;
    int64_t splits = want / groups;
    if (splits > kt / 8) splits = kt / 8;                // at least two tiles for a wave
    if (splits > 256) splits = 256;
    const int64_t per = total_q * hq * (dv + 2);
    if (per > 0 && splits > ws_floats_avail / per) splits = ws_floats_avail / per;
    if (splits < 1) splits = 1;
    int64_t chunk = (kt + splits - 1) / splits;
    chunk = (chunk + kAttnWaves - 1) / kAttnWaves * kAttnWaves;
    splits = (kt + chunk - 1) / chunk;
    a.splits = (int32_t)splits;
    a.chunk = splits == 1 ? INT32_MAX : (int32_t)chunk;
    a.ws_floats = splits > 1 ? splits * per : 0;
    return a;
}

// The attention launch, then the join when keys are split.  row_tile: rows of
// one workgroup's tile, as the join has to see them.
static hipError_t launch_parts(void (*k)(AttnParams, int64_t), int waves, int row_tile, const AttnParams& p, hipStream_t s) {
    const int64_t units = (int64_t)p.tiles * p.splits;
    const bool join = p.splits > 1;
    const hipError_t e = launch_span(k, (units + 7) / 8 * 8 * p.hk, waves * kWave, s, true, !join, p);
    if (e != hipSuccess || !join) return e;
    AttnParams q = p;
    q.row_tile = row_tile;
    const int64_t rows = (int64_t)p.total_q * p.hq;
    return launch_span(k_attention_join, (rows + kWavesPerBlock - 1) / kWavesPerBlock, kBlockThreads, s, false, true, q);
}
// 16 keys of one page within 32-bit offsets of the first.
static bool uniform_pages(const AttnParams& p) {
    const int64_t span = 16 * (p.L.data_token_stride + p.L.scale_token_stride) +
                         p.hk * (p.L.data_head_stride + p.L.scale_head_stride) + p.L.side_stride + 1024;
    return p.div.size % 16 == 0 && span < INT32_MAX;
}

template <int DP, bool MLA, int R, bool ROWS = false>
static hipError_t launch_r(const AttnParams& p, hipStream_t s) {
    const bool uni = uniform_pages(p);
    if constexpr (ROWS)
        return launch_parts(p.mask ? (uni ? k_attention_rows<DP, R, true, true> : k_attention_rows<DP, R, false, true>)
                                   : (uni ? k_attention_rows<DP, R, true, false> : k_attention_rows<DP, R, false, false>),
                            kAttnWaves, 16 * R * kAttnWaves, p, s);
    else
        return launch_parts(p.mask ? (uni ? k_attention<DP, MLA, R, true, true> : k_attention<DP, MLA, R, false, true>)
                                   : (uni ? k_attention<DP, MLA, R, true, false> : k_attention<DP, MLA, R, false, false>),
                            kAttnWaves, 16 * R, p, s);
}

hipError_t launch_attention_kv(const AttnParams& p, int r, hipStream_t s) {
    if (p.hs <= 64)
        return r == 1 ? launch_r<64, false, 1>(p, s) : r == 2 ? launch_r<64, false, 2>(p, s) : launch_r<64, false, 2, true>(p, s);
    if (p.hs <= 128)
        return r == 1 ? launch_r<128, false, 1>(p, s)
               : r == 2 ? launch_r<128, false, 2>(p, s) : launch_r<128, false, 2, true>(p, s);
    return r == 1 ? launch_r<256, false, 1>(p, s) : launch_r<256, false, 2, true>(p, s);
}
hipError_t launch_attention_ds_mla(const AttnParams& p, int r, hipStream_t s) {
    if (r == 1) return launch_r<512, true, 1>(p, s);
    const bool uni = uniform_pages(p);
    return launch_parts(p.mask ? (uni ? k_attention_latent<true, true> : k_attention_latent<false, true>)
                               : (uni ? k_attention_latent<true, false> : k_attention_latent<false, false>),
                        kLatentWaves, kLatentRows, p, s);
}

}  // namespace gcache
