// attention_device.h -- what the attention kernels over quantized pages share:
// the walk from positions to cache bytes, the conversion to matrix operands,
// query rows, masks.
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
// Layout.  16 query rows (query token x head of the group) and 16 or 32 keys
// meet in one 16x16x32 matrix instruction:
//   S^T = K Q^T     matrix rows are keys, columns are query rows;
//   O^T = V^T P^T   matrix rows are value dims, columns are query rows.
// The result layout (lane: column l % 16, rows 4 (l / 16) + i) makes the
// scores of two 16-key tiles exactly the k-operand of the second product when
// its 8 k-slots of lane group g are taken as keys 4g..4g+3 and
// 16+4g..16+4g+3, so weights need not leave their lane, and the row
// statistics are per column, i.e. lane local.  Contraction order over the
// head dim is free, so lane group g takes the contiguous quarter g of a key's
// row (one 16-byte load for 128 dims).  For V, lane column c takes
// contiguous dims of its 8 keys and pairs the codes of two keys in one byte
// with masks and shifts before the converter, which then returns exactly the
// operand's register order.
#pragma once

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
// log2 units: weights are 2^kShift * exp2(s - m), m trails the true maximum
// by at most kLag before the accumulators are rescaled, so weights stay
// below 2^(kShift + kLag) = 2^14.
constexpr float kShift = 6.0f, kLag = 8.0f;
constexpr float kNegInf = -__builtin_inff();
constexpr float kLn2 = 0.6931471805599453f;

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
    int split, splits, chunk;    // the unit's key split, splits of the request, key tiles of one
};

__device__ __forceinline__ int query_start(const AttnParams& p, int b) {
    const int v = p.qs[b];
    return min(max(v, 0), p.total_q);
}

// Visible 32-key tiles of rows [row0, row0 + rows) of request b.
__device__ __forceinline__ void tile_range(const AttnParams& p, RowTile& t) {
    // key numbers stay clear of int32's end, so key0 + 32 cannot wrap
    const int64_t table_keys =
        p.blocks > 0 ? min(p.bt_stride * p.div.size, (int64_t)INT32_MAX - 2 * kTileKeys) : 0;
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

// Sum over the lanes up to this one.
__device__ __forceinline__ int scan_lanes(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, true);   // row_shr 1, 2, 4, 8
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // last lane of rows 0 and 2 to rows 1 and 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // last lane of the lower half to the upper
    return x;
}

// 32-key tiles of a request, as far as the plan counts them: at most key_tiles,
// the bound from max_seq_len and the window.
__device__ __forceinline__ int request_work(const AttnParams& p, int b) {
    return min((int)(((uint32_t)max(p.seq_lens[b], 0) + kTileKeys - 1) / kTileKeys), p.key_tiles);
}
// Key splits of a request: as many pieces of `chunk` 32-key tiles (a multiple
// of 4) as its counted tiles give, at least one.
__device__ __forceinline__ int request_splits(int work, int chunk) { return max(1, (work + chunk - 1) / chunk); }

// What work unit `unit` of a kv head is.  The host knows the packed rows and
// the longest sequence, but not how rows fall into requests nor how long each
// is.  It launches p.units workgroups a head, and each counts for itself: the
// size of a split is the smallest (in steps of about 1/16) for which all
// requests' splits fit the launched units, so that every unit has work of the
// same size whatever the lengths are.  Counts are sums over the lanes, each with
// batch / 64 requests, then over the requests of one lane.  Units run from the
// last to the first: causal tiles grow along a request, and the longest start
// first.  The split is rotated by the request, or the short last splits of
// equal requests would share an XCD.
// The count costs each workgroup a load for every 64 requests.  Batches with
// many requests and heads are not split, and their row tiles are numbered by a
// bound, which leaves unused numbers at even distances (every second one for
// requests of one full tile: workgroups go to XCDs and their shader engines
// round robin, and half of the engines have no work).  Counted against numbered:
//   128 x 1 token, 16 heads, 2048 latent keys        51 us against 73
//   512 x 1 token, 16 heads, 512 latent keys         39 against 52
//   1024 x 1 token, 16 heads, 256 latent keys        59 against 53
//   256 x 32 tokens, 8 kv heads, 512 per-head keys  135 against 149
//   512 x 1 token, 8 kv heads, 256 per-head keys     64 against 55
// (One long request in such a batch is then a single workgroup's for each kv
// head: 257 x 1 token over 256 keys, one of 32768 among them, 311 us; 256 x 1 85.)
__host__ __device__ __forceinline__ bool counts_requests(int batch, int kv_heads) {
    return batch <= 256 || (batch <= 512 && batch * kv_heads <= 512);
}
__device__ __forceinline__ bool find_tile(const AttnParams& p, int64_t unit, int RT, RowTile& t) {
    const int lane = lane_id();
    const auto tiles_of = [&](int rows) { return (max(rows, 0) + RT - 1) / RT; };
    int index, before;
    t.splits = 1;
    t.chunk = INT32_MAX;
    if (counts_requests(p.batch, p.hk)) {
        const bool split = p.splits > 1;
        const int per = (p.batch + kWave - 1) / kWave;
        const int b0 = lane * per;                       // requests behind the last have no rows
        const int q_first = query_start(p, min(b0, p.batch)), q_last = query_start(p, min(b0 + 1, p.batch));
        const int tiles1 = tiles_of((q_last - q_first) * p.group);                  // where a lane has one request
        const int work1 = split ? request_work(p, min(b0, p.batch - 1)) : 0;
        const auto sum = [&](auto of) {                  // of(row tiles, work) over the lane's requests
            if (per == 1) return of(tiles1, work1);
            decltype(of(0, 0)) n = 0;
            int q = q_first;
#pragma unroll 4
            for (int i = 0; i < per; i++) {
                const int next = query_start(p, min(b0 + i + 1, p.batch));
                n += of(tiles_of((next - q) * p.group), split ? request_work(p, min(b0 + i, p.batch - 1)) : 0);
                q = next;
            }
            return n;
        };
        int n, upto, all;
        if (split) {
            float work = sum([](int tiles, int w) { return (float)tiles * (float)w; });
#pragma unroll
            for (int d = 1; d < kWave; d <<= 1) work += __shfl_xor(work, d);
            const int least = max((int)(work / (float)p.units), (p.key_tiles - 1) / p.splits + 1);
            t.chunk = __builtin_amdgcn_readfirstlane((max(least, 1) + 3) / 4 * 4);
        }
        for (;;) {
            const int chunk = t.chunk;
            n = sum([&](int tiles, int w) { return split ? tiles * request_splits(w, chunk) : tiles; });
            upto = scan_lanes(n);
            all = __builtin_amdgcn_readlane(upto, kWave - 1);
            if (!split || all <= p.units || chunk >= p.key_tiles) break;
            t.chunk += max(4, chunk >> 4 & ~3);
        }
        if (split && unit == 0 && threadIdx.x == 0) *p.ws_chunk = t.chunk;
        if (unit >= all) return false;
        index = all - 1 - (int)unit;
        // (both ballots have a bit unless the metadata is written meanwhile; the mask keeps lanes and rows in range)
        int at = (__builtin_ffsll(__ballot(upto > index)) - 1) & (kWave - 1);
        before = __builtin_amdgcn_readlane(upto - n, at);
        int work = work1;
        if (per == 1) {
            t.b = at;
            t.q0 = __builtin_amdgcn_readlane(q_first, at);
            t.qlen = __builtin_amdgcn_readlane(q_last, at) - t.q0;
        } else {
            const int first = at * per, b = min(first + min(lane, per), p.batch);
            const int q = query_start(p, b), next = query_start(p, min(b + 1, p.batch));
            work = split && lane < per && b < p.batch ? request_work(p, b) : 0;
            const int tiles = lane < per ? tiles_of((next - q) * p.group) : 0;
            n = split ? tiles * request_splits(work, t.chunk) : tiles;
            upto = scan_lanes(n);
            at = (__builtin_ffsll(__ballot(before + upto > index)) - 1) & (kWave - 1);
            t.b = first + at;
            before += __builtin_amdgcn_readlane(upto - n, at);
            t.q0 = __builtin_amdgcn_readlane(q, at);
            t.qlen = __builtin_amdgcn_readlane(next, at) - t.q0;
        }
        if (split) t.splits = request_splits(__builtin_amdgcn_readlane(work, at), t.chunk);
    } else {                                             // request b from tile floor((qs[b] group + b (RT - 1)) / RT) on
        const auto first_tile = [&](int b) { return (int)(((int64_t)query_start(p, b) * p.group + (int64_t)b * (RT - 1)) / RT); };
        if (unit >= p.tiles) return false;
        index = p.tiles - 1 - (int)unit;
        int lo = 0, hi = p.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first_tile(mid) <= index) lo = mid;
            else hi = mid;
        }
        t.b = lo;
        before = first_tile(lo);
        t.q0 = query_start(p, lo);
        t.qlen = query_start(p, lo + 1) - t.q0;
    }
    t.b = min(t.b, p.batch - 1);
    const int in = index - before, tile = in / t.splits;
    t.split = (int)((uint32_t)(in - tile * t.splits + t.b) % (uint32_t)t.splits);
    const int64_t row0 = (int64_t)tile * RT, rows = (int64_t)t.qlen * p.group;
    if (t.qlen <= 0 || row0 < 0 || row0 >= rows) return false;
    t.row0 = (int)row0;
    t.rows = (int)min((int64_t)RT, rows - row0);
    tile_range(p, t);
    return true;
}
// Key tiles [v0, v1) of the unit; false: the split is behind the tile's last key.
__device__ __forceinline__ bool key_range(const RowTile& t, int& v0, int& v1) {
    v0 = t.split > 0 ? t.split * t.chunk : 0;
    // a sequence longer than the call's bound: the last split takes the rest
    v1 = t.split == t.splits - 1 ? t.total : min(t.total, v0 + t.chunk);
    return t.split == 0 || v0 < t.total;
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
// Block (0 when there is none, which is then masked) and token of 16-key group
// h (UNI) or of key i.
template <bool UNI>
__device__ __forceinline__ void take_page(const AttnParams& p, const KeyPages& g, int h, int i, int& blk, int& off) {
    blk = UNI ? __builtin_amdgcn_readlane(g.blk, h) : __shfl(g.blk, i);
    off = UNI ? __builtin_amdgcn_readlane(g.off, h) : __shfl(g.off, i);
    const bool ok = off >= 0 && (uint32_t)blk < (uint32_t)p.blocks;
    blk = ok ? blk : 0;
    off = ok ? off : 0;
}
// Bit 4 h + i: the page of the lane's key 16 h + 4 (lane / 16) + i exists.
template <bool UNI, int KEYS>
__device__ __forceinline__ uint32_t live_keys(const AttnParams& p, const KeyPages& g, int lane) {
    const uint64_t bits = __ballot(g.off >= 0 && (uint32_t)g.blk < (uint32_t)p.blocks);
    uint32_t live = 0;
#pragma unroll
    for (int h = 0; h < KEYS / 16; h++)
        live |= UNI ? ((uint32_t)bits >> h & 1) * 0xFu << (4 * h) : (uint32_t)(bits >> (16 * h + 4 * (lane >> 4)) & 0xF) << (4 * h);
    return live;
}

// Data and scale bytes of a token's row.  UNI: of group h's first key, at
// wave-uniform addresses; a lane adds 32-bit offsets that include its key's
// distance (the launcher sees to it that they fit).  Otherwise: of the lane's
// own key 16 h + i, and the offsets leave the distance out.
struct RowBytes {
    const uint8_t *d, *s;
};
template <bool UNI>
__device__ __forceinline__ RowBytes row_bytes(const AttnParams& p, const KeyPages& g, int h, int i) {
    int blk, off;
    take_page<UNI>(p, g, h, 16 * h + i, blk, off);
    const uint8_t* page = p.cache + (uint64_t)(uint32_t)blk * (uint64_t)p.L.block_stride;
    if (UNI)
        return RowBytes{page + (p.data_offset + (uint32_t)off * p.data_token), page + (p.scale_offset + (uint32_t)off * p.scale_token)};
    return RowBytes{page + p.L.data_offset + off * p.L.data_token_stride, page + p.L.scale_offset + off * p.L.scale_token_stride};
}
// row_bytes of a group, once for all of a lane's keys in it (UNI only).
template <bool UNI>
__device__ __forceinline__ RowBytes group_bytes(const AttnParams& p, const KeyPages& g, int h) {
    return UNI ? row_bytes<true>(p, g, h, 0) : RowBytes{nullptr, nullptr};
}
// The lane's offset of its part of a row: key i of a group, `part` bytes in.
template <bool UNI>
__device__ __forceinline__ uint32_t data_part(const AttnParams& p, int i, uint32_t part) {
    return (UNI ? (uint32_t)i * p.data_token : 0u) + part;
}
template <bool UNI>
__device__ __forceinline__ uint32_t scale_part(const AttnParams& p, int i, uint32_t part) {
    return (UNI ? (uint32_t)i * p.scale_token : 0u) + part;
}

// Called in a loop, makes the lane's offsets look new: otherwise their zero
// extension is hoisted, and a load's address takes a 64-bit vector add and a
// register more, instead of a scalar base with a 32-bit offset.  (64-row latent
// kernel 497 to 457 us, few rows 1 to 4 per cent; the kernel for many per-head
// rows lost 2 per cent and goes without.)
template <int N>
__device__ __forceinline__ void renew(uint32_t (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; i++) asm volatile("" : "+v"(x[i]));
}
__device__ __forceinline__ void renew(uint32_t& x) { asm volatile("" : "+v"(x)); }

// One row of queries a column: lane l takes row t.row0 + row_off + l % 16.
// Rows behind the tile are zeros at position -1.
__device__ __forceinline__ bool pos_in(const RowTile& t, int row_off, int lane) { return row_off + (lane & 15) < t.rows; }
__device__ __forceinline__ const uint16_t* query_row(const AttnParams& p, const RowTile& t, int kvh, int row_off, int lane,
                                                     int& pos, int& tok) {
    const bool in = pos_in(t, row_off, lane);
    const int row = in ? t.row0 + row_off + (lane & 15) : t.row0;
    const int tl = row / p.group;
    const int head = kvh * p.group + row - tl * p.group;
    tok = t.q0 + tl;
    pos = in ? t.ctx + tl : -1;
    return p.q + (int64_t)tok * p.q_ts + (int64_t)head * p.q_hs;
}
// First of the 8 dims of step st that lane group g holds (the last two steps of the latent form are RoPE).
template <int DP>
__device__ __forceinline__ int query_dim(int st, int g) {
    return st < DP / 32 ? (DP / 4) * g + 8 * st : kNope + 16 * g + 8 * (st - DP / 32);
}
__device__ __forceinline__ float row_amax(const u32x4& raw, float amax) {
#pragma unroll
    for (int i = 0; i < 4; i++) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(raw[i])), fabsf(bf16_hi(raw[i]))));
    return amax;
}
// The row's power of two, and in fac the factor from scores to logits in log2 units.
__device__ __forceinline__ float query_scale(const AttnParams& p, float amax, float key_scale, float& fac) {
    const int e = (int)(__float_as_uint(amax) >> 23);
    const int up = min(max(264 - e, 1), 253);            // biased exponent of the row's scaling
    fac = p.scale_log2 * key_scale * __uint_as_float((uint32_t)(254 - up) << 23);
    return __uint_as_float((uint32_t)up << 23);
}
__device__ __forceinline__ f16x8 query_operand(const u32x4& raw, float mul) {
    f16x8 q;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        q[2 * i] = (_Float16)(bf16_lo(raw[i]) * mul);
        q[2 * i + 1] = (_Float16)(bf16_hi(raw[i]) * mul);
    }
    return q;
}
// The whole row as the second operand of S^T = K Q^T.
template <int DP, bool MLA>
__device__ __forceinline__ void load_query(const AttnParams& p, const RowTile& t, int kvh, int row_off, int lane,
                                           f16x8* q, float& fac, int& pos, int& tok) {
    constexpr int N = DP / 32 + (MLA ? 2 : 0);
    const uint16_t* src = query_row(p, t, kvh, row_off, lane, pos, tok);
    u32x4 raw[N];
    float amax = 0.0f;
#pragma unroll
    for (int s = 0; s < N; s++) {
        const int dim = query_dim<DP>(s, lane >> 4);
        raw[s] = u32x4{0, 0, 0, 0};
        if (pos_in(t, row_off, lane) && (MLA || dim < p.hs)) raw[s] = *reinterpret_cast<const u32x4*>(src + dim);
    }
#pragma unroll
    for (int s = 0; s < N; s++) amax = row_amax(raw[s], amax);
    const float mul = query_scale(p, group_max(amax), MLA ? 1.0f : *p.gscale[0], fac);
#pragma unroll
    for (int s = 0; s < N; s++) q[s] = query_operand(raw[s], mul);
}

// A row at position pos sees the keys <= hi that are > lo or sinks, and of a
// tree's drafted tokens those that its mask names.
template <bool TREE>
__device__ __forceinline__ int sight_hi(const RowTile& t, int pos) {
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
    uint32_t see = live & keys_upto<H>(sight_hi<TREE>(t, pos), key0);
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
// No row at positions pos_lo .. pos_hi needs a mask for keys [key0, key0 + n) of existing pages.
template <bool TREE>
__device__ __forceinline__ bool all_seen(const AttnParams& p, const RowTile& t, int pos_lo, int pos_hi, int key0, int n) {
    if (key0 + n > t.kv_len) return false;
    if (TREE) return key0 + n <= t.ctx;
    return key0 + n - 1 <= pos_lo && (p.window <= 0 || key0 + n <= p.sinks || key0 > pos_hi - p.window);
}

// Operands from packed words.
// 8 e2m1 codes of one word, one scale -> 8 values in order.
__device__ __forceinline__ f16x8 k_operand(uint32_t w, f16x2 sc) {
    const f16x2 a = e2m1x2_f16<0>(w) * sc, b = e2m1x2_f16<1>(w) * sc, c = e2m1x2_f16<2>(w) * sc, d = e2m1x2_f16<3>(w) * sc;
    return f16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
__device__ __forceinline__ f16x8 rope_operand(uint32_t x, uint32_t y) {
    const f16x2 a = e4m3x2_f16<false>(x), b = e4m3x2_f16<true>(x), c = e4m3x2_f16<false>(y), d = e4m3x2_f16<true>(y);
    return f16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
// Scale bytes of eight keys -> pairs (key 2i, key 2i + 1).
__device__ __forceinline__ void v_scales(const uint32_t* s, f16x2* out) {
    const uint32_t a = drop_nan_e4m3x4((s[0] | s[1] << 8) | (s[2] | s[3] << 8) << 16);
    const uint32_t b = drop_nan_e4m3x4((s[4] | s[5] << 8) | (s[6] | s[7] << 8) << 16);
    out[0] = e4m3x2_f16<false>(a);
    out[1] = e4m3x2_f16<true>(a);
    out[2] = e4m3x2_f16<false>(b);
    out[3] = e4m3x2_f16<true>(b);
}
// Words of the same (up to 8) dims of eight keys, as bytes that hold one dim of
// two keys: even dims in ev, odd dims in od.
struct PairedCodes {
    uint32_t ev[4], od[4];
};
__device__ __forceinline__ PairedCodes pair_codes(const uint32_t* v) {
    PairedCodes x;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t a = v[2 * i], b = v[2 * i + 1];
        x.ev[i] = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
        x.od[i] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
    }
    return x;
}
template <int D>                                         // dim D of the word
__device__ __forceinline__ f16x8 v_operand(const PairedCodes& x, const f16x2* sc) {
    f16x8 a;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const f16x2 h = e2m1x2_f16<D / 2>(D & 1 ? x.od[i] : x.ev[i]) * sc[i];
        a[2 * i] = h.x;
        a[2 * i + 1] = h.y;
    }
    return a;
}

// Runs use(i, fragment i) over N fragments in LDS with DEPTH reads in flight.
// The barrier keeps reads and matrix instructions in this order (other
// instructions may move): left alone, the compiler reads each fragment right
// before its use and waits out the LDS latency N times.
template <int N, int DEPTH, typename Use>
__device__ __forceinline__ void stream_fragments(const f16x8* src, Use use) {
    f16x8 b[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH; i++) b[i] = src[i * kWave];
    __builtin_amdgcn_sched_barrier(0x676);
#pragma unroll
    for (int i = 0; i < N; i++) {
        use(i, b[i % DEPTH]);
        if (i + DEPTH < N) b[i % DEPTH] = src[(i + DEPTH) * kWave];
        __builtin_amdgcn_sched_barrier(0x676);
    }
}

__device__ __forceinline__ float row_lse(float m, float l) {
    return l == 0.0f ? kNegInf : (m - kShift + __builtin_log2f(l)) * kLn2;
}

// The launch of one of the kernels, then the join when keys are split.
// row_tile: rows of one workgroup's tile, as the join has to see them.
hipError_t launch_attention_parts(void (*kernel)(AttnParams, int64_t), int waves, int row_tile, const AttnParams& p,
                                  hipStream_t s);
bool uniform_pages(const AttnParams& p);

}  // namespace gcache
