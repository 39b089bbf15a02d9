// attention_tiles.h -- attention of many query rows over keys and values that
// reach the matrix instructions through LDS as they lie in memory: bf16 rows
// of packed prompts, or e4m3 rows of a paged cache.
//
// Four waves share a stream of 64-key steps; a wave has 32 query rows (query
// token x head of the group) of a 128-row tile.
//   S^T = K Q^T    32x32x16: matrix rows are keys, columns query rows;
//   O^T = V^T P^T  32x32x16: matrix rows are value dims.
// A result lane (column l % 32, half h = l / 32) holds the keys 8 a + 4 h + i
// (a, i < 4) of a 32-key tile: registers 8 s .. 8 s + 7 are the k-operand of
// the second product's 16-key step s when V's operand takes its 8 k-slots as
// keys 16 s + 4 h + i and 16 s + 8 + 4 h + i.  So weights stay in their lane,
// row statistics are per column, and V's transposition is done by the LDS
// transpose reads, whose lanes name any 4 (bf16) or 8 (e4m3) rows.
//
// Loads go from memory straight to LDS (16 bytes a lane, a wave's 1 KiB in
// one piece), double buffered: step i + 1 is in flight while step i is
// multiplied.  A lane's place in LDS is fixed, so rows are swizzled by which
// 16-byte chunk of a row a lane asks for: chunk ^ f(row) with f chosen so
// that the lanes that LDS serves in one clock (8 of a 16-byte read, 16 of a
// transpose read) fall into distinct banks.
#pragma once

#include <type_traits>

#include "attention_join.h"
#include "fp8_scale.h"

namespace gcache {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

constexpr int kStep = 64, kTileWaves = 4, kTileRows = 128;   // keys of a step, waves, rows of a tile

// One load from memory to LDS: 16 bytes a lane, lane l's to `lds` + 16 l.  The
// instruction has no register result; its end is counted by vmcnt, and the
// kernels wait for it themselves (tile_ready), because the compiler would make
// every read of any LDS buffer wait for the newest load.  m0 needs a wait state
// before an LDS load uses it.
__device__ __forceinline__ void load_lds(uint32_t lds, const void* base, uint32_t offset) {
    // (the base is the same in all lanes, which the compiler does not always see)
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    const uint64_t s = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32)) << 32 |
                       (uint32_t)__builtin_amdgcn_readfirstlane((int)b);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 : : "s"(lds), "v"(offset), "s"(s) : "memory", "m0");
}
__device__ __forceinline__ void load_lds(uint32_t lds, const void* lane_address) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 : : "s"(lds), "v"(lane_address) : "memory", "m0");
}
// Every wave's loads have landed and every wave's reads are done.
__device__ __forceinline__ void tile_ready() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" : : : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// Which chunk of its row stands at chunk c (of NC) of LDS row r: c ^ swizzle,
// within a window of the largest power of two that divides NC, at most 16
// chunks.  LDS has 64 banks: the 16 lanes of a 16-byte read, or the 32 of an
// 8-byte transpose read, that it serves in one clock have to cover 256 bytes.
template <int NC>
constexpr int kWindow = NC % 16 == 0 ? 16 : NC % 8 == 0 ? 8 : 4;
// Keys: 16 neighbouring rows read the same chunk.
template <int NC>
__device__ __forceinline__ int key_swizzle(int r) {
    return kWindow<NC> == 16 ? r & 15 : kWindow<NC> == 8 ? r >> 1 & 7 : r >> 2 & 3;
}
// Values in bf16: rows 4 n .. 4 n + 3, four neighbouring chunks each; in e4m3:
// rows 4 n + i and 4 n + 8 + i, two neighbouring chunks each.
template <int NC, bool FP8>
__device__ __forceinline__ int value_swizzle(int r) {
    constexpr int W = kWindow<NC>;
    if (!FP8) return W == 16 ? (r & 3) << 2 : (r & 3) << 1;
    return W == 16 ? (r & 3) << 1 | (r & 8) : W == 8 ? (r & 2) | (r >> 1 & 4) : r >> 2 & 2;
}
// Chunk number a + b of a row, where `at` is the place of its chunk a < the
// smallest power of two in b's numbers: an exclusive or inside a window, an
// addition from window to window.
template <int NC>
__device__ __forceinline__ uint32_t chunk_at(uint32_t at, int b) {
    constexpr int W = kWindow<NC>;
    return (at ^ (uint32_t)(b % W) << 4) + b / W * W * 16;
}

// What differs between the two sources.
struct PackedBf16 {
    typedef bf16x8 frag;
    static constexpr bool kFp8 = false;
    static constexpr int kBytes = 2;
    // Weights become bf16, the values' type, because a product takes both operands in one; a row's sum has them unrounded.
    static constexpr float kShiftUp = 0.0f;              // (they have binary32's range)
    static constexpr int kDepth = 3;                     // reads in flight (2, 3, 4: 1007, 1019, 1013 TFLOP/s with 128 dims)
    static __device__ __forceinline__ f32x16 mma(const frag& a, const frag& b, const f32x16& c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
struct PagedFp8 {
    typedef f16x8 frag;
    static constexpr bool kFp8 = true;
    static constexpr int kBytes = 1;
    static constexpr float kShiftUp = kShift;
    static constexpr int kDepth = 2;                     // 2, 3, 4: 520, 535, 540 us for 4 x 2048 tokens over 4096 keys
    static __device__ __forceinline__ f32x16 mma(const frag& a, const frag& b, const f32x16& c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

// First of the 8 dims that lane half h holds in step st of the first product.
template <typename T>
__device__ __forceinline__ int step_dim(int st, int h) {
    return T::kFp8 ? 32 * (st >> 1) + 16 * h + 8 * (st & 1) : 16 * st + 8 * h;
}

__device__ __forceinline__ f16x8 fp8_operand(uint32_t x, uint32_t y) { return rope_operand(x, y); }

// Over the two lanes of a column.
__device__ __forceinline__ float pair_max(float v) {
    const u32x2 b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b.x), __uint_as_float(b.y));
}
__device__ __forceinline__ float pair_sum(float v) {
    const u32x2 b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b.x) + __uint_as_float(b.y);
}

// Bit 4 a + i: the lane's key key0 + 8 a + i (a < 8, i < 4; key0 counts the
// lane half) is <= last.
__device__ __forceinline__ uint32_t step_keys_upto(int last, int key0) {
    uint32_t bits = 0;
#pragma unroll
    for (int a = 0; a < 8; a++) bits |= ((1u << min(max(last - key0 + 1 - 8 * a, 0), 4)) - 1) << (4 * a);
    return bits;
}

__device__ __forceinline__ float max16(const f32x16& a) {
    const float x = max3(max3(a[0], a[1], a[2]), a[3], a[4]), y = max3(max3(a[5], a[6], a[7]), a[8], a[9]);
    return fmaxf(max3(x, max3(a[10], a[11], a[12]), a[13]), max3(y, a[14], a[15]));
}

// hide() of one row for a 64-key step: bit 4 a + i of live, and the logits, as
// step_keys_upto counts.
template <bool TREE>
__device__ __forceinline__ void hide_step(const AttnParams& p, const RowTile& t, int pos, int tok, int key0, uint32_t live,
                                          f32x16* x) {
    if (!TREE && p.window <= 0 && __all(live == ~0u)) {  // causal alone
        const int last = sight_hi<TREE>(t, pos) - key0;
#pragma unroll
        for (int j = 0; j < 32; j++) x[j >> 4][j & 15] = 8 * (j >> 2) + (j & 3) <= last ? x[j >> 4][j & 15] : kNegInf;
        return;
    }
    uint32_t see = live & step_keys_upto(sight_hi<TREE>(t, pos), key0);
    if (TREE) {
        const uint8_t* row = p.mask + (int64_t)tok * p.mask_ts;
        uint32_t named = 0;
#pragma unroll 1
        for (int a = 0; a < 8; a++) {
            const int d0 = key0 + 8 * a - t.ctx;
            uint32_t byte[4];
#pragma unroll
            for (int i = 0; i < 4; i++)
                byte[i] = (see >> (4 * a + i) & 1) && d0 + i >= 0 && d0 + i < p.mask_cols ? row[d0 + i] : 0;
#pragma unroll
            for (int i = 0; i < 4; i++) named |= (uint32_t)(byte[i] != 0) << (4 * a + i);
        }
        see &= step_keys_upto(t.ctx - 1, key0) | named;
    } else if (p.window > 0) {
        see &= ~step_keys_upto(sight_lo(p, pos), key0) | step_keys_upto(p.sinks - 1, key0);
    }
#pragma unroll
    for (int j = 0; j < 32; j++) x[j >> 4][j & 15] = see >> j & 1 ? x[j >> 4][j & 15] : kNegInf;
}

// A 16-key group's page and what its weights are scaled with.
struct PageScale {
    float k, log2_v, inv_v;      // K's scale; V's as log2 and reciprocal
    uint32_t live;               // the page exists
};

template <bool FP8, int N> struct ScaleLds { PageScale at[4][N]; };
template <int N> struct ScaleLds<false, N> {};
// The kernel's part of LDS: two buffers of a step's K and V rows, and the
// scales of the groups of four steps (of their keys where pages are not whole
// groups): a step's are written two steps before its weights need them.
template <typename T, int DK, int DV, bool UNI>
struct StepLds : ScaleLds<T::kFp8, UNI ? kStep / 16 : kStep> {
    static constexpr int KB = DK * T::kBytes, VB = DV * T::kBytes;       // bytes of a row
    alignas(256) uint8_t k[2][kStep * KB];
    alignas(256) uint8_t v[2][kStep * VB];
};

// One side's 64 rows of a packed prompt into LDS: wave w issues every fourth
// KiB.  EX: heads of exactly N dims.  Otherwise chunks behind the head's last
// dim come from zeros (K: they meet zeros of the query, so they must be
// finite), and rows behind the last key are the last key's.
__device__ const u32x4 g_zero_chunk = {0, 0, 0, 0};
template <int NC, bool VALUES, bool EX>
__device__ __forceinline__ void load_rows(const uint8_t* base, int64_t stride, int dims, int left, uint32_t lds, int lane, int w) {
    constexpr int N = NC / kTileWaves;                   // KiB a wave: 64 rows of 16 NC bytes
    static_assert(kStep * NC == N * kTileWaves * kWave, "whole KiB");
    const bool all = left >= kStep;
#pragma unroll
    for (int n = 0; n < N; n++) {
        const int at = (n * kTileWaves + w) * kWave + lane, row = at / NC, place = at % NC;
        const int chunk = place ^ (VALUES ? value_swizzle<NC, false>(row) : key_swizzle<NC>(row));
        const uint32_t to = lds + (n * kTileWaves + w) * 1024;
        const uint32_t off = (uint32_t)(all ? row : min(row, left - 1)) * (uint32_t)stride + 16 * chunk;
        if (EX) load_lds(to, base, off);
        else load_lds(to, 8 * chunk < dims ? base + off : reinterpret_cast<const uint8_t*>(&g_zero_chunk));
    }
}

// Scalar loads of what the whole wave needs.  They count on another counter
// than the loads to LDS: a vector load's wait would drain those too.
template <typename V>
__device__ __forceinline__ V load_scalar(const V* p) {
    return *reinterpret_cast<const __attribute__((address_space(4))) V*>(reinterpret_cast<uint64_t>(p));
}

// A page as a wave (UNI: 16 keys of one page, scalars) or a lane finds it.
struct PageAt {
    int blk, off;                // as in the table; off -1: behind the table's row
};
template <bool UNI>
__device__ __forceinline__ PageAt find_page(const AttnParams& p, const int32_t* bt_row, int pos) {
    int bi;
    PageAt g;
    split_position(p, pos, bi, g.off);
    const bool in = bi < p.bt_stride;
    const int32_t* at = bt_row + (in ? bi : 0);
    g.blk = UNI ? load_scalar(at) : *at;
    if (!in) g.off = -1;
    return g;
}
__device__ __forceinline__ bool page_exists(const AttnParams& p, const PageAt& g) {
    return g.off >= 0 && (uint32_t)g.blk < (uint32_t)p.blocks;
}
// Rows of pages that do not exist are page 0's, and hidden.
__device__ __forceinline__ const uint8_t* page_row(const AttnParams& p, const PageAt& g) {
    const bool ok = page_exists(p, g);
    return p.cache + (int64_t)(ok ? g.blk : 0) * p.L.block_stride + (int64_t)(ok ? g.off : 0) * p.L.data_token_stride;
}
// The layout's scale strides count floats: offset from K's to V's, token from
// page to page, head.
struct RawScale {
    float k, v;
};
template <bool UNI>
__device__ __forceinline__ RawScale raw_scale(const AttnParams& p, const PageAt& g, int kvh) {
    const float* at = p.gscale[0] + (int64_t)(page_exists(p, g) ? g.blk : 0) * p.L.scale_token_stride + kvh * p.L.scale_head_stride;
    return UNI ? RawScale{load_scalar(at), load_scalar(at + p.L.scale_offset)} : RawScale{at[0], at[p.L.scale_offset]};
}
__device__ __forceinline__ PageScale scale_of(const RawScale& r, bool exists) {
    const float v = page_scale(r.v);
    return PageScale{page_scale(r.k), __builtin_log2f(v), 1.0f / v, exists ? 1u : 0u};
}

// The pages of a step of the paged cache.  Wave w loads the rows of keys 16 w ..
// 16 w + 15 of both sides, and writes their scales to LDS for all.
// UNI: the 16 keys lie in one page, whose id and scales are scalars; else every
// lane looks up the pages of the rows that it loads, and of key lane % 16.
template <int DP, bool UNI>
struct PageWalk {
    static constexpr int NC = DP / 16, N = 16 * NC / kWave;      // loads of a side: 16 rows of NC chunks
    static constexpr int LR = kWave / NC;                // rows of a load
    static constexpr int IDS = UNI ? 1 : N + 1;
    const int32_t* bt_row;
    int kvh, wave;
    PageAt next[IDS], at[IDS], was[IDS];
    RawScale scale;

    __device__ __forceinline__ void init(const AttnParams& p, const RowTile& t, int head, int w) {
        bt_row = p.block_table + (int64_t)t.b * p.bt_stride;
        kvh = head;
        wave = w;
    }
    // Ids of the step at key0; take() looks at them a step later.
    __device__ __forceinline__ void find(const AttnParams& p, int key0, int lane) {
        const int first = key0 + 16 * wave;
#pragma unroll
        for (int n = 0; n < IDS; n++)
            next[n] = find_page<UNI>(p, bt_row, first + (UNI ? 0 : n < N ? n * LR + lane / NC : lane & 15));
    }
    __device__ __forceinline__ void take(const AttnParams& p) {
#pragma unroll
        for (int n = 0; n < IDS; n++) {
            was[n] = at[n];
            at[n] = next[n];
        }
        scale = raw_scale<UNI>(p, at[IDS - 1], kvh);
    }
    // Keys (side 0) of the step taken last, values (side 1) of the one before.
    __device__ __forceinline__ void issue(const AttnParams& p, uint32_t to, int side, int lane) const {
        const int64_t far = kvh * p.L.data_head_stride + side * p.L.side_stride;
        const PageAt* from = side ? was : at;
#pragma unroll
        for (int n = 0; n < N; n++) {
            const int row = n * LR + lane / NC, place = lane % NC;
            const int chunk = place ^ (side ? value_swizzle<NC, true>(row) : key_swizzle<NC>(row));
            const uint32_t there = to + 16 * wave * DP + n * 1024;
            if constexpr (UNI) load_lds(there, page_row(p, from[0]) + far, (uint32_t)row * p.data_token + 16 * chunk);
            else                                         // chunks behind the head's last dim are zeros
                load_lds(there, 16 * chunk < p.hs ? page_row(p, from[n]) + far + 16 * chunk
                                                  : reinterpret_cast<const uint8_t*>(&g_zero_chunk));
        }
    }
    __device__ __forceinline__ void publish(const AttnParams& p, PageScale* to, int lane) const {
        const PageScale s = scale_of(scale, page_exists(p, at[IDS - 1]));
        if (UNI ? lane == 0 : lane < 16) to[UNI ? wave : 16 * wave + lane] = s;
    }
};
// Rows that see a far page hold the sum of their weights with a maximum of its
// own, that of their logits alone: 2^(top - shift) l.
struct FarSum {
    float top, l;
};
// Adds N weights; logit(j) in log2 units, `most` their maximum over the lanes of the row.
template <int N, typename Logit>
__device__ __forceinline__ void far_add(FarSum& f, float most, float shift, Logit logit) {
    const float to = fmaxf(f.top, most);
    if (to == kNegInf) return;
    const float by = shift - to;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < N; j++) sum += __builtin_amdgcn_exp2f(logit(j) + by);
    f.l = __builtin_fmaf(f.l, __builtin_amdgcn_exp2f(f.top - to), sum);
    f.top = to;
}
// The row's end in the form that joins have: the factor that makes its weighted
// values their mean, with m and a sum of 1 (0 where nothing was seen) beside it.
// l: over the lanes of the row.
__device__ __forceinline__ float far_end(const FarSum& f, float& m, float& l) {
    if (l == 0.0f) return 1.0f;
    const float mean = __builtin_amdgcn_exp2f(m - f.top) / l;
    m = f.top + __builtin_log2f(l);
    l = 1.0f;
    return mean;
}

// Whether the page of `key` is far; scales behind the last key may be anything.
__device__ __forceinline__ bool far_page(const RowTile& t, const RawScale& r, bool exists, int key) {
    return exists && key < t.kv_len && far_scale(page_scale(r.v));
}
// Whether a page with keys of the 32-key tiles [v0, v1) is far: the workgroup's
// lanes look at a page each, two at once.
struct FarLook {
    static constexpr int N = 2, THREADS = kTileWaves * kWave;
    const int32_t* bt_row;
    const float* scales;
    int first[2], pages[2];      // of the sinks and of the window
    int id[N];
    float scale[N];

    __device__ __forceinline__ int page_id(uint32_t i) const {       // of the i-th page, -1 behind the last
        const bool sink = i < (uint32_t)pages[0];
        const uint32_t k = sink ? i : i - pages[0];
        return k < (uint32_t)pages[sink ? 0 : 1] ? bt_row[first[sink ? 0 : 1] + k] : -1;
    }
    // (a page that does not exist counts as ordinary)
    __device__ __forceinline__ float scale_of_page(const AttnParams& p, int blk) const {
        return page_exists(p, PageAt{blk, 0}) ? scales[(int64_t)blk * p.L.scale_token_stride] : 1.0f;
    }
    __device__ __forceinline__ void find(const AttnParams& p, const RowTile& t, int kvh, int v0, int v1) {
        bt_row = p.block_table + (int64_t)t.b * p.bt_stride;
        scales = p.gscale[0] + p.L.scale_offset + kvh * p.L.scale_head_stride;
        const int from[2] = {v0, max(v0, t.sink_tiles) - t.sink_tiles + t.win_tile0};
        const int to[2] = {min(v1, t.sink_tiles), v1 - t.sink_tiles + t.win_tile0};      // 32-key tiles
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const int key0 = from[k] * kTileKeys, key1 = min(to[k] * kTileKeys, t.kv_len);
            int last = 0, off;
            first[k] = pages[k] = 0;
            if (key0 < key1) {
                split_position(p, key0, first[k], off);
                split_position(p, key1 - 1, last, off);
                pages[k] = last + 1 - first[k];
            }
        }
#pragma unroll
        for (int n = 0; n < N; n++) id[n] = page_id(threadIdx.x + n * THREADS);
    }
    __device__ __forceinline__ void load(const AttnParams& p) {
#pragma unroll
        for (int n = 0; n < N; n++) scale[n] = scale_of_page(p, id[n]);
    }
    __device__ __forceinline__ bool far(const AttnParams& p) const {         // the lane's pages
        bool x = false;
#pragma unroll
        for (int n = 0; n < N; n++) x = x || far_scale(page_scale(scale[n]));
        const uint32_t all = (uint32_t)pages[0] + (uint32_t)pages[1];
        for (uint32_t i = threadIdx.x + N * THREADS; i < all; i += THREADS) x = x || far_scale(page_scale(scale_of_page(p, page_id(i))));
        return x;
    }
};

// The lane's part of it, in one go.
__device__ __forceinline__ bool sees_far(const AttnParams& p, const RowTile& t, int kvh, int v0, int v1) {
    FarLook look;
    look.find(p, t, kvh, v0, v1);
    look.load(p);
    return look.far(p);
}
struct NoWalk {};

// N fragments with DEPTH reads in flight.  Piece i of `side`, vector work that
// needs none of them, follows the matrix instructions of fragment i and runs
// beside them.  The barriers keep reads and matrix instructions in this order,
// and with PIN the pieces too.
template <int N, int DEPTH, bool PIN, typename F, typename Load, typename Use, typename Side>
__device__ __forceinline__ void stream(Load load, Use use, Side side) {
    F b[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH; i++) b[i] = load(i);
    __builtin_amdgcn_sched_barrier(PIN ? 0x274 : 0x676);
#pragma unroll
    for (int i = 0; i < N; i++) {
        use(i, b[i % DEPTH]);
        if (i + DEPTH < N) b[i % DEPTH] = load(i + DEPTH);
        side(i);
        __builtin_amdgcn_sched_barrier(PIN ? 0x274 : 0x676);
    }
}
// The i-th of N parts of COUNT pieces: run(piece) for each.
template <int N, int COUNT, typename Run>
__device__ __forceinline__ void part_of(int i, Run run) {
#pragma unroll
    for (int k = 0; k < COUNT; k++)
        if (k * N / COUNT == i) run(k);
}

template <typename V>
__device__ __forceinline__ V read_lds(uint32_t at) {
    return *reinterpret_cast<const __attribute__((address_space(3))) V*>(at);
}
__device__ __forceinline__ void write_lds(uint32_t at, u32x2 x) {
    *reinterpret_cast<__attribute__((address_space(3))) u32x2*>(at) = x;
}
// Between a wave's own writes and reads of LDS: they are done in order, the
// compiler only has to keep them so.
__device__ __forceinline__ void wave_lds_ready() {
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
}
__device__ __forceinline__ i16x4 read_transposed16(uint32_t at) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<__attribute__((address_space(3))) i16x4*>(at));
}
__device__ __forceinline__ i32x2 read_transposed8(uint32_t at) {
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<__attribute__((address_space(3))) i32x2*>(at));
}

// Raw words of a fragment, and the operand they make.
template <typename T> struct RawFrag;
template <> struct RawFrag<PackedBf16> { u32x4 w; };
template <> struct RawFrag<PagedFp8> { u32x2 w; };
__device__ __forceinline__ bf16x8 operand(const RawFrag<PackedBf16>& r) { return __builtin_bit_cast(bf16x8, r.w); }
__device__ __forceinline__ f16x8 operand(const RawFrag<PagedFp8>& r) { return fp8_operand(r.w.x, r.w.y); }

// Values that some rows of a step do not see: what is not finite becomes 0
// before the product, where a weight of 0 would make it a NaN.  Returns whether
// there was any.  (An e4m3 NaN code, which no write makes, counts as 0 there.)
__device__ __forceinline__ uint32_t drop_nonfinite(RawFrag<PackedBf16>& r) {
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t x = r.w[i];
        const uint32_t lo = (x & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u, hi = (x & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u;
        any |= lo | hi;
        r.w[i] = x & ~(lo | hi);
    }
    return any;
}
__device__ __forceinline__ uint32_t drop_nonfinite(RawFrag<PagedFp8>& r) {
    const u32x2 x = r.w;
    r.w.x = drop_nan_e4m3x4(x.x);
    r.w.y = drop_nan_e4m3x4(x.y);
    return (r.w.x ^ x.x) | (r.w.y ^ x.y);
}
// What is NaN or an infinity of one sign (0 or 0x8000) as bf16's largest value of
// that sign, the rest as 0.
__device__ __forceinline__ uint32_t keep_nonfinite(uint32_t x, uint32_t sign) {      // a value in the lower half
    const bool keep = (x & 0x7F80u) == 0x7F80u && ((x & 0x7Fu) != 0 || (x & 0x8000u) == sign);
    return keep ? 0x7F7Fu | sign : 0u;
}
__device__ __forceinline__ void keep_nonfinite(RawFrag<PackedBf16>& r, uint32_t sign) {
#pragma unroll
    for (int i = 0; i < 4; i++) r.w[i] = keep_nonfinite(r.w[i] & 0xFFFFu, sign) | keep_nonfinite(r.w[i] >> 16, sign) << 16;
}

// row_end for weights shifted by T's shift (row_lse takes kShift off).
template <typename T, typename P>
__device__ __forceinline__ RowEnd row_end_shifted(const P& p, int64_t token, int head, float m, float l) {
    return row_end(p, token, head, m - T::kShiftUp + kShift, l, 1.0f);
}

// Query rows as the second operand of S^T = K Q^T.  For the e4m3 cache they
// are scaled by a power of two into binary16; mul undoes it in the logits.
template <int DK>
__device__ __forceinline__ void load_rows_q(const PromptParams& p, const uint16_t* src, bool in, int h, bf16x8* q, float& fac) {
#pragma unroll
    for (int st = 0; st < DK / 16; st++) {
        const int dim = step_dim<PackedBf16>(st, h);
        u32x4 raw = {0, 0, 0, 0};
        if (in && dim < p.dk) raw = *reinterpret_cast<const u32x4*>(src + dim);
        q[st] = __builtin_bit_cast(bf16x8, raw);
    }
    fac = p.scale_log2;
}
template <int DK>
__device__ __forceinline__ void load_rows_q(const AttnParams& p, const uint16_t* src, bool in, int h, f16x8* q, float& fac) {
    u32x4 raw[DK / 16];
    float amax = 0.0f;
#pragma unroll
    for (int st = 0; st < DK / 16; st++) {
        const int dim = step_dim<PagedFp8>(st, h);
        raw[st] = u32x4{0, 0, 0, 0};
        if (in && dim < p.hs) raw[st] = *reinterpret_cast<const u32x4*>(src + dim);
    }
#pragma unroll
    for (int st = 0; st < DK / 16; st++) amax = row_amax(raw[st], amax);
    const float mul = query_scale(p, pair_max(amax), 1.0f, fac);
#pragma unroll
    for (int st = 0; st < DK / 16; st++) q[st] = query_operand(raw[st], mul);
}

// Scores of a step: S^T = K Q^T.  A 16-byte read is one step's operand in bf16,
// two steps' in e4m3.
template <typename T, int KS, int KB, bool PIN, typename Side>
__device__ __forceinline__ void multiply_keys(uint32_t k_at, const typename T::frag* q, f32x16* s, Side side) {
    constexpr int PER = T::kFp8 ? 2 : 1, J = KS / PER;
#pragma unroll
    for (int kt = 0; kt < 2; kt++)
#pragma unroll
        for (int j = 0; j < 16; j++) s[kt][j] = 0.0f;
    stream<2 * J, T::kDepth, PIN, u32x4>(
        [&](int n) { return read_lds<u32x4>(chunk_at<KB / 16>(k_at, 2 * (n % J)) + n / J * 32 * KB); },
        [&](int n, const u32x4& x) {
            const int kt = n / J, st = n % J * PER;
            if constexpr (T::kFp8) {
                const f16x8 a = fp8_operand(x.x, x.y), b = fp8_operand(x.z, x.w);
                s[kt] = T::mma(a, q[st], s[kt]);
                s[kt] = T::mma(b, q[st + 1], s[kt]);
            } else {
                const bf16x8 a = __builtin_bit_cast(bf16x8, x);
                s[kt] = T::mma(a, q[st], s[kt]);
            }
        },
        side);
}

// One tile of up to 128 rows over the 32-key tiles [v0, v1).
// EX: packed prompts with head sizes of exactly DK and DV; a cache whose head
// size is DK and whose pages are whole 16-key groups within 32 bits.
// CAREFUL: values of hidden keys may be infinities or NaN, which a weight of 0
// would let through: looked for in every step with a mask.  Without it such a
// value makes a NaN, and the tile is computed again with it.  When not CAREFUL,
// returns kSawNan and kSawFar where there is a NaN in the workgroup's tile or a far
// page among its keys; nothing is written then.
// apart: sum the weights apart (FarSum; CAREFUL only).
//
// The scores of step i + 1 are multiplied while step i's weights are computed,
// and its values while the next logits are scaled: a wave's matrix instructions
// and its vector ones are independent, and run side by side.
constexpr uint32_t kSawNan = 1, kSawFar = 2;
// A tile of many rows looks for far pages behind its last step, when the scales
// are in L2 (3 chunks over 2 k to 6 k keys 441 us, 438 without a look; before the
// first step 453, in every step 460); with 256 dims before the first (4 x 2048
// tokens over 4096 keys 460 us, 548 behind the last, 530 without: the compiler
// then spills fewer registers).
template <int DK>
constexpr bool kLookFirst = DK > 128;
template <typename T, int DK, int DV, bool EX, bool TREE, bool CAREFUL, typename P>
__device__ __forceinline__ uint32_t attend_once(const P& p, const RowTile& t, int kvh, int v0, int v1, bool apart,
                                                StepLds<T, DK, DV, EX>& lds) {
    typedef StepLds<T, DK, DV, EX> L;
    typedef typename T::frag frag;
    constexpr int KS = DK / 16, DT = DV / 32, KC = L::KB / 16, VC = L::VB / 16;
    constexpr bool FP8 = T::kFp8;
    // Pieces of vector work stay between the matrix instructions they are written beside.  Left to the compiler they may
    // all come last: 192 dims 1071 against 1120 TFLOP/s, 256 681 against 910, 128 929 to 1018 from one build to the next
    // against 1019; but with e4m3's conversions among them 569 us against 540, and 64 dims 841 against 825.
    constexpr bool kPin = !FP8 && DK >= 128;
    // Sums of weights where the weights are made: as late as possible, 32 weights stay in registers, and 192 dims spill
    // (724 against 1029 TFLOP/s); e4m3 540 against 557 us.
    constexpr bool kSumEarly = FP8 || DK % 128 != 0;
    // A higher wave priority while matrix instructions are issued: 128 dims 963 against 949 TFLOP/s, e4m3 531 against 557
    // us, 192 as before; but 64 dims 761 against 780 and 256 919 against 936.
    constexpr bool kRaise = DK == 128 || DK == 192;
    const int lane = lane_id(), w = wave_id(), c = lane & 31, h = lane >> 5;

    // ---- steps: one or two consecutive 32-key tiles of one run (sinks, then the window)
    const auto step_key = [&](int v) { return (v < t.sink_tiles ? v : v - t.sink_tiles + t.win_tile0) * kTileKeys; };
    const auto after = [&](int v) { return v < v1 ? min(v + 2, v < t.sink_tiles ? min(t.sink_tiles, v1) : v1) : v1; };

    // ---- loads of a step
    const uint32_t lds_k = lds_address(lds.k[0]), lds_v = lds_address(lds.v[0]);
    const uint8_t* base[2] = {nullptr, nullptr};
    int64_t stride[2] = {0, 0};
    std::conditional_t<FP8, PageWalk<DK, EX>, NoWalk> walk;
    if constexpr (FP8) walk.init(p, t, kvh, w);
    else {
        const int64_t first = __builtin_amdgcn_readfirstlane(t.k0);
        stride[0] = 2 * p.k_ts;
        stride[1] = 2 * p.v_ts;
        base[0] = reinterpret_cast<const uint8_t*>(p.k + first * p.k_ts + kvh * p.k_hs);
        base[1] = reinterpret_cast<const uint8_t*>(p.v + first * p.v_ts + kvh * p.v_hs);
    }
    // keys of step number n at v, values of step number n at v
    const auto issue_keys = [&](int v, int n) {
        const uint32_t to = lds_k + (n & 1) * (int)sizeof(lds.k[0]);
        if constexpr (FP8) {
            walk.issue(p, to, 0, lane);
            walk.publish(p, lds.at[n & 3], lane);
        } else {
            const int key0 = step_key(v);
            load_rows<KC, false, EX>(base[0] + key0 * stride[0], stride[0], p.dk, t.kv_len - key0, to, lane, w);
        }
    };
    const auto issue_values = [&](int v, int n) {
        const uint32_t to = lds_v + (n & 1) * (int)sizeof(lds.v[0]);
        if constexpr (FP8) walk.issue(p, to, 1, lane);
        else {
            const int key0 = step_key(v);
            load_rows<VC, true, EX>(base[1] + key0 * stride[1], stride[1], p.hs, t.kv_len - key0, to, lane, w);
        }
    };

    int v = v0, vn = after(v), vp = after(vn);           // this step, the next, the one after
    if (v < v1) {
        if constexpr (FP8) {
            walk.find(p, step_key(v), lane);
            walk.take(p);
            walk.find(p, step_key(vn < v1 ? vn : v), lane);
        }
        issue_keys(v, 0);
        if constexpr (FP8) {
            walk.take(p);
            walk.find(p, step_key(vp < v1 ? vp : v), lane);
        }
        issue_values(v, 0);
    }

    // ---- query rows
    frag q[KS];
    float fac;
    int pos, tok, row_of;
    {
        const int off = 32 * w + c;
        const bool in = off < t.rows;
        const int row = in ? t.row0 + off : t.row0, tl = row_token(p, row), head = kvh * p.group + row - tl * p.group;
        row_of = in ? row : -1;
        tok = t.q0 + tl;
        pos = in ? t.ctx + tl : -1;
        load_rows_q<DK>(p, p.q + (int64_t)tok * p.q_ts + (int64_t)head * p.q_hs, in, h, q, fac);
    }
    const bool busy = 32 * w < t.rows;                   // the other waves of a partly filled tile only load
    const int pos_lo = t.ctx + row_token(p, min(t.row0 + 32 * w, t.row0 + t.rows - 1));
    const int pos_hi = t.ctx + row_token(p, min(t.row0 + 32 * (w + 1) - 1, t.row0 + t.rows - 1));

    // ---- where a lane reads: K rows c and 32 + c; V rows of its 16-lane group
    const uint32_t k_lane = lds_k + c * L::KB + ((h ^ key_swizzle<KC>(c)) << 4);
    const int i = lane & 15, dim_half = lane >> 4 & 1;
    const int v_row = FP8 ? 4 * h + (i >> 1 & 3) + 8 * (i >> 3) : 4 * h + (i >> 2);
    const int v_chunk = FP8 ? dim_half : 2 * dim_half + (i >> 1 & 1);
    const uint32_t v_lane = lds_v + v_row * L::VB + ((v_chunk ^ value_swizzle<VC, FP8>(v_row)) << 4) + 8 * (i & 1);

    f32x16 o[DT];
    // weights are exp2(x), x the logits + sub, sub = shift - m (0 before the first visible key); a step whose largest
    // exponent passes lim moves m
    float m = kNegInf, l = 0.0f, sub = 0.0f, lim = kNegInf;
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
        for (int j = 0; j < 16; j++) o[d][j] = 0.0f;
    f32x16 s[2];                                         // of the step whose weights come next
    bool seen_all = true;                                // no key of it is hidden
    FarSum fs{kNegInf, 0.0f};                            // apart: the row's sum, in place of l

    // ---- logits of a step from its scores: scaled, shifted, the hidden ones -infinity; the running maximum, which the
    // accumulators follow with a lag
    constexpr int kPieces = 16;                          // of a step's logits or weights: two of a lane's 32 each
    // the scales of a step's four groups, read before the products start
    constexpr int G = FP8 && EX ? 4 : 1;
    float mul[G], plus[G], inv[G], inv_next[G];
    const auto read_scales = [&](int n) {
        if constexpr (FP8 && EX) {
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const PageScale ps = lds.at[n & 3][g];
                inv_next[g % G] = ps.inv_v;
                mul[g % G] = fac * ps.k;
                plus[g % G] = sub + ps.log2_v;
            }
        }
    };
    const auto scale_piece = [&](int n, f32x16* x, float& top, int piece) {
        const int kt = piece / 8, j = piece % 8 * 2;
        if constexpr (FP8 && EX) {
            const int g = 2 * kt + j / 8;
            x[kt][j] = __builtin_fmaf(x[kt][j], mul[g % G], plus[g % G]);
            x[kt][j + 1] = __builtin_fmaf(x[kt][j + 1], mul[g % G], plus[g % G]);
        } else if constexpr (FP8) {
#pragma unroll
            for (int i = j; i < j + 2; i++) {
                const PageScale& ps = lds.at[n & 3][32 * kt + 8 * (i >> 2) + 4 * h + (i & 3)];
                x[kt][i] = __builtin_fmaf(x[kt][i], fac * ps.k, sub + ps.log2_v);
            }
        } else {
            x[kt][j] = __builtin_fmaf(x[kt][j], fac, sub);
            x[kt][j + 1] = __builtin_fmaf(x[kt][j + 1], fac, sub);
        }
        top = max3(top, x[kt][j], x[kt][j + 1]);
    };
    // (top: over the lane's logits of x)
    const auto settle = [&](int v, int n, f32x16* x, float top) {
        top = pair_max(top);
        uint32_t live = after(v) - v == 1 ? 0xFFFFu : ~0u;   // 16 keys of the lane a 32-key tile
        if constexpr (FP8) {
            constexpr int PER = EX ? 8 : 1;
#pragma unroll
            for (int j = 0; j < 32 / PER; j++)
                if (!lds.at[n & 3][EX ? j : 8 * (j >> 2) + 4 * h + (j & 3)].live) live &= ~((PER == 8 ? 0xFFu : 1u) << (PER * j));
        }
        seen_all = __all(live == ~0u && all_seen<TREE>(p, t, pos_lo, pos_hi, step_key(v), kStep));
        if (!seen_all) {
            hide_step<TREE>(p, t, pos, tok, step_key(v) + 4 * h, live, x);
            top = pair_max(fmaxf(max16(x[0]), max16(x[1])));
        }
        if (__builtin_expect(__any(top > lim), 0)) {      // wave-uniform, rare after the first steps
            const float mn = fmaxf(m, top - sub);
            const bool any = mn != kNegInf;
            const float al = any ? __builtin_amdgcn_exp2f(m - mn) : 1.0f;
            const float to = any ? T::kShiftUp - mn : 0.0f, by = to - sub;
            m = mn;
            sub = to;
            lim = any ? T::kShiftUp + kLag : kNegInf;
            l *= al;
#pragma unroll
            for (int kt = 0; kt < 2; kt++)
#pragma unroll
                for (int j = 0; j < 16; j++) x[kt][j] += by;
            if (n > 0) {
#pragma unroll
                for (int d = 0; d < DT; d++)
#pragma unroll
                    for (int j = 0; j < 16; j++) o[d][j] *= al;
            }
        }
        if constexpr (FP8 && CAREFUL) {
            if (apart) {
                const auto logit = [&](int j) {
                    return x[j >> 4][j & 15] - (sub + lds.at[n & 3][EX ? j >> 3 : 8 * (j >> 2) + 4 * h + (j & 3)].log2_v);
                };
                float most = kNegInf;
#pragma unroll
                for (int j = 0; j < 32; j++) most = fmaxf(most, logit(j));
                far_add<32>(fs, pair_max(most), T::kShiftUp, logit);
            }
        }
    };
    frag pw[4];
    float sums[4];                                       // of a 16-key group's weights
    const auto weigh_piece = [&](int n, int piece) {
        const int g = piece / 4, j = piece % 4 * 2;
        const float e0 = __builtin_amdgcn_exp2f(s[g >> 1][8 * (g & 1) + j]);
        const float e1 = __builtin_amdgcn_exp2f(s[g >> 1][8 * (g & 1) + j + 1]);
        if constexpr (FP8) {
            pw[g][j] = (_Float16)e0;
            pw[g][j + 1] = (_Float16)e1;
        } else {
            pw[g][j] = (__bf16)e0;
            pw[g][j + 1] = (__bf16)e1;
        }
        float part;
        if constexpr (FP8 && !EX) {
            const PageScale* ps = lds.at[n & 3] + 16 * g + 8 * (j >> 2) + 4 * h + (j & 3);
            part = __builtin_fmaf(e0, ps[0].inv_v, e1 * ps[1].inv_v);
        } else part = e0 + e1;
        sums[g] = j == 0 ? part : sums[g] + part;
        if (j == 6) {
            if constexpr (FP8 && EX) l = __builtin_fmaf(sums[g], inv[g % G], l);
            else l += sums[g];
            if constexpr (kSumEarly) asm volatile("" : "+v"(l));
        }
    };
    const auto add_values = [&](int n, auto side) {
        const uint32_t v_at = v_lane + (n & 1) * (int)sizeof(lds.v[0]);
        const auto load_v = [&](int n) {
            const int d = n % DT;
            const uint32_t at = chunk_at<VC>(v_at, (FP8 ? 2 : 4) * d) + n / DT * 16 * L::VB;
            RawFrag<T> x;
            if constexpr (FP8) x.w = __builtin_bit_cast(u32x2, read_transposed8(at));
            else {
                const u32x2 a = __builtin_bit_cast(u32x2, read_transposed16(at));
                const u32x2 b = __builtin_bit_cast(u32x2, read_transposed16(at + 8 * L::VB));
                x.w = u32x4{a.x, a.y, b.x, b.y};
            }
            return x;
        };
        const auto add = [&](int n, const frag& a) { o[n % DT] = T::mma(a, pw[n / DT], o[n % DT]); };
        if constexpr (!CAREFUL) {
            stream<4 * DT, T::kDepth, kPin, RawFrag<T>>(load_v, [&](int n, const RawFrag<T>& x) { add(n, operand(x)); }, side);
        } else {
            uint32_t odd = 0;
            stream<4 * DT, 2, false, RawFrag<T>>(load_v, [&](int n, RawFrag<T> x) {
                odd |= drop_nonfinite(x);
                add(n, operand(x));
            }, side);
            // rows that do see a value that is not finite get it in its dim: an infinity as the product of two large
            // values, a NaN as one of each sign (in two passes: of one instruction's products the large ones might cancel)
            if constexpr (!FP8) {
                if (__any(odd != 0)) {
#pragma unroll
                    for (int j = 0; j < 32; j++)
                        pw[j >> 3][j & 7] = (__bf16)(s[j >> 4][j & 15] != kNegInf ? 0x1p100f : 0.0f);
#pragma unroll 1
                    for (uint32_t sign = 0; sign <= 0x8000u; sign += 0x8000u)
                        stream<4 * DT, 2, false, RawFrag<T>>(load_v, [&](int n, RawFrag<T> x) {
                            keep_nonfinite(x, sign);
                            add(n, operand(x));
                        }, [](int) {});
                }
            }
        }
    };

    int n = 0;                                           // number of the step at v
    if (v < v1) {
        tile_ready();
        if (vn < v1) issue_keys(vn, 1);
        if (busy) {
            read_scales(0);
            multiply_keys<T, KS, L::KB, kPin>(k_lane, q, s, [](int) {});
            float top = kNegInf;
#pragma unroll
            for (int k = 0; k < kPieces; k++) scale_piece(0, s, top, k);
#pragma unroll
            for (int g = 0; g < G; g++) inv[g] = inv_next[g];
            settle(v, 0, s, top);
        }
    }
    while (vn < v1) {                                    // workgroup-uniform
        // ---- keys of the next step and values of this one are there; the places of this step's keys and of the last
        // step's values are free
        tile_ready();
        if constexpr (FP8) {
            walk.take(p);                                // the pages of step vp; those of vn are the ones before
            const int vq = after(vp);
            walk.find(p, step_key(vq < v1 ? vq : v), lane);
        }
        if (vp < v1) issue_keys(vp, n + 2);
        issue_values(vn, n + 1);
        if (busy) {                                      // wave-uniform
            f32x16 x[2];
            float top = kNegInf;
            if constexpr (kRaise) __builtin_amdgcn_s_setprio(1);
            constexpr int NK = 2 * KS / (FP8 ? 2 : 1), NV = 4 * DT;
            read_scales(n + 1);
            multiply_keys<T, KS, L::KB, kPin>(k_lane + ((n + 1) & 1) * (int)sizeof(lds.k[0]), q, x,
                                        [&](int i) { part_of<NK, kPieces>(i, [&](int k) { weigh_piece(n, k); }); });
            add_values(n, [&](int i) { part_of<NV, kPieces>(i, [&](int k) { scale_piece(n + 1, x, top, k); }); });
            if constexpr (kRaise) __builtin_amdgcn_s_setprio(0);
#pragma unroll
            for (int g = 0; g < G; g++) inv[g] = inv_next[g];
            settle(vn, n + 1, x, top);
#pragma unroll
            for (int kt = 0; kt < 2; kt++) s[kt] = x[kt];
        }
        v = vn;
        vn = vp;
        vp = after(vp);
        n++;
    }
    if (v < v1) {
        tile_ready();
        if (busy) {
#pragma unroll
            for (int k = 0; k < kPieces; k++) weigh_piece(n, k);
            add_values(n, [](int) {});
        }
    }

    if constexpr (!CAREFUL) {
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};         // a NaN anywhere makes one here
#pragma unroll
        for (int d = 0; d < DT; d++)
#pragma unroll
            for (int j = 0; j < 16; j++) sum[j & 3] += o[d][j];
        const float any = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        // a place that the last step does not use, nor the output rows below
        uint32_t* flag;
        if constexpr (FP8) flag = reinterpret_cast<uint32_t*>(lds.at[(n + 1) & 3]);
        else flag = reinterpret_cast<uint32_t*>(lds.v[(n + 1) & 1]);
        uint32_t saw = __any(busy && any != any) ? kSawNan : 0;
        if constexpr (FP8 && !kLookFirst<DK>) saw |= __any(sees_far(p, t, kvh, v0, v1)) ? kSawFar : 0;
        if (lane == 0) flag[w] = saw;
        __syncthreads();
        saw = flag[0] | flag[1] | flag[2] | flag[3];
        if (saw) return saw;
    }

    // ---- each lane holds runs of four dims of its rows.  They go through LDS, so that a store writes whole rows (16 bytes
    // a lane; as they are, 32 rows would get 16 bytes each a store), but for sums that meet what out holds
    const bool partial = p.splits > 1 && t.total > t.chunk;
    constexpr int OC = DV / 8, OW = OC < 16 ? OC : 16;   // chunks of an output row, and those that a row's swizzle permutes
    static_assert(kTileWaves * 32 * 16 * OC <= sizeof(lds.k) + (FP8 ? sizeof(lds.v) : 0), "rows of all waves fit");
    const uint32_t mine = lds_k + w * 32 * 16 * OC;
    if (CAREFUL) tile_ready();
    float ll = pair_sum(l);
    if constexpr (FP8 && CAREFUL) {
        if (apart) {
            ll = pair_sum(fs.l);
            const float mean = far_end(fs, m, ll);
#pragma unroll
            for (int d = 0; d < DT; d++)
#pragma unroll
                for (int j = 0; j < 16; j++) o[d][j] *= mean;
        }
    }
    const bool in = row_of >= 0;
    const int row = max(row_of, 0), tl = row_token(p, row), head = kvh * p.group + row - tl * p.group;
    const int64_t token = t.q0 + tl, id = token * p.hq + head;
    if (partial) {
        if (!in) return 0;
        if (h == 0) {
            float* ml = p.ws_ml + 2 * ((int64_t)t.split * p.total_q * p.hq + id);
            ml[0] = m - T::kShiftUp + kShift;         // the join takes kShift off
            ml[1] = ll;
        }
        float* dst = p.ws_o + ((int64_t)t.split * p.total_q * p.hq + id) * p.hs + 4 * h;
#pragma unroll
        for (int d = 0; d < DT; d++)
#pragma unroll
            for (int a = 0; a < 4; a++)
                if (EX || 32 * d + 8 * a + 4 * h < p.hs)
                    *reinterpret_cast<f32x4*>(dst + 32 * d + 8 * a) =
                        f32x4{o[d][4 * a], o[d][4 * a + 1], o[d][4 * a + 2], o[d][4 * a + 3]};
        return 0;
    }
    RowEnd end{0.0f, 0.0f, 0.0f};
    if (in) {
        end = row_end_shifted<T>(p, token, head, m, ll);
        if (h == 0 && p.lse) p.lse[token * p.lse_ts + head] = end.lse;
    }
    uint16_t* dst = p.out + token * p.o_ts + (int64_t)head * p.o_hs;
    if (accumulates(p)) {
        if (!in) return 0;
#pragma unroll
        for (int d = 0; d < DT; d++)
#pragma unroll
            for (int a = 0; a < 4; a++)
                if (EX || 32 * d + 8 * a + 4 * h < p.hs)
                    write_dims(p, end, dst + 32 * d + 8 * a + 4 * h, o[d][4 * a], o[d][4 * a + 1], o[d][4 * a + 2],
                               o[d][4 * a + 3]);
        return 0;
    }
    if (!busy) return 0;                             // wave-uniform
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
        for (int a = 0; a < 4; a++)
            write_lds(mine + c * 16 * OC + (((4 * d + a) ^ (c & (OW - 1))) << 4) + 8 * h,
                      u32x2{pack_bf16x2(o[d][4 * a] * end.scale, o[d][4 * a + 1] * end.scale),
                            pack_bf16x2(o[d][4 * a + 2] * end.scale, o[d][4 * a + 3] * end.scale)});
    const uint64_t to = in ? reinterpret_cast<uint64_t>(dst) : 0;
    wave_lds_ready();
#pragma unroll
    for (int k = 0; k < 32 * OC / kWave; k++) {
        const int from = (k * kWave + lane) / OC, chunk = (k * kWave + lane) % OC;
        const u32x4 x = read_lds<u32x4>(mine + from * 16 * OC + ((chunk ^ (from & (OW - 1))) << 4));
        const uint64_t at = (uint64_t)(uint32_t)__shfl((int)(to >> 32), from) << 32 | (uint32_t)__shfl((int)to, from);
        if (at != 0 && (EX || 8 * chunk < p.hs)) *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(at) + 8 * chunk) = x;
    }
    return 0;
}

template <typename T, int DK, int DV, bool EX, bool TREE, typename P>
__device__ __forceinline__ void attend_tile(const P& p, const RowTile& t, int kvh, int v0, int v1, StepLds<T, DK, DV, EX>& lds) {
    uint32_t saw = 0;
    if constexpr (T::kFp8 && kLookFirst<DK>) saw = __syncthreads_or(sees_far(p, t, kvh, v0, v1)) ? kSawFar : 0;
    if (!saw) saw = attend_once<T, DK, DV, EX, TREE, false>(p, t, kvh, v0, v1, false, lds);
    if (saw) {
        __syncthreads();
        attend_once<T, DK, DV, EX, TREE, true>(p, t, kvh, v0, v1, (saw & kSawFar) != 0, lds);
    }
}

// The kv head and work unit of workgroup wg.  Workgroups of a head get numbers
// that are equal modulo 8 (or its divisor): one XCD, whose L2 then serves a
// request's keys to all of its row tiles.
__device__ __forceinline__ bool head_and_unit(const AttnParams& p, uint32_t wg, uint32_t& kvh, uint32_t& unit) {
    const uint32_t units = (uint32_t)p.units, hk = (uint32_t)p.hk;
    if (hk % 8 == 0) {
        const uint32_t part = wg / (8 * units), in = wg - part * 8 * units;
        kvh = part * 8 + in % 8;
        unit = in / 8;
    } else {
        unit = wg / hk;
        kvh = wg - unit * hk;
    }
    return kvh < hk;
}

}  // namespace gcache
