// rope_append.hip -- new tokens into the paged e4m3 cache: keys rotated, both
// sides quantized with a scale for each page, side and head; and the rotated
// queries of the same tokens.
//
// Mathematics.  A page's scale is its largest magnitude over 448 when the page
// begins in this call.  When it holds older tokens the scale may only grow, and
// by powers of two, which moves older codes by a change of exponent: a code
// that was rounded once is not rounded again (but for subnormal numbers).
// So appending one token at a time loses no more than a factor below two of the
// scale, and the result does not depend on how a page's tokens fall into calls
// otherwise.
//
// One launch.  The first workgroups own a page and as many heads as fit the
// lanes (16 values a lane): no two of them write the same scale, so there are
// no atomics on memory, and the order of tokens does not matter.  The page's
// maximum over its tokens is joined in LDS; the tokens' values stay in
// registers meanwhile (pages of up to four rounds; larger ones are read twice,
// the second time from L2).  The other workgroups rotate queries, a wave a
// token.
// Bound by memory: 4 x 4096 tokens, 32 query and 8 kv heads of 128, take 85 us
// with pages of 16 tokens, 81 with 64, 83 with 128 (4.9 TB/s of reads and
// writes).  Registers for four rounds of rows leave fewer waves a SIMD; held to
// 128 of them for four waves it takes 102 us.
#include "attention_device.h"
#include "fp8_scale.h"

namespace gcache {

struct Turn {
    float c[8], s[8];
};
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// The 16 values of a row that unit u of head_size / 16 holds: two runs of 8.
// Pairs are value i of the first run with value i of the second, or neighbours.
struct UnitDims {
    int d0, d1;
    bool turned;
};
template <bool INTER>
__device__ __forceinline__ UnitDims unit_dims(const AppendParams& p, int u) {
    const bool turned = 16 * u < p.rot;
    if (turned && !INTER) return UnitDims{8 * u, p.rot / 2 + 8 * u, true};
    return UnitDims{16 * u, 16 * u + 8, turned};
}
// The angles of unit u at table row r; false: the row is outside the table.
__device__ __forceinline__ bool load_turn(const AppendParams& p, int64_t r, int u, bool turned, Turn& t) {
    if (p.rot == 0) return true;
    if (r < 0 || r >= p.max_pos) return false;
    if (!turned) return true;
    if (p.cs_bf16) {
        const uint16_t* at = static_cast<const uint16_t*>(p.cos_sin) + r * p.cs_stride + 8 * u;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            t.c[i] = __uint_as_float((uint32_t)at[i] << 16);
            t.s[i] = __uint_as_float((uint32_t)at[p.rot / 2 + i] << 16);
        }
    } else {
        const float* at = static_cast<const float*>(p.cos_sin) + r * p.cs_stride + 8 * u;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const f32x4 c = *reinterpret_cast<const f32x4_a4*>(at + i), s = *reinterpret_cast<const f32x4_a4*>(at + p.rot / 2 + i);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                t.c[i + j] = c[j];
                t.s[i + j] = s[j];
            }
        }
    }
    return true;
}
__device__ __forceinline__ void unpack(const u32x4& a, const u32x4& b, float* x) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        x[2 * i] = bf16_lo(a[i]);
        x[2 * i + 1] = bf16_hi(a[i]);
        x[8 + 2 * i] = bf16_lo(b[i]);
        x[9 + 2 * i] = bf16_hi(b[i]);
    }
}
// Each product and each sum is rounded by itself.
template <bool INTER>
__device__ __forceinline__ void rotate(const UnitDims& d, const Turn& t, bool ok, float* x) {
    if (d.turned) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            float &a = INTER ? x[2 * i] : x[i], &b = INTER ? x[2 * i + 1] : x[8 + i];
            const float ra = a * t.c[i] - b * t.s[i], rb = b * t.c[i] + a * t.s[i];
            a = ra;
            b = rb;
        }
    }
#pragma unroll
    for (int i = 0; i < 16; i++) x[i] = ok ? x[i] : 0.0f;
}
__device__ __forceinline__ void store_bf16(uint16_t* row, const UnitDims& d, const float* x) {
    *reinterpret_cast<u32x4*>(row + d.d0) =
        u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
    *reinterpret_cast<u32x4*>(row + d.d1) =
        u32x4{pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]), pack_bf16x2(x[14], x[15])};
}

// The request of a packed token or of a page unit: the largest b whose
// first(b) <= at, for non-decreasing first.  64 requests a step.
template <typename First>
__device__ __forceinline__ int find_request64(int batch, int64_t at, int lane, First first) {
    int lo = 0, n = batch;
    while (n > 1) {
        const int step = (n + kWave - 1) / kWave, i = lane * step;
        const uint64_t below = __ballot(i < n && first(lo + min(i, n - 1)) <= at);
        const int j = max(__popcll(below) - 1, 0);
        lo += j * step;
        n = min(step, n - j * step);
    }
    return lo;
}

struct Request {
    int b, q0, qlen, ctx, seq;
};
__device__ __forceinline__ int token_start(const AppendParams& p, int b) { return min(max(p.qs[b], 0), p.num_tokens); }
__device__ __forceinline__ Request request(const AppendParams& p, int b) {
    Request r;
    r.b = b;
    r.q0 = token_start(p, b);
    r.qlen = max(token_start(p, b + 1) - r.q0, 0);
    r.seq = max(p.lens[b], 0);
    r.ctx = r.seq - r.qlen;
    return r;
}

// ---------------------------------------------------------------------------
// A page: its new tokens [pos0, pos1), its older ones before them.
// ---------------------------------------------------------------------------
constexpr int kKeep = 4;                                 // rounds of rows that stay in registers

template <bool INTER>
__device__ __forceinline__ void append_page(const AppendParams& p, int64_t wg, uint32_t* s_max) {
    const int lane = lane_id(), w = wave_id();
    const int chunk = (int)(wg % p.head_chunks);
    const int64_t unit = wg / p.head_chunks;
    const int bs = (int)p.div.size;
    Request r;
    int page;
    if (p.by_token) {
        r = request(p, __builtin_amdgcn_readfirstlane(find_request64(p.batch, unit, lane, [&](int b) { return (int64_t)token_start(p, b); })));
        const int64_t i = unit - r.q0;
        if (i < 0 || i >= r.qlen) return;
        const int pos = r.ctx + (int)i;
        if (pos < 0 || (i > 0 && pos % bs != 0)) return; // the page's first new token does the work
        page = pos / bs;
    } else {
        const auto first = [&](int b) { return page_unit(token_start(p, b), b, bs); };
        r = request(p, __builtin_amdgcn_readfirstlane(find_request64(p.batch, unit, lane, first)));
        const int64_t at = max(r.ctx, 0) / bs + (unit - first(r.b));
        if (r.qlen == 0 || unit < first(r.b) || at * bs >= r.seq) return;
        page = (int)at;
    }
    const int base = page * bs;                          // its first position, below seq
    const int pos0 = max(max(r.ctx, 0), base), n = (int)min((int64_t)r.seq, (int64_t)base + bs) - pos0;
    const int kept = pos0 - base;
    const int id = page < p.bt_stride ? p.block_table[(int64_t)r.b * p.bt_stride + page] : -1;
    const bool there = id >= 0 && id < p.num_blocks;
    if (!there && !p.ko) return;

    // lanes: unit u of a row, head hh of the chunk, row rs of the wave's rows of a round
    const int units = p.hs / 16, u = lane % units, grp = lane / units;
    const int rs = grp / p.chunk_heads, hh = grp - rs * p.chunk_heads, head = chunk * p.chunk_heads + hh;
    const bool on = rs < p.wave_rows && head < p.hk;
    const int round = kWavesPerBlock * p.wave_rows, rounds = (n + round - 1) / round;
    const int row0 = w * p.wave_rows + rs;               // of each round
    const UnitDims d = unit_dims<INTER>(p, u);

    for (int i = threadIdx.x; i < 2 * kWave; i += kBlockThreads) s_max[i] = 0;
    float old[2] = {0.0f, 0.0f};
    float* scale_at = p.scales + (int64_t)(there ? id : 0) * p.s_block + (int64_t)(on ? head : 0) * p.s_head;
    if (there && on && kept > 0) {
        old[0] = page_scale(scale_at[0]);
        old[1] = page_scale(scale_at[p.s_side]);
    }
    const auto load_key = [&](int row, float* x) {
        const int64_t tok = r.q0 + (pos0 - r.ctx) + row;
        const uint16_t* at = p.k + tok * p.k_ts + head * p.k_hs;
        const u32x4 a = *reinterpret_cast<const u32x4*>(at + d.d0), b = *reinterpret_cast<const u32x4*>(at + d.d1);
        Turn t;
        const bool ok = load_turn(p, p.positions ? p.positions[tok] : pos0 + row, u, d.turned, t);
        unpack(a, b, x);
        rotate<INTER>(d, t, ok, x);
    };
    struct Raw {
        u32x4 a, b;
    };
    const auto load_value = [&](int row) {
        const uint16_t* at = p.v + (int64_t)(r.q0 + (pos0 - r.ctx) + row) * p.v_ts + head * p.v_hs + 16 * u;
        return Raw{*reinterpret_cast<const u32x4*>(at), *reinterpret_cast<const u32x4*>(at + 8)};
    };
    const auto largest = [](const float* x) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i++) m = fmaxf(m, fabsf(x[i]));
        return m;
    };
    float kx[kKeep][16];
    Raw vx[kKeep];
    float top[2] = {0.0f, 0.0f};
    if (on && rounds <= kKeep) {
#pragma unroll
        for (int i = 0; i < kKeep; i++) {
            const int row = i * round + row0;
            if (row < n) {
                load_key(row, kx[i]);
                if (there) vx[i] = load_value(row);
            }
        }
#pragma unroll
        for (int i = 0; i < kKeep; i++) {
            if (i * round + row0 < n) {
                float v[16];
                top[0] = fmaxf(top[0], largest(kx[i]));
                if (there) {
                    unpack(vx[i].a, vx[i].b, v);
                    top[1] = fmaxf(top[1], largest(v));
                }
            }
        }
    } else if (on) {
        for (int row = row0; row < n; row += round) {
            float x[16], v[16];
            load_key(row, x);
            top[0] = fmaxf(top[0], largest(x));
            if (there) {
                const Raw y = load_value(row);
                unpack(y.a, y.b, v);
                top[1] = fmaxf(top[1], largest(v));
            }
        }
    }
    __syncthreads();
    if (on) {                                            // magnitudes order as their bits
        atomicMax(&s_max[hh], __float_as_uint(top[0]));
        atomicMax(&s_max[kWave + hh], __float_as_uint(top[1]));
    }
    __syncthreads();
    if (!on) return;
    float inv[2], shrink[2];
#pragma unroll
    for (int side = 0; side < 2; side++) {
        const float need = append_need(__uint_as_float(s_max[side * kWave + hh]));
        const int times = kept > 0 ? doublings(old[side], need) : 0;
        const float scale = kept > 0 ? ldexpf(old[side], times) : need;
        inv[side] = 1.0f / scale;
        shrink[side] = ldexpf(1.0f, -min(times, 30));    // 448 / 2^30 rounds to 0 as any smaller number
        if (there && w == 0 && rs == 0 && u == 0 && (kept == 0 || times > 0)) scale_at[side * p.s_side] = scale;
    }
    uint8_t* cache = p.cache + (int64_t)(there ? id : 0) * p.block_stride + head * p.head_stride;
    const auto put8 = [&](uint8_t* at, const float* x, float by) {
        uint32_t a = put_e4m3x2<false>(0, x[0] * by, x[1] * by), b = put_e4m3x2<false>(0, x[4] * by, x[5] * by);
        a = put_e4m3x2<true>(a, x[2] * by, x[3] * by);
        b = put_e4m3x2<true>(b, x[6] * by, x[7] * by);
        *reinterpret_cast<u32x2*>(at) = u32x2{a, b};
    };
    const auto write = [&](int row, const float* x, const Raw& y) {
        if (p.ko) store_bf16(p.ko + (int64_t)(r.q0 + (pos0 - r.ctx) + row) * p.ko_ts + head * p.ko_hs, d, x);
        if (!there) return;
        uint8_t* at = cache + (int64_t)(kept + row) * p.token_stride;
        put8(at + d.d0, x, inv[0]);
        put8(at + d.d1, x + 8, inv[0]);
        float v[16];
        unpack(y.a, y.b, v);
        put8(at + p.side_stride + 16 * u, v, inv[1]);
        put8(at + p.side_stride + 16 * u + 8, v + 8, inv[1]);
    };
    if (rounds <= kKeep) {
#pragma unroll
        for (int i = 0; i < kKeep; i++)
            if (i * round + row0 < n) write(i * round + row0, kx[i], vx[i]);
    } else {
        for (int row = row0; row < n; row += round) {
            float x[16];
            load_key(row, x);
            Raw y{};
            if (there) y = load_value(row);
            write(row, x, y);
        }
    }
    // older codes, where the scale has grown
    if (!there || kept == 0) return;
#pragma unroll
    for (int side = 0; side < 2; side++) {
        if (shrink[side] == 1.0f) continue;
        for (int row = row0; row < kept; row += round) {
            u32x4* at = reinterpret_cast<u32x4*>(cache + row * p.token_stride + side * p.side_stride + 16 * u);
            u32x4 x = *at;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const f32x2 a = e4m3x2_f32<false>(x[i]), b = e4m3x2_f32<true>(x[i]);
                x[i] = put_e4m3x2<true>(put_e4m3x2<false>(0, a.x * shrink[side], a.y * shrink[side]), b.x * shrink[side],
                                        b.y * shrink[side]);
            }
            *at = x;
        }
    }
}

// ---------------------------------------------------------------------------
// Queries: heads of a token, and the keys of tokens that have no page.
// ---------------------------------------------------------------------------
template <bool INTER>
__device__ __forceinline__ void rotate_rows(const AppendParams& p, const uint16_t* x, uint16_t* y, int64_t x_hs, int64_t y_hs,
                                            int head0, int heads, int64_t r, int lane) {
    const int units = p.hs / 16, per = kWave / units, u = lane % units, grp = lane / units;
    if (grp >= per) return;
    const UnitDims d = unit_dims<INTER>(p, u);
    Turn t;
    const bool ok = load_turn(p, r, u, d.turned, t);
#pragma unroll 4
    for (int h = head0 + grp; h < heads; h += per) {
        float v[16];
        unpack(*reinterpret_cast<const u32x4*>(x + h * x_hs + d.d0), *reinterpret_cast<const u32x4*>(x + h * x_hs + d.d1), v);
        rotate<INTER>(d, t, ok, v);
        store_bf16(y + h * y_hs, d, v);
    }
}
template <bool INTER>
__device__ __forceinline__ void rotate_token(const AppendParams& p, int64_t wave) {
    const int lane = lane_id();
    const int64_t tok = wave / p.q_waves;
    const int part = (int)(wave - tok * p.q_waves);
    if (tok >= p.num_tokens) return;
    const Request r = request(p, __builtin_amdgcn_readfirstlane(find_request64(p.batch, tok, lane, [&](int b) { return (int64_t)token_start(p, b); })));
    if (tok < r.q0 || tok >= r.q0 + r.qlen) return;
    const int pos = r.ctx + (int)(tok - r.q0);
    const int64_t row = p.positions ? p.positions[tok] : pos;
    if (p.hq) {
        const int each = (p.hq + p.q_waves - 1) / p.q_waves;
        rotate_rows<INTER>(p, p.q + tok * p.q_ts, p.qo + tok * p.qo_ts, p.q_hs, p.qo_hs, part * each, min(p.hq, part * each + each),
                           row, lane);
    }
    if (pos < 0 && p.ko && part == 0)
        rotate_rows<INTER>(p, p.k + tok * p.k_ts, p.ko + tok * p.ko_ts, p.k_hs, p.ko_hs, 0, p.hk, row, lane);
}

template <bool INTER>
__global__ __launch_bounds__(kBlockThreads) void k_rope_append(AppendParams p, int64_t wg0) {
    __shared__ uint32_t s_max[2 * kWave];
    const int64_t wg = wg0 + blockIdx.x;
    if (wg < p.page_groups) append_page<INTER>(p, wg, s_max);
    else rotate_token<INTER>(p, (wg - p.page_groups) * kWavesPerBlock + wave_id());
}

hipError_t launch_rope_append(const AppendParams& in, hipStream_t s) {
    AppendParams p = in;
    const int units = p.hs / 16, per = kWave / units;    // (row, head) pairs of a wave
    // Units: the pages that the requests' tokens can lie in, a bound that the
    // host knows, or the tokens where those are fewer (decoding).
    const int64_t pages = page_unit(p.num_tokens, p.batch, p.div.size);
    p.by_token = p.num_tokens <= pages;
    // Heads of a workgroup: as many as a wave holds, or for large pages so many
    // that a page's rows take kKeep rounds (pages of 128 tokens, 8 heads of 128:
    // 123 us with all heads, whose rows 128 workgroups then read twice).
    const int64_t rows = p.by_token ? 1 : (p.div.size + kKeep * kWavesPerBlock - 1) / (kKeep * kWavesPerBlock);
    p.chunk_heads = (int32_t)(per / rows > 1 ? per / rows : 1);
    if (p.chunk_heads > p.hk) p.chunk_heads = p.hk;
    p.wave_rows = per / p.chunk_heads;
    p.head_chunks = (p.hk + p.chunk_heads - 1) / p.chunk_heads;
    p.page_groups = (p.by_token ? p.num_tokens : pages) * p.head_chunks;
    // a wave a token, and more of them for few tokens
    const int most = (p.hq + per - 1) / per;
    p.q_waves = p.num_tokens >= 2048 || most < 1 ? 1 : most;
    const int64_t waves = p.num_tokens * (int64_t)p.q_waves;
    const int64_t groups = p.page_groups + (waves + kWavesPerBlock - 1) / kWavesPerBlock;
    return launch_span(p.interleaved ? k_rope_append<true> : k_rope_append<false>, groups, kBlockThreads, s, true, true, p);
}

}  // namespace gcache
