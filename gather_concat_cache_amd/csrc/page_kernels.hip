// page_kernels.hip -- ownership of cache pages on the device: forking,
// extending and freeing requests, compacting the live pages, copying pages.
//
// State: block table rows with their lengths, and a reference count for each
// page; a page is free when its count is 0.  Pages are handed out lowest id
// first in the order of the requests of a call, so results do not depend on
// the order in which workgroups run.  A page that is not full belongs to one
// row only: a fork shares the full pages and copies the partial one.
//
// The bookkeeping is a few kilobytes and latency bound (one workgroup, a
// handful of dependent steps); the copies are HBM bound streams and run one
// page a workgroup and step, all of a thread's loads before its stores (1.39 GB
// of a compaction in 257 us, 5.4 TB/s; a plain copy without a loop reaches 6.1).
#include "gcache_operators.h"

namespace gcache {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / kWave;

__device__ __forceinline__ int pages_of(int len, int bs) { return len <= 0 ? 0 : (len - 1) / bs + 1; }

// Workgroup-wide barrier that also orders global writes and atomics.
__device__ __forceinline__ void plan_sync() {
    __threadfence();
    __syncthreads();
}

// Exclusive sum of v over the workgroup's threads in order; *total gets the
// sum.  Two barriers; s holds kPlanWaves values.
__device__ __forceinline__ int64_t wg_exclusive(int v, int64_t* s, int64_t* total) {
    const int lane = lane_id(), w = wave_id();
    int64_t x = v;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int64_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == kWave - 1) s[w] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kPlanWaves; i++) {
        before += i < w ? s[i] : 0;
        all += s[i];
    }
    *total = all;
    return before + x - v;
}

// Tokens the row of request f would get, -1: refused.
template <bool FORK>
__device__ __forceinline__ int grant_len(const GrantParams& p, int row, int arg) {
    const int rows = p.t.num_rows;
    if (row < 0 || row >= rows) return -1;
    const int have = p.t.lens[row];
    int len = arg;
    if (FORK) {                                          // arg: the parent row
        if (arg < 0 || arg >= rows || arg == row || have != 0) return -1;
        len = p.t.lens[arg];
    } else if (have < 0 || len < have) {
        return -1;
    }
    return len >= 0 && pages_of(len, p.t.block_size) <= p.t.stride ? len : -1;
}

// The lowest `want` free pages (all of them when there are fewer) into
// free_ids; returns how many there are.
__device__ __forceinline__ int64_t list_free(const GrantParams& p, int64_t want, int64_t* s_scan) {
    constexpr int kIds = 4;
    int64_t found = 0;
    for (int64_t b0 = 0; b0 < p.t.num_blocks && found < want; b0 += kIds * kPlanThreads) {
        const int64_t id0 = b0 + kIds * threadIdx.x;
        bool fr[kIds];
        int cnt = 0;
#pragma unroll
        for (int i = 0; i < kIds; i++) {
            fr[i] = id0 + i < p.t.num_blocks && p.t.refs[id0 + i] == 0;
            cnt += fr[i];
        }
        int64_t sum;
        int64_t at = found + wg_exclusive(cnt, s_scan, &sum);
#pragma unroll
        for (int i = 0; i < kIds; i++)
            if (fr[i]) p.free_ids[at++] = (int)(id0 + i);
        found += sum;
    }
    return found;
}

// Pages of the requests up to one as its entry of upto: -1 when they are more
// than there are pages, so that no clipped number looks like one that fits.
// (Sums are 64 bits; a request's own need is at most INT32_MAX.)
__device__ __forceinline__ int upto_entry(const GrantParams& p, int64_t upto) {
    return upto > p.t.num_blocks ? -1 : (int)upto;
}

// One workgroup, at most a request a thread: which requests are valid (the
// lowest-numbered one of a row wins), how many pages each needs, the lowest
// free pages for all of them.  FORK: a = parent rows, b = child rows; else a =
// rows, b = new lengths.  Grants are decided in request order: request i is
// granted when the pages of requests 0..i all fit the free ones.  Everything
// stays in registers and LDS: three dependent memory round trips (extending
// and freeing 256 rows: 25 us, against 31 with the form below).
template <bool FORK>
__global__ __launch_bounds__(kPlanThreads) void k_grant_small(GrantParams p, int64_t) {
    __shared__ int64_t s_scan[kPlanWaves];
    constexpr int kSlots = 2 * kPlanThreads;             // 2048: the hash takes 11 bits
    __shared__ int s_row[kSlots], s_first[kSlots];
    const int f = threadIdx.x, bs = p.t.block_size;
    const int a = f < p.n ? p.a[f] : -1, b = f < p.n ? p.b[f] : -1;
    const int row = FORK ? b : a;
    int len = f < p.n ? grant_len<FORK>(p, row, FORK ? a : b) : -1;
    // the lowest request of each row, by a hash table at most half full
    for (int i = f; i < kSlots; i += kPlanThreads) {
        s_row[i] = -1;
        s_first[i] = INT32_MAX;
    }
    __syncthreads();
    int slot = 0;
    if (len >= 0) {
        slot = (int)((uint32_t)row * 2654435761u >> 21);
        for (;;) {                                       // ends: more slots than rows
            const int old = atomicCAS(&s_row[slot], -1, row);
            if (old == -1 || old == row) break;
            slot = (slot + 1) & (kSlots - 1);
        }
        atomicMin(&s_first[slot], f);
    }
    __syncthreads();
    if (len >= 0 && s_first[slot] != f) len = -1;
    int need = 0;
    if (len >= 0) need = FORK ? len % bs != 0 : pages_of(len, bs) - pages_of(p.t.lens[row], bs);
    int64_t all;
    const int64_t upto = wg_exclusive(need, s_scan, &all) + need;
    const int64_t found = list_free(p, all, s_scan);
    if (f < p.n) {
        const bool ok = len >= 0 && upto <= found;
        p.status[f] = ok;
        p.len[f] = ok ? len : -1;
        p.upto[f] = upto_entry(p, upto);
    }
}

// The same for any number of requests, with the claims of rows in memory.
template <bool FORK>
__global__ __launch_bounds__(kPlanThreads) void k_grant_plan(GrantParams p, int64_t) {
    __shared__ int64_t s_scan[kPlanWaves];
    const int tid = threadIdx.x, bs = p.t.block_size, rows = p.t.num_rows;
    const auto row_of = [&](int f) { return FORK ? p.b[f] : p.a[f]; };
    for (int f = tid; f < p.n; f += kPlanThreads) {
        const int r = row_of(f);
        if (r >= 0 && r < rows) atomicExch(&p.claim[r], INT32_MAX);
    }
    plan_sync();
    const auto valid_len = [&](int f) { return grant_len<FORK>(p, row_of(f), FORK ? p.a[f] : p.b[f]); };
    for (int f = tid; f < p.n; f += kPlanThreads)
        if (valid_len(f) >= 0) atomicMin(&p.claim[row_of(f)], f);
    plan_sync();
    int64_t need_all = 0;
    for (int f0 = 0; f0 < p.n; f0 += kPlanThreads) {     // workgroup-uniform
        const int f = f0 + tid;
        int need = 0;
        if (f < p.n) {
            int len = valid_len(f);
            if (len >= 0 && __hip_atomic_load(&p.claim[row_of(f)], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != f)
                len = -1;
            if (len >= 0)
                need = FORK ? len % bs != 0 : pages_of(len, bs) - pages_of(p.t.lens[row_of(f)], bs);
            p.len[f] = len;
        }
        int64_t sum;
        const int64_t upto = need_all + wg_exclusive(need, s_scan, &sum) + need;
        if (f < p.n) p.upto[f] = upto_entry(p, upto);
        need_all += sum;
    }
    const int64_t found = list_free(p, need_all, s_scan);
    for (int f = tid; f < p.n; f += kPlanThreads) {
        const bool ok = p.len[f] >= 0 && p.upto[f] >= 0 && p.upto[f] <= found;
        p.status[f] = ok;
        if (!ok) p.len[f] = -1;
    }
}

// First page in free_ids of a granted request f (its need is upto[f] - upto[f - 1]; both fit).
__device__ __forceinline__ int first_page(const GrantParams& p, int f) { return f > 0 ? p.upto[f - 1] : 0; }

// The row of fork f, by one workgroup.
__device__ __forceinline__ void fork_row(const GrantParams& p, int f) {
    const int len = p.len[f];
    if (len < 0) return;
    const int full = len / p.t.block_size;
    const int32_t* src = p.t.table + (int64_t)p.a[f] * p.t.stride;
    int32_t* dst = p.t.table + (int64_t)p.b[f] * p.t.stride;
    for (int i = threadIdx.x; i < full; i += kBlockThreads) {
        const int id = src[i];
        dst[i] = id;
        if (id >= 0 && id < p.t.num_blocks) atomicAdd(&p.t.refs[id], 1);
    }
    if (threadIdx.x == 0) {
        if (len % p.t.block_size) {
            const int id = p.free_ids[first_page(p, f)];
            dst[full] = id;
            atomicAdd(&p.t.refs[id], 1);
        }
        p.t.lens[p.b[f]] = len;
    }
}

__global__ __launch_bounds__(kBlockThreads) void k_extend_rows(GrantParams p, int64_t wg0) {
    const int64_t f = wg0 + blockIdx.x;
    if (f >= p.n) return;
    const int len = p.len[f];
    if (len < 0) return;
    const int row = p.a[f], first = first_page(p, (int)f), need = p.upto[f] - first;
    const int have = pages_of(len, p.t.block_size) - need;
    int32_t* dst = p.t.table + (int64_t)row * p.t.stride;
    for (int i = threadIdx.x; i < need; i += kBlockThreads) {
        const int id = p.free_ids[first + i];
        dst[have + i] = id;
        atomicAdd(&p.t.refs[id], 1);
    }
    if (threadIdx.x == 0) p.t.lens[row] = len;
}

// One workgroup a listed row.  A row listed twice is freed once: each table
// entry is taken by exchange, and a workgroup that already reads length 0
// leaves the row to the other, so nothing has to be ordered between the two.
__global__ __launch_bounds__(kBlockThreads) void k_free_rows(PageTable t, const int32_t* rows, int32_t n) {
    const int row = rows[blockIdx.x];
    if (row < 0 || row >= t.num_rows) return;
    const int len = __hip_atomic_load(&t.lens[row], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int pages = (int)min((int64_t)pages_of(len, t.block_size), t.stride);
    int32_t* e = t.table + (int64_t)row * t.stride;
    for (int i = threadIdx.x; i < pages; i += kBlockThreads) {
        const int id = atomicExch(&e[i], -1);
        if (id >= 0 && id < t.num_blocks && atomicAdd(&t.refs[id], -1) <= 0) atomicAdd(&t.refs[id], 1);
    }
    __syncthreads();                                     // every thread has read the length
    if (threadIdx.x == 0) __hip_atomic_store(&t.lens[row], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------------------
// page copies: (cache, pair) items over a fixed grid
// ---------------------------------------------------------------------------
template <typename V>
__device__ __forceinline__ void copy_page(const uint8_t* __restrict__ src, uint8_t* __restrict__ dst, int64_t bytes) {
    constexpr int U = 6;                                 // loads in flight a thread
    const int64_t n = bytes / (int64_t)sizeof(V);
    const V* s = reinterpret_cast<const V*>(src);
    V* d = reinterpret_cast<V*>(dst);
    for (int64_t i0 = threadIdx.x; i0 < n; i0 += U * kBlockThreads) {
        V v[U];
#pragma unroll
        for (int u = 0; u < U; u++)
            if (i0 + u * kBlockThreads < n) v[u] = __builtin_nontemporal_load(s + i0 + u * kBlockThreads);
#pragma unroll
        for (int u = 0; u < U; u++)
            if (i0 + u * kBlockThreads < n) __builtin_nontemporal_store(v[u], d + i0 + u * kBlockThreads);
    }
    for (int64_t i = n * (int64_t)sizeof(V) + threadIdx.x; i < bytes; i += kBlockThreads) dst[i] = src[i];
}

struct PairList {                // explicit pairs, or a compaction's moves
    const int32_t* src;
    const int32_t* dst;
    const int32_t* count;        // device count, or nullptr: n
    int64_t n;
};
struct CopyParams {
    CacheList c;
    PairList l;
};

template <typename V>
__global__ __launch_bounds__(kBlockThreads) void k_copy_pages(CopyParams p, int64_t wg0) {
    const int64_t n = p.l.count ? *p.l.count : p.l.n;
    const int64_t items = n * p.c.n, step = gridDim.x;
    for (int64_t it = wg0 + blockIdx.x; it < items; it += step) {
        const int64_t k = it % n;
        const int cache = (int)(it / n);
        const int64_t a = p.l.src[k], b = p.l.dst[k];
        if (a < 0 || a >= p.c.num_blocks || b < 0 || b >= p.c.num_blocks || a == b) continue;
        uint8_t* base = p.c.base[cache];
        copy_page<V>(base + a * p.c.block_stride, base + b * p.c.block_stride, p.c.page_bytes);
    }
}

// The rows of the forks, then their partial pages.  Up to kForkBlock
// consecutive forks of one cache go to a workgroup, which reads a page once for
// the forks of the same parent that follow each other: samples of one prompt
// then cost one read and their writes (one 8-fold fork of 64 prompts over 32
// caches: 101 us against 174 us with a read for every copy).
constexpr int kForkBlock = 8;
struct ForkCopyParams {
    CacheList c;
    GrantParams g;
    int32_t block;               // forks of a workgroup, <= kForkBlock
    bool rows;                   // this launch also does the rows
};

template <typename V>
__global__ __launch_bounds__(kBlockThreads) void k_fork_apply(ForkCopyParams p, int64_t wg0) {
    constexpr int U = 6;                                 // loads in flight a thread
    __shared__ int s_src[kForkBlock], s_dst[kForkBlock];
    const GrantParams& g = p.g;
    if (p.rows)
        for (int64_t f = wg0 + blockIdx.x; f < g.n; f += gridDim.x) fork_row(g, (int)f);
    const int64_t blocks = (g.n + p.block - 1) / p.block, items = blocks * p.c.n;
    const int tid = threadIdx.x;
    for (int64_t it = wg0 + blockIdx.x; it < items; it += gridDim.x) {   // workgroup-uniform
        const int64_t k0 = it % blocks * p.block;
        __syncthreads();
        if (tid < p.block) {
            int src = -1, dst = -1;
            const int64_t k = k0 + tid;
            const int len = k < g.n ? g.len[k] : -1;
            if (len >= 0 && len % g.t.block_size) {
                src = g.t.table[(int64_t)g.a[k] * g.t.stride + len / g.t.block_size];
                dst = g.free_ids[first_page(g, (int)k)];
                if (src < 0 || src >= p.c.num_blocks || src == dst) src = -1;
            }
            s_src[tid] = src;
            s_dst[tid] = dst;
        }
        __syncthreads();
        uint8_t* base = p.c.base[it / blocks];
        const int64_t n = p.c.page_bytes / (int64_t)sizeof(V);
        for (int64_t i0 = tid; i0 < n; i0 += U * kBlockThreads) {
            V v[U];
            int have = -1;
            for (int k = 0; k < p.block; k++) {
                const int src = s_src[k];
                if (src < 0) continue;
                if (src != have) {
                    const V* s = reinterpret_cast<const V*>(base + (int64_t)src * p.c.block_stride);
#pragma unroll
                    for (int u = 0; u < U; u++)
                        if (i0 + u * kBlockThreads < n) v[u] = __builtin_nontemporal_load(s + i0 + u * kBlockThreads);
                    have = src;
                }
                V* d = reinterpret_cast<V*>(base + (int64_t)s_dst[k] * p.c.block_stride);
#pragma unroll
                for (int u = 0; u < U; u++)
                    if (i0 + u * kBlockThreads < n) __builtin_nontemporal_store(v[u], d + i0 + u * kBlockThreads);
            }
        }
        for (int64_t i = n * (int64_t)sizeof(V) + tid; i < p.c.page_bytes; i += kBlockThreads)
            for (int k = 0; k < p.block; k++)
                if (s_src[k] >= 0)
                    base[(int64_t)s_dst[k] * p.c.block_stride + i] = base[(int64_t)s_src[k] * p.c.block_stride + i];
    }
}

// Widest access that every page of the caches is aligned to, in bytes.
static int page_align(const CacheList& c) {
    uintptr_t bits = (uintptr_t)c.block_stride;
    for (int i = 0; i < c.n; i++) bits |= reinterpret_cast<uintptr_t>(c.base[i]);
    return bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 1;
}
// A fixed grid that fills the device eight workgroups a CU deep.
static int64_t copy_grid(int64_t items) { return items < 1 ? 1 : items < 2048 ? items : 2048; }

static hipError_t copy_pairs(const CopyParams& p, int64_t items, hipStream_t s, bool first, bool last) {
    const int al = page_align(p.c);
    return launch_span(al == 16 ? k_copy_pages<u32x4> : al == 8 ? k_copy_pages<u32x2> : al == 4 ? k_copy_pages<uint32_t>
                                                                                                : k_copy_pages<uint8_t>,
                       copy_grid(items), kBlockThreads, s, first, last, p);
}

// ---------------------------------------------------------------------------
// compaction: L live pages end up in ids 0 .. L-1.  Holes (free ids below L)
// and movers (live ids from L on) are as many; the highest mover takes the
// lowest hole, so both ranks follow from the count of live pages before an id.
// ---------------------------------------------------------------------------
constexpr int kIdsPerThread = kCompactIds / kBlockThreads;   // 16

__device__ __forceinline__ int live_ids(const PageTable& t, int64_t id0, uint32_t& bits) {
    bits = 0;
#pragma unroll
    for (int i = 0; i < kIdsPerThread; i++)
        if (id0 + i < t.num_blocks && t.refs[id0 + i] > 0) bits |= 1u << i;
    return __popc(bits);
}

__global__ __launch_bounds__(kBlockThreads) void k_compact_count(CompactParams p, int64_t wg0) {
    __shared__ int s_n[kWavesPerBlock];
    const int64_t wg = wg0 + blockIdx.x;
    uint32_t bits;
    int n = live_ids(p.t, wg * kCompactIds + (int64_t)threadIdx.x * kIdsPerThread, bits);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d);
    if (lane_id() == 0) s_n[wave_id()] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
        int sum = 0;
        for (int i = 0; i < kWavesPerBlock; i++) sum += s_n[i];
        p.counts[wg] = sum;
    }
}

__global__ __launch_bounds__(kBlockThreads) void k_compact_rank(CompactParams p, int64_t wg0) {
    __shared__ int s_n[3][kWavesPerBlock];
    const int64_t wg = wg0 + blockIdx.x;
    const int wgs = (p.t.num_blocks - 1) / kCompactIds + 1, tid = threadIdx.x, lane = lane_id(), w = wave_id();
    const int64_t id0 = wg * kCompactIds + (int64_t)tid * kIdsPerThread;
    uint32_t bits;
    const int mine = live_ids(p.t, id0, bits);
    int before = 0, all = 0, x = mine;
    for (int i = tid; i < wgs; i += kBlockThreads) {
        const int c = p.counts[i];
        all += c;
        before += i < wg ? c : 0;
    }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int y = __shfl_up(x, d);
        if (lane >= d) x += y;
        before += __shfl_xor(before, d);
        all += __shfl_xor(all, d);
    }
    if (lane == kWave - 1) {
        s_n[0][w] = x;
        s_n[1][w] = before;
        s_n[2][w] = all;
    }
    __syncthreads();
    int live = x - mine, total = 0;                      // live ids before id0; live pages in all
    for (int i = 0; i < kWavesPerBlock; i++) {
        live += (i < w ? s_n[0][i] : 0) + s_n[1][i];
        total += s_n[2][i];
    }
    if (wg == 0 && tid == 0 && total == 0) *p.moves = 0;
#pragma unroll
    for (int i = 0; i < kIdsPerThread; i++) {
        const int64_t id = id0 + i;
        if (id >= p.t.num_blocks) break;
        const bool on = bits >> i & 1;
        int to = -1;
        if (on && id < total) to = (int)id;
        if (on && id >= total) {
            const int k = total - 1 - live;              // rank from the top
            p.movers[k] = (int)id;
            to = -2 - k;
        }
        if (!on && id < total) p.holes[id - live] = (int)id;
        p.page_map[id] = to;
        live += on;
        if (id == total - 1) *p.moves = total - live;    // holes below total
    }
}

// Renames: the table's entries, the counts of the moved pages, the map.
__global__ __launch_bounds__(kBlockThreads) void k_compact_finish(CompactParams p, int64_t wg0) {
    const int64_t wg = wg0 + blockIdx.x;
    const auto resolve = [&](int m) { return m <= -2 ? p.holes[-2 - m] : m; };
    if (wg < p.t.num_rows) {
        const int pages = (int)min((int64_t)pages_of(p.t.lens[wg], p.t.block_size), p.t.stride);
        int32_t* e = p.t.table + wg * p.t.stride;
        for (int i = threadIdx.x; i < pages; i += kBlockThreads) {
            const int id = e[i];
            // the map's entry is either the rank or, already, the page: both resolve alike
            if (id >= 0 && id < p.t.num_blocks)
                e[i] = resolve(__hip_atomic_load(&p.page_map[id], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
        }
        return;
    }
    const int64_t n = *p.moves;
    const int64_t k = (wg - p.t.num_rows) * kBlockThreads + threadIdx.x;
    if (k >= n) return;
    const int to = p.holes[k], from = p.movers[k];
    p.t.refs[to] = p.t.refs[from];
    p.t.refs[from] = 0;
    __hip_atomic_store(&p.page_map[from], to, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
hipError_t launch_copy_pages(const CacheList& c, const int32_t* src, const int32_t* dst, int64_t n, hipStream_t s,
                             bool first, bool last) {
    CopyParams p{c, {src, dst, nullptr, n}};
    return copy_pairs(p, n * c.n, s, first, last);
}
static hipError_t launch_plan(bool fork, const GrantParams& g, hipStream_t s) {
    auto k = g.n <= kPlanThreads ? (fork ? k_grant_small<true> : k_grant_small<false>)
                                 : (fork ? k_grant_plan<true> : k_grant_plan<false>);
    return launch_span(k, 1, kPlanThreads, s, true, false, g);
}
hipError_t launch_fork_plan(const GrantParams& g, hipStream_t s) { return launch_plan(true, g, s); }
hipError_t launch_fork_apply(const GrantParams& g, const CacheList& c, bool rows, hipStream_t s, bool last) {
    // as many forks a workgroup as still leave the device full
    int64_t block = (int64_t)g.n * c.n / 2048;
    block = block < 1 ? 1 : block > kForkBlock ? kForkBlock : block;
    ForkCopyParams p{c, g, (int32_t)block, rows};
    const int64_t items = (g.n + block - 1) / block * c.n, wgs = rows && g.n > items ? g.n : items;
    const int al = page_align(c);
    return launch_span(al == 16 ? k_fork_apply<u32x4> : al == 8 ? k_fork_apply<u32x2> : al == 4 ? k_fork_apply<uint32_t>
                                                                                                : k_fork_apply<uint8_t>,
                       copy_grid(wgs), kBlockThreads, s, false, last, p);
}
hipError_t launch_extend(const GrantParams& g, hipStream_t s) {
    const hipError_t e = launch_plan(false, g, s);
    return e != hipSuccess ? e : launch_span(k_extend_rows, g.n, kBlockThreads, s, false, true, g);
}
hipError_t launch_free(const PageTable& t, const int32_t* rows, int32_t n, hipStream_t s) {
    void* args[] = {const_cast<PageTable*>(&t), &rows, &n};
    return launch_piece(reinterpret_cast<const void*>(k_free_rows), n, kBlockThreads, args, s, true, true);
}
hipError_t launch_compact_plan(const CompactParams& c, hipStream_t s) {
    const int64_t wgs = (c.t.num_blocks - 1) / kCompactIds + 1;
    const hipError_t e = launch_span(k_compact_count, wgs, kBlockThreads, s, true, false, c);
    return e != hipSuccess ? e : launch_span(k_compact_rank, wgs, kBlockThreads, s, false, false, c);
}
hipError_t launch_compact_move(const CompactParams& c, const CacheList& l, hipStream_t s) {
    CopyParams p{l, {c.movers, c.holes, c.moves, 0}};
    // at most half of the pages move; the count itself is on the device
    return copy_pairs(p, (int64_t)(c.t.num_blocks / 2 + 1) * l.n, s, false, false);
}
hipError_t launch_compact_finish(const CompactParams& c, hipStream_t s) {
    const int64_t wgs = c.t.num_rows + (c.t.num_blocks / 2 + kBlockThreads) / kBlockThreads;
    return launch_span(k_compact_finish, wgs, kBlockThreads, s, false, true, c);
}

}  // namespace gcache
