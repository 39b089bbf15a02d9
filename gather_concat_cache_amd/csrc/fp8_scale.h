// fp8_scale.h -- scales of the pages of the e4m3 cache, as the append makes
// them and the attention takes them.
#pragma once

#include "gcache_device.h"

namespace gcache {

// What a scale counts as: within 2^-100 .. 2^121; what is not a positive number
// (NaN among it) as the least.
constexpr float kLeastScale = 0x1p-100f, kLargestScale = 0x1p121f;
__device__ __forceinline__ float page_scale(float s) { return fminf(fmaxf(s, kLeastScale), kLargestScale); }

// Value scales that the attention's sums take as they come: a row's weights carry
// their pages' value scales, P = exp2(s + log2 scale - m), and its sum adds P /
// scale.  Between these bounds that stays below 2^14 2^40 a key, and a P that
// exp2 flushes to 0 is a weight below 2^-68 of the row's largest.  Scales outside
// are far: rows that see one sum their weights apart (an append of zeros makes
// the least scale).
__device__ __forceinline__ bool far_scale(float s) { return s < 0x1p-40f || s > 0x1p24f; }

// The scale that values up to `largest` need.
__device__ __forceinline__ float append_need(float largest) { return fminf(fmaxf(largest / 448.0f, kLeastScale), 0x1p120f); }

// The least k >= 0 with scale * 2^k >= need; both are normal numbers.
__device__ __forceinline__ int doublings(float scale, float need) {
    const uint32_t a = __float_as_uint(scale), b = __float_as_uint(need);
    return max((int)(b >> 23) - (int)(a >> 23) + ((b & 0x7FFFFF) > (a & 0x7FFFFF) ? 1 : 0), 0);
}

// First page unit of request b whose first packed token is q: from there on are
// at least as many units as its tokens can touch pages, floor((n + 2 bs - 2) / bs).
__host__ __device__ __forceinline__ int64_t page_unit(int64_t q, int64_t b, int64_t bs) { return (q + b * (2 * bs - 2)) / bs; }

}  // namespace gcache
