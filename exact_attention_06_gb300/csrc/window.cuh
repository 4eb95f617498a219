// Which keys a query of a sliding window sees, as bits: key j of a query at position p is visible when j <= p and
// (j > p - window or j < sinks).
#pragma once
#include <cstdint>

namespace fattn {

// The lowest n bits of a word (n may be anything: none below 1, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return __funnelshift_lc(0xffffffffu, 0u, static_cast<uint32_t>(max(n, 0)));
}

// Of the keys key0 .. key0 + 31, those that the query at position p sees.
__device__ __forceinline__ uint32_t visible_keys(int key0, int p, int window, int sinks) {
  return low_bits(p - key0 + 1) & (~low_bits(p - window + 1 - key0) | low_bits(sinks - key0));
}

// Of the queries at positions pos0 .. pos0 + 31, those that see the key.
__device__ __forceinline__ uint32_t visible_queries(int pos0, int key, int window, int sinks) {
  return ~low_bits(key - pos0) & (key < sinks ? 0xffffffffu : low_bits(key + window - pos0));
}

// The w-th work item of `heads` heads with `ranks` items each, in the order of grouped_block: heads in ng groups (the first
// heads % ng one larger), and within a group rank 0 of every head first, then rank 1, and so on.
__device__ __forceinline__ void grouped_item(int w, int heads, int ranks, int ng, int& head, int& rank) {
  const int q = heads / ng, r = heads % ng, big = r * (q + 1) * ranks;
  const int size = w < big ? q + 1 : q, in = w < big ? w : w - big;
  const int g = in / (size * ranks), i = in - g * size * ranks;
  rank = i / size;
  head = (w < big ? 0 : r * (q + 1)) + g * size + (i - rank * size);
}

// Scores of hidden keys become -inf.
__device__ __forceinline__ void hide(uint32_t* s, uint32_t visible) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (!(visible & (1u << i))) s[i] = 0xff800000u;
}

}  // namespace fattn
