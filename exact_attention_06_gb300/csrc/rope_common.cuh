// Pieces shared by the rotary kernels (fa_rope.cu, fa_norm_rope.cu): a thread's part of a row, its angles.
#pragma once
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace fattn {
namespace {

constexpr int kThreads = 128;
constexpr int kPairs = 8;   // pairs per thread: two 16-byte vectors of a row
constexpr int kUnroll = 4;  // heads whose loads are in flight together

template <int D>
struct RopeCfg {
  static constexpr int TPR = D / (2 * kPairs);   // threads per row
  static constexpr int ROWS = kThreads / TPR;    // rows per block
};

// The thread's two vectors of a row: pairs 8t .. 8t + 7 are the 16 adjacent elements from 16t
// (pairs side by side), or elements 8t .. of either half of the row.
template <int D, bool INTER>
__device__ __forceinline__ int second_vec() { return INTER ? 8 : D / 2; }
template <int D, bool INTER>
__device__ __forceinline__ int first_vec(int t) { return INTER ? 16 * t : 8 * t; }

// cos and sin of the thread's 8 pairs.  turns, axis: the plan's tables in shared memory.
__device__ __forceinline__ void angles(const unsigned long long* turns, const unsigned char* axis, int t,
                                       const int (&p)[FA_ROPE_MAX_AXES], float sign, float (&c)[kPairs],
                                       float (&s)[kPairs]) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int a = axis[t * kPairs + i];
    int pv = p[0];
#pragma unroll
    for (int k = 1; k < FA_ROPE_MAX_AXES; ++k)
      if (a == k) pv = p[k];
    const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(pv)) * turns[t * kPairs + i];
    const float half_turns = static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f;  // 2^-31
    sincospif(half_turns, &s[i], &c[i]);
    s[i] *= sign;
  }
}

__device__ __forceinline__ void load_tables(const fa_rope_axes_plan_t& plan, int d, unsigned long long* turns,
                                            unsigned char* axis) {
  for (int i = threadIdx.x; i < d / 2; i += kThreads) {
    turns[i] = plan.turns[i];
    axis[i] = plan.axis[i];
  }
  __syncthreads();
}

}  // namespace
}  // namespace fattn
