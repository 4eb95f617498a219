// Exponentials of a softmax step, shared by the forward kernels.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace fattn {

// P~ = 2^(s c - m) of this thread's N scores (64 or 32) as packed bf16 pairs, in place into sr[0..N/2-1]
// (entry i holds keys 2i, 2i + 1 of the half row); their fp32 sum goes to rs_a + rs_b.
template <int N>
__device__ __forceinline__ void exp_pack_bf16(uint32_t (&sr)[N], uint64_t c2, uint64_t nmb2, uint64_t& rs_a,
                                              uint64_t& rs_b) {
#pragma unroll
  for (int i = 0; i < N / 2; i += 2) {
    float x0, x1, x2, x3;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[2 * i]), __uint_as_float(sr[2 * i + 1])), c2, nmb2), x0, x1);
    f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[2 * i + 2]), __uint_as_float(sr[2 * i + 3])), c2, nmb2), x2, x3);
    const float p0 = ex2(x0), p1 = ex2(x1), p2 = ex2(x2), p3 = ex2(x3);
    rs_a = f2_add(rs_a, f2_pack(p0, p1));
    rs_b = f2_add(rs_b, f2_pack(p2, p3));
    sr[i] = pack_bf16(p0, p1);
    sr[i + 1] = pack_bf16(p2, p3);
  }
}

}  // namespace fattn
