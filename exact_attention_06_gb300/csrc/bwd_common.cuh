// Pieces shared by the backward kernels (fa_bwd.cu, fa_cross_bwd.cu): bounded waits, the elementwise steps
// and gradient rows out of TMEM.
#pragma once
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"
#include "tmem_io.cuh"

namespace fattn {

// Each translation unit has its own status word and reads it itself.
static __device__ unsigned int g_bwd_status = 0;

namespace {

constexpr int kTile = 128;                // rows per tile on either side
constexpr uint32_t kBox = 128u * 128u;    // bytes of a 128-row x 64-column bf16 box
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ bool bwait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                      unsigned long long budget) {
  return mbar_wait(bar, parity, abort_flag, budget, &g_bwd_status);
}
__device__ __forceinline__ bool bwait_all(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          unsigned long long budget) {
  return __all_sync(0xffffffffu, bwait(bar, parity, abort_flag, budget));
}
__device__ __forceinline__ void bdrain(uint32_t bar, uint32_t parity, unsigned long long budget) {
  mbar_drain(bar, parity, budget, &g_bwd_status);
}

// One thread per row: a D-column fp32 tile row in TMEM * scale -> global (fp32), or as bf16 into the
// staged tile (box0: columns 0..63, box1: 64..127, 128-byte swizzle).
template <int D>
__device__ __forceinline__ void store_grad_row(void* out, size_t row_off, bool valid, uint32_t taddr, float scale) {
#pragma unroll
  for (int half = 0; half < D / 64; ++half) {
    uint32_t ur[64];
    tmem_ld_x64(taddr + 64u * half, ur);
    if (!valid) continue;
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + row_off * D + 64 * half);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      dst[i] = make_float4(__uint_as_float(ur[4 * i]) * scale, __uint_as_float(ur[4 * i + 1]) * scale,
                           __uint_as_float(ur[4 * i + 2]) * scale, __uint_as_float(ur[4 * i + 3]) * scale);
  }
}
template <int D>
__device__ __forceinline__ void stage_row_bf16(uint32_t box0, uint32_t box1, int r, uint32_t taddr, float scale) {
#pragma unroll
  for (int half = 0; half < D / 64; ++half) {
    uint32_t ur[64];
    tmem_ld_x64(taddr + 64u * half, ur);
    const uint32_t srow = (half ? box1 : box0) + static_cast<uint32_t>(r) * 128u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t* u = ur + 8 * i;
      sts128(srow + ((static_cast<uint32_t>(i) ^ static_cast<uint32_t>(r & 7)) << 4),
             pack_bf16(__uint_as_float(u[0]) * scale, __uint_as_float(u[1]) * scale),
             pack_bf16(__uint_as_float(u[2]) * scale, __uint_as_float(u[3]) * scale),
             pack_bf16(__uint_as_float(u[4]) * scale, __uint_as_float(u[5]) * scale),
             pack_bf16(__uint_as_float(u[6]) * scale, __uint_as_float(u[7]) * scale));
    }
  }
  fence_proxy_async_smem();
}

// S = A B^T into TMEM: A and B are resident/streamed 128 x d K-major tiles.
template <int D>
__device__ __forceinline__ void issue_product(uint32_t d_tmem, uint64_t da, uint64_t db, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = static_cast<uint32_t>(kk >> 2) * kBox + static_cast<uint32_t>(kk & 3) * 32u;
    if (kk == 0) mma_ss_c<0>(d_tmem, sdesc_add(da, off), sdesc_add(db, off), idesc);
    else mma_ss_c<1>(d_tmem, sdesc_add(da, off), sdesc_add(db, off), idesc);
  }
}
// Elementwise step of the dK/dV kernel on 32 query columns of one key row (column pairs packed
// as f32x2): P^T = 2^(S^T c - lse2), dS^T = P^T (dP^T - D), both rounded to bf16 pairs.  MASK
// (the diagonal tile only) zeroes P^T where the query precedes the key.
template <bool MASK>
__device__ __forceinline__ void ew_pairs_dkdv(const uint32_t (&sv)[32], const uint32_t (&pv)[32], const float4* nv,
                                              uint64_t c2, int col0, int qrow0, int key, uint32_t (&pp)[16],
                                              uint32_t (&dp)[16]) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const int col = col0 + e;  // query row within the tile
    const float4 x = nv[col >> 1];
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), c2, f2_pack(x.x, x.y)), x0, x1);
    float p0 = ex2(x0), p1 = ex2(x1);
    if (MASK) {
      if (qrow0 + col < key) p0 = 0.f;
      if (qrow0 + col + 1 < key) p1 = 0.f;
    }
    const uint64_t p2 = f2_pack(p0, p1);
    float s0, s1;
    f2_unpack(f2_mul(p2, f2_add(f2_pack(__uint_as_float(pv[e]), __uint_as_float(pv[e + 1])), f2_pack(x.z, x.w))),
              s0, s1);
    pp[e / 2] = pack_bf16(p0, p1);
    dp[e / 2] = pack_bf16(s0, s1);
  }
}

// Elementwise step of the dQ kernel on 32 key columns of one query row: dS = P (dP - D) with
// P = 2^(S c - lse2), rounded to bf16 pairs.  MASK zeroes keys past the row's last key; with CLEAR
// their dS is cleared after the product, so that padding behind them may hold anything.
template <bool MASK, bool CLEAR = false>
__device__ __forceinline__ void ew_pairs_dq(const uint32_t (&sv)[32], const uint32_t (&pv)[32], uint64_t c2,
                                            uint64_t nl2, uint64_t nd2, int key0, int lim, uint32_t (&dp)[16]) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), c2, nl2), x0, x1);
    float p0 = ex2(x0), p1 = ex2(x1);
    if (MASK) {
      if (key0 + e > lim) p0 = 0.f;
      if (key0 + e + 1 > lim) p1 = 0.f;
    }
    float s0, s1;
    f2_unpack(f2_mul(f2_pack(p0, p1), f2_add(f2_pack(__uint_as_float(pv[e]), __uint_as_float(pv[e + 1])), nd2)), s0,
              s1);
    if (MASK && CLEAR) {
      if (key0 + e > lim) s0 = 0.f;
      if (key0 + e + 1 > lim) s1 = 0.f;
    }
    dp[e / 2] = pack_bf16(s0, s1);
  }
}

}  // namespace
}  // namespace fattn
