// Pieces shared by the forward kernels (fa_fwd.cu, fa_window_fwd.cu): tile sizes, shared-memory layouts, bounded
// waits, and a row's steps in TMEM (row maximum, rescaling, outputs and partials).
#pragma once
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"
#include "softmax.cuh"
#include "stage_io.cuh"
#include "tmem_io.cuh"

namespace fattn {

// Each translation unit has its own status word and reads it itself.
static __device__ unsigned int g_fwd_status = 0;

namespace {

constexpr int kBr = 128;                 // query rows per tile (TMEM lanes, MMA M)
constexpr int kBc = 128;                 // keys per tile
constexpr int kRowsPerCta = 2 * kBr;
constexpr uint32_t kBox = 128u * 128u;   // bytes of a 128-row x 128-byte box (64 bf16 or 128 E4M3 columns)
constexpr int kSoftmaxWarps = 8;          // per query tile
constexpr int kWarpMma = 2 * kSoftmaxWarps;  // first MMA warp; also allocates TMEM
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;
constexpr float kLn2 = 0.6931471805599453f;

template <int D, bool FP8 = false>
struct FwdCfg {
  static constexpr int ESZ = FP8 ? 1 : 2;           // bytes per element (E4M3 or bf16)
  static constexpr int ROW = D * ESZ;               // bytes per row
  static constexpr int NH = ROW / 128;              // 128-byte boxes per row
  static constexpr int BOX_X = 128 / ESZ;           // elements per box row (TMA x step)
  static constexpr int K_MMA = 32 / ESZ;            // K elements per MMA instruction (32 bytes)
  static constexpr int KST = FP8 ? 4 : ((D == 128) ? 3 : 4);  // K ring stages
  static constexpr int VST = FP8 ? 4 : ((D == 128) ? 2 : 4);  // V ring stages
  static constexpr uint32_t QB = NH * kBox;         // bytes of one Q tile
  static constexpr uint32_t KVB = NH * kBox;        // bytes of one K (or V) tile
  static constexpr int B_Q = 0, B_QE = B_Q + 1, B_KF = B_QE + 1, B_KE = B_KF + KST, B_VF = B_KE + KST, B_VE = B_VF + VST,
                       B_SF = B_VE + VST, B_PF = B_SF + 2, B_SC = B_PF + 2, B_OF = B_SC + 2, B_DRAIN = B_OF + 2,
                       B_OSF = B_DRAIN + 2, B_OW = B_OSF + 2, B_VC = B_OW + 2, NBAR = B_VC + 1;
  // d = 64 leaves 128 TMEM columns free: P~_t gets its own columns there, so S_t(j+1) can be
  // computed while the softmax of tile j still runs ("separate P~").  At d = 128 P~ aliases S,
  // for bf16 (two keys a column) and E4M3 (four keys a column) alike.
  static constexpr bool SEP = D == 64;
  // E4M3: a second 16 KB box per tile, which with the Q tile's stages O in bf16 (128 x 256 bytes)
  static constexpr bool P_SMEM = FP8;
  static constexpr uint32_t COL_P = SEP ? 384u : 0u;        // separate P~ columns (+ 64 t)
  static constexpr uint32_t PB = P_SMEM ? kBr * 128u : 0u;  // bytes of one tile's second O staging box (E4M3)
  // With separate P~ each tile gets its own MMA warp (at d = 64 the PV MMAs, N = 64, are also too
  // short for one issuing thread); with P~ aliasing S (bf16, d = 128) one MMA warp alternating
  // between the tiles measured faster.
  static constexpr bool TWO_ISSUERS = SEP;
  // Softmax warps per query tile: with P~ aliasing S (d = 128) one thread per row (4 warps,
  // .32x32b TMEM access); the separate-P~ schedule (d = 64) two threads per row (8 warps, .16x32bx2).
  static constexpr bool ONE = !SEP;
  static constexpr int SMW = ONE ? 4 : 8;
  static constexpr int WARP_MMA = 2 * SMW;
  static constexpr int WARP_TMA = WARP_MMA + (TWO_ISSUERS ? 2 : 1);
  static constexpr int THREADS = (WARP_TMA + 1) * 32;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = 2 * QB;
  static constexpr uint32_t OFF_V = OFF_K + KST * KVB;
  static constexpr uint32_t OFF_P = OFF_V + VST * KVB;       // E4M3 only: O staging boxes of both tiles
  static constexpr uint32_t OFF_BAR = OFF_P + 2 * PB;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 8u * NBAR;  // TMEM address slot, abort flag
  static constexpr uint32_t SMEM = OFF_MISC + 16u + 1024u;   // + slack to align the base to 1 KB
};
static_assert(FwdCfg<128>::SMEM <= 232448, "shared memory of the d=128 kernel exceeds 227 KB");
static_assert(FwdCfg<128, true>::SMEM <= 232448, "shared memory of the FP8 kernel exceeds 227 KB");

__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         unsigned long long budget) {
  const bool ok = mbar_wait(bar, parity, abort_flag, budget, &g_fwd_status);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, unsigned long long budget) {
  mbar_drain(bar, parity, budget, &g_fwd_status);
}

// This thread's half of a U_t row (D/2 columns) *= alpha, in one TMEM round trip.
template <int D>
__device__ __forceinline__ void rescale_half_row(uint32_t taddr, float alpha) {
  const uint64_t a2 = f2_pack(alpha, alpha);
  uint32_t ur[D / 2];
  if constexpr (D == 128) tmem_ld2_x64<64>(taddr, ur); else tmem_ld2_x32<32>(taddr, ur);
#pragma unroll
  for (int i = 0; i < D / 4; ++i) {
    float lo, hi;
    f2_unpack(f2_mul(f2_pack(__uint_as_float(ur[2 * i]), __uint_as_float(ur[2 * i + 1])), a2), lo, hi);
    ur[2 * i] = __float_as_uint(lo);
    ur[2 * i + 1] = __float_as_uint(hi);
  }
  if constexpr (D == 128) tmem_st2_x64<64>(taddr, ur); else tmem_st2_x32<32>(taddr, ur);
}

// This thread's half of an O row = U / l to global memory (columns h*D/2 ..), and
// lse from the h = 0 thread.  Every lane runs the TMEM load (it is warp-collective);
// only rows < N are stored.
template <int D>
__device__ __forceinline__ void store_half_row(void* o, float* lse, size_t row_off, int h, bool valid, bool o_fp32,
                                               uint32_t taddr, float l, float m2, float o_mult) {
  uint32_t ur[D / 2];
  if constexpr (D == 128) tmem_ld2_x64<64>(taddr, ur); else tmem_ld2_x32<32>(taddr, ur);
  if (!valid) return;
  const float inv = (l > 0.f) ? o_mult / l : 0.f;
  if (o_fp32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(o) + row_off * D + h * (D / 2));
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      dst[i] = make_float4(__uint_as_float(ur[4 * i]) * inv, __uint_as_float(ur[4 * i + 1]) * inv,
                           __uint_as_float(ur[4 * i + 2]) * inv, __uint_as_float(ur[4 * i + 3]) * inv);
  } else {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(o) + row_off * D + h * (D / 2));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint4 w;
      w.x = pack_bf16(__uint_as_float(ur[8 * i + 0]) * inv, __uint_as_float(ur[8 * i + 1]) * inv);
      w.y = pack_bf16(__uint_as_float(ur[8 * i + 2]) * inv, __uint_as_float(ur[8 * i + 3]) * inv);
      w.z = pack_bf16(__uint_as_float(ur[8 * i + 4]) * inv, __uint_as_float(ur[8 * i + 5]) * inv);
      w.w = pack_bf16(__uint_as_float(ur[8 * i + 6]) * inv, __uint_as_float(ur[8 * i + 7]) * inv);
      dst[i] = w;
    }
  }
  if (h == 0) lse[row_off] = (l > 0.f) ? (m2 + log2f(l)) * kLn2 : -INFINITY;
}

// This thread's half of a partial (U, m, l) row for a key shard: U unnormalised (relative to
// exp(s - m)), m in natural-log units, l; an empty row (no admissible key) gets m = -inf,
// l = 0 and no U.
template <int D>
__device__ __forceinline__ void store_half_partial(const FwdAux& aux, size_t slot, int h, bool valid, uint32_t taddr,
                                                   float l, float m2, bool have_u) {
  uint32_t ur[D / 2];
  if (have_u) {
    if constexpr (D == 128) tmem_ld2_x64<64>(taddr, ur); else tmem_ld2_x32<32>(taddr, ur);
  }
  if (!valid) return;
  const bool empty = !(l > 0.f);
  if (!empty) {  // an empty partial's U is never read (the combine skips m = -inf)
    float4* dst = reinterpret_cast<float4*>(aux.u_part + slot * D + h * (D / 2));
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      dst[i] = make_float4(__uint_as_float(ur[4 * i]), __uint_as_float(ur[4 * i + 1]),
                           __uint_as_float(ur[4 * i + 2]), __uint_as_float(ur[4 * i + 3]));
  }
  if (h == 0) {
    aux.m_part[slot] = empty ? -INFINITY : m2 * kLn2;
    aux.l_part[slot] = empty ? 0.f : l;
  }
}

// The new running row max, in exponent units (scores x c), from this thread's 64 scores of
// the row (sr, raw fp32 bits; those from index `nvalid` on are masked to -inf in place) joined
// with the other half of the row held by lane ^ 16.
__device__ __forceinline__ float row_max_update(uint32_t (&sr)[64], int nvalid, float m2, float c) {
  if (nvalid < 64) {
#pragma unroll
    for (int i = 0; i < 64; ++i)
      if (i >= nvalid) sr[i] = __float_as_uint(-INFINITY);
  }
  float a0 = __uint_as_float(sr[0]), a1 = __uint_as_float(sr[1]);
  float a2 = __uint_as_float(sr[2]), a3 = __uint_as_float(sr[3]);
#pragma unroll
  for (int i = 4; i < 60; i += 8) {
    a0 = fmax3(a0, __uint_as_float(sr[i]), __uint_as_float(sr[i + 1]));
    a1 = fmax3(a1, __uint_as_float(sr[i + 2]), __uint_as_float(sr[i + 3]));
    a2 = fmax3(a2, __uint_as_float(sr[i + 4]), __uint_as_float(sr[i + 5]));
    a3 = fmax3(a3, __uint_as_float(sr[i + 6]), __uint_as_float(sr[i + 7]));
  }
  a0 = fmax3(a0, __uint_as_float(sr[60]), __uint_as_float(sr[61]));
  a1 = fmax3(a1, __uint_as_float(sr[62]), __uint_as_float(sr[63]));
  float mx = fmax3(a0, a1, fmaxf(a2, a3));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));  // join the two halves of the row
  return fmaxf(m2, mx * c);
}

// One thread per row (d = 128): the row max over its 128 scores (sr: columns 0..63, sr2: 64..127,
// raw fp32 bits; those from index `nvalid` on masked to -inf in place), in exponent units.
__device__ __forceinline__ float row_max_full(uint32_t (&sr)[64], uint32_t (&sr2)[64], int nvalid, float m2, float c) {
  if (nvalid < 128) {
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      if (i >= nvalid) sr[i] = __float_as_uint(-INFINITY);
      if (64 + i >= nvalid) sr2[i] = __float_as_uint(-INFINITY);
    }
  }
  float a[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    a[k] = fmax3(__uint_as_float(sr[2 * k]), __uint_as_float(sr[2 * k + 1]), __uint_as_float(sr[8 + 2 * k]));
    a[4 + k] = fmax3(__uint_as_float(sr2[2 * k]), __uint_as_float(sr2[2 * k + 1]), __uint_as_float(sr2[8 + 2 * k]));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    a[k] = fmaxf(a[k], __uint_as_float(sr[9 + 2 * k]));
    a[4 + k] = fmaxf(a[4 + k], __uint_as_float(sr2[9 + 2 * k]));
  }
#pragma unroll
  for (int i = 16; i < 64; i += 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = fmax3(a[k], __uint_as_float(sr[i + 2 * k]), __uint_as_float(sr[i + 2 * k + 1]));
      a[4 + k] = fmax3(a[4 + k], __uint_as_float(sr2[i + 2 * k]), __uint_as_float(sr2[i + 2 * k + 1]));
    }
  }
  const float mx = fmax3(fmax3(a[0], a[1], a[2]), fmax3(a[3], a[4], a[5]), fmaxf(a[6], a[7]));
  return fmaxf(m2, mx * c);
}

// One thread per row (d = 128): U_t row *= alpha in two TMEM round trips of 64 columns.
__device__ __forceinline__ void rescale_row128(uint32_t taddr, float alpha) {
  const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t ur[64];
    tmem_ld_x64(taddr + 64u * half, ur);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      float lo, hi;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(ur[2 * i]), __uint_as_float(ur[2 * i + 1])), a2), lo, hi);
      ur[2 * i] = __float_as_uint(lo);
      ur[2 * i + 1] = __float_as_uint(hi);
    }
    tmem_st_x64(taddr + 64u * half, ur);
  }
}

// One thread per row (d = 128): O row = U / l as bf16 into the staged tile (box0: columns 0..63,
// box1: 64..127, 128-byte swizzle), with the proxy fence the TMA store needs.
__device__ __forceinline__ void stage_full_row_bf16(uint32_t box0, uint32_t box1, int r, uint32_t taddr, float mult) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t ur[64];
    tmem_ld_x64(taddr + 64u * half, ur);
    const uint32_t srow = (half ? box1 : box0) + static_cast<uint32_t>(r) * 128u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t* u = ur + 8 * i;
      sts128(srow + ((static_cast<uint32_t>(i) ^ static_cast<uint32_t>(r & 7)) << 4),
             pack_bf16(__uint_as_float(u[0]) * mult, __uint_as_float(u[1]) * mult),
             pack_bf16(__uint_as_float(u[2]) * mult, __uint_as_float(u[3]) * mult),
             pack_bf16(__uint_as_float(u[4]) * mult, __uint_as_float(u[5]) * mult),
             pack_bf16(__uint_as_float(u[6]) * mult, __uint_as_float(u[7]) * mult));
    }
  }
  fence_proxy_async_smem();
}

// One thread per row (d = 128): O row = U * o_mult / l (fp32 or bf16; o_mult carries the E4M3 V
// scale) and lse to global memory, rows < N.
__device__ __forceinline__ void store_full_row(void* o, float* lse, size_t row_off, bool valid, bool o_fp32,
                                               uint32_t taddr, float l, float m2, float o_mult) {
  const float inv = (l > 0.f) ? o_mult / l : 0.f;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t ur[64];
    tmem_ld_x64(taddr + 64u * half, ur);
    if (!valid) continue;
    if (o_fp32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(o) + row_off * 128 + 64 * half);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        dst[i] = make_float4(__uint_as_float(ur[4 * i]) * inv, __uint_as_float(ur[4 * i + 1]) * inv,
                             __uint_as_float(ur[4 * i + 2]) * inv, __uint_as_float(ur[4 * i + 3]) * inv);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(o) + row_off * 128 + 64 * half);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint4 w;
        w.x = pack_bf16(__uint_as_float(ur[8 * i + 0]) * inv, __uint_as_float(ur[8 * i + 1]) * inv);
        w.y = pack_bf16(__uint_as_float(ur[8 * i + 2]) * inv, __uint_as_float(ur[8 * i + 3]) * inv);
        w.z = pack_bf16(__uint_as_float(ur[8 * i + 4]) * inv, __uint_as_float(ur[8 * i + 5]) * inv);
        w.w = pack_bf16(__uint_as_float(ur[8 * i + 6]) * inv, __uint_as_float(ur[8 * i + 7]) * inv);
        dst[i] = w;
      }
    }
  }
  if (valid) lse[row_off] = (l > 0.f) ? (m2 + log2f(l)) * kLn2 : -INFINITY;
}

// One thread per row (d = 128): the key shard's partial (U, m, l) of the row, as store_half_partial.
__device__ __forceinline__ void store_full_partial(const FwdAux& aux, size_t slot, bool valid, uint32_t taddr, float l,
                                                   float m2) {
  const bool empty = !(l > 0.f);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t ur[64];
    tmem_ld_x64(taddr + 64u * half, ur);
    if (!valid || empty) continue;
    float4* dst = reinterpret_cast<float4*>(aux.u_part + slot * 128 + 64 * half);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      dst[i] = make_float4(__uint_as_float(ur[4 * i]), __uint_as_float(ur[4 * i + 1]), __uint_as_float(ur[4 * i + 2]),
                           __uint_as_float(ur[4 * i + 3]));
  }
  if (valid) {
    aux.m_part[slot] = empty ? -INFINITY : m2 * kLn2;
    aux.l_part[slot] = empty ? 0.f : l;
  }
}

// lse of this thread's row from the h = 0 thread, rows < N only.
__device__ __forceinline__ void store_lse(float* lse, size_t row_off, int h, bool valid, float l, float m2) {
  if (h == 0 && valid) lse[row_off] = (l > 0.f) ? (m2 + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace
}  // namespace fattn
