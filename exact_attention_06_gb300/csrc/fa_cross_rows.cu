// Cross attention of few query rows (fa_cross_fwd with at most 32 rows per key head, or 16 over at most 128
// keys: a decode step and its shared heads), for sm_103a.
//
// Such a call reads each key head's K and V once for 4 * rows * d flops a key: it is bound by HBM, and
// what counts is bytes in flight and a short path from the last byte to the output.  A 128-row
// tcgen05 tile would spend its softmax on empty rows and a round trip through TMEM on every step
// (measured below), so the products are the warp-level 16 x 8 x 16 matrix instruction on rows that stay in registers:
//   S (16 rows x 16 keys)  = Q K^T    Q's fragments loaded once, K's by ldmatrix
//   U (16 rows x d)       += P~ V     P~ = bf16(2^(s c - m)) is S's fragment repacked, V's by ldmatrix.trans
// One producer thread streams 64-key stages of K and V through a 3-stage TMA ring (128-byte swizzle);
// compute warp w takes keys 16 (w % 4) .. of every stage for rows 16 (w / 4) .. and keeps an
// online softmax (m, l, U) of its own, so warps meet only once, at the end.
//
// A sequence's stages are shared out evenly over S blocks.  Up to 8 of them are a thread-block
// cluster: each leaves its partial (U, m, l) in shared memory, and after a cluster barrier each
// combines a share of the output from all of them through distributed shared memory -- one launch, no
// workspace.  Where more are needed to fill the GPU they write partials for the combine kernel.
//
// Padding.  Scores behind the sequence are replaced by -inf; V's words behind it are cleared in the
// fragments, so that 0 times what the padding holds never reaches U.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace fattn {

__device__ unsigned int g_rows_status = 0;

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSk = kRowsStageKeys;  // keys per stage
constexpr int kSt = 3;               // ring stages
constexpr int kKw = kSk / 16;        // warps along the keys of a stage

template <int D, int RB>
struct RowsCfg {
  static constexpr int NH = D / 64;
  static constexpr uint32_t BOX = kSk * 128u;  // bytes of one [kSk keys x 64 dims] box
  static constexpr uint32_t TB = NH * BOX;     // bytes of K (or V) per stage
  static constexpr int NW = RB * kKw;          // compute warps
  static constexpr int THREADS = (NW + 1) * 32;
  static constexpr int ROWS = 16 * RB;
  static constexpr int B_KF = 0, B_VF = kSt, B_EMPTY = 2 * kSt, NBAR = 3 * kSt;
  static constexpr uint32_t OFF_K = 0, OFF_V = kSt * TB, OFF_BAR = 2 * kSt * TB;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 8u * NBAR;  // abort flag
  // The block's partial: m, l [ROWS], U [ROWS][D]; the warps' partials it is merged from take the ring
  // (m, l [NW][16], U [NW][16][D + 4]: the padding spreads the fragment rows over the banks).
  static constexpr uint32_t OFF_PART = (OFF_MISC + 16u + 127u) & ~127u;
  static constexpr uint32_t SMEM = OFF_PART + 4u * ROWS * (D + 2) + 1024u;
  static constexpr int LDU = D + 4;
  // Blocks an SM holds.  Measured at d = 64 with two instead of four: 64 key heads x 32768 keys 94 instead of
  // 79 us (6.8 TB/s), 512 x 1500 40.5 instead of 34.3 us.
  static constexpr int PER_SM = cross_rows_per_sm(D, ROWS);
  static_assert(4u * NW * 16 * (LDU + 2) <= OFF_BAR, "the warps' partials fit the ring");
  static_assert(PER_SM * (SMEM + 1024) <= 233472, "shared memory of the resident blocks");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c (16 x 8, fp32) += a (16 x 16, bf16) b (16 x 8, bf16)
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// A float of the same shared-memory address in block `rank` of the cluster.
__device__ __forceinline__ float peer_f32(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("{\n\t.reg .u32 p;\n\tmapa.shared::cluster.u32 p, %1, %2;\n\tld.shared::cluster.f32 %0, [p];\n}\n"
               : "=f"(v)
               : "r"(addr), "r"(rank)
               : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_f32x4(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .u32 p;\n\tmapa.shared::cluster.u32 p, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [p];\n}\n"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

__device__ __forceinline__ bool rwait_all(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          unsigned long long budget) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, budget, &g_rows_status));
}
__device__ __forceinline__ void rdrain(uint32_t bar, uint32_t parity, unsigned long long budget) {
  mbar_drain(bar, parity, budget, &g_rows_status);
}

// Block blockIdx.x = key head * S + share.  CLUSTER: the S blocks of a key head are a cluster and write O and lse;
// otherwise they write partial slots (rows, S) for the combine kernel.
template <int D, int RB, bool CLUSTER>
__global__ void __launch_bounds__(RowsCfg<D, RB>::THREADS, RowsCfg<D, RB>::PER_SM)
    cross_rows_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                      const CrossRowsArgs a) {
  using C = RowsCfg<D, RB>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // (the same offset in every block of a cluster)
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sK = base + C::OFF_K, sV = base + C::OFF_V, sBar = base + C::OFF_BAR;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_MISC);
#define BAR(i) (sBar + 8u * static_cast<uint32_t>(i))
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = a.S;
  const int bh = static_cast<int>(blockIdx.x / static_cast<unsigned>(S));
  const int sp = static_cast<int>(blockIdx.x % static_cast<unsigned>(S));
  if constexpr (!CLUSTER) grid_dep_launch();  // the combine kernel may launch

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSt; ++s) {
      mbar_init(BAR(C::B_KF + s), 1);
      mbar_init(BAR(C::B_VF + s), 1);
      mbar_init(BAR(C::B_EMPTY + s), C::NW);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  grid_dep_wait();  // every global access below comes after the previous kernel in the stream
  const int len = a.kv_lens ? min(max(a.kv_lens[bh / a.kv_heads], 0), a.Nk) : a.Nk;
  const long long stages = (static_cast<long long>(len) + kSk - 1) / kSk;
  const int st0 = static_cast<int>(stages * sp / S), n_st = static_cast<int>(stages * (sp + 1) / S) - st0;
  __syncthreads();

  if (warp == C::NW) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int issued = 0;
      for (int i = 0; i < n_st; ++i) {
        const int s = i % kSt;
        if (i >= kSt && !mbar_wait(BAR(C::B_EMPTY + s), ((i / kSt) - 1) & 1, abort_flag, a.budget, &g_rows_status)) break;
        const int key = (st0 + i) * kSk;
        mbar_arrive_expect_tx(BAR(C::B_KF + s), C::TB);
        for (int h = 0; h < C::NH; ++h) tma_load_3d(sK + s * C::TB + h * C::BOX, &tk, BAR(C::B_KF + s), h * 64, key, bh);
        mbar_arrive_expect_tx(BAR(C::B_VF + s), C::TB);
        for (int h = 0; h < C::NH; ++h) tma_load_3d(sV + s * C::TB + h * C::BOX, &tv, BAR(C::B_VF + s), h * 64, key, bh);
        issued = i + 1;
      }
      for (int i = max(issued - kSt, 0); i < issued; ++i) {  // every copy lands before the ring is reused
        rdrain(BAR(C::B_KF + i % kSt), (i / kSt) & 1, a.budget);
        rdrain(BAR(C::B_VF + i % kSt), (i / kSt) & 1, a.budget);
      }
    }
    __syncwarp();
    named_bar_sync(1, C::THREADS);
  } else {
    // ------------------------------------------------------------ compute warps
    const int kw = warp % kKw, rb = warp / kKw;
    const int g = lane >> 2, t = lane & 3;  // fragment row (and g + 8), fragment column pair
    // Q's fragments: words (row g, dims 16 kk + 2t), (g + 8, ..), (g, .. + 8), (g + 8, .. + 8)
    uint32_t qf[D / 16][4];
    {
      const int r0 = rb * 16 + g, r1 = r0 + 8;
      const uint32_t* q0 = reinterpret_cast<const uint32_t*>(a.q) + (static_cast<size_t>(bh) * a.R + r0) * (D / 2) + t;
      const uint32_t* q1 = q0 + 8 * (D / 2);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][0] = r0 < a.R ? q0[8 * kk] : 0u;
        qf[kk][1] = r1 < a.R ? q1[8 * kk] : 0u;
        qf[kk][2] = r0 < a.R ? q0[8 * kk + 4] : 0u;
        qf[kk][3] = r1 < a.R ? q1[8 * kk + 4] : 0u;
      }
    }
    float u[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) u[i][j] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows g, g + 8 (l: this lane's share)
    // ldmatrix row of this lane: K: key (lane & 7) of an 8-key group, 16-byte chunk lane >> 3 of four;
    // V (transposed): key lane & 15, chunk lane >> 4 of two.  Chunk c of row r is at c ^ (r & 7).
    const uint32_t krow = static_cast<uint32_t>(16 * kw + (lane & 7)) * 128u, kchunk = lane >> 3;
    const uint32_t vrow = static_cast<uint32_t>(16 * kw + (lane & 15)) * 128u, vchunk = lane >> 4;
    const uint32_t swz = lane & 7;
    for (int i = 0; i < n_st; ++i) {
      const int s = i % kSt;
      const uint32_t par = (i / kSt) & 1;
      if (!rwait_all(BAR(C::B_KF + s), par, abort_flag, a.budget)) break;
      const uint32_t kb = sK + s * C::TB + krow;
      float c[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {  // keys 8n .. 8n + 7 of the warp's 16
#pragma unroll
        for (int j = 0; j < 4; ++j) c[n][j] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; kk += 2) {
          const uint32_t ch = 2u * kk + kchunk;  // 16-byte chunk of the row
          uint32_t b[4];
          ldsm4(kb + n * 1024u + (ch >> 3) * C::BOX + (((ch & 7) ^ swz) << 4), b);
          mma16816(c[n], qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3], b[0], b[1]);
          mma16816(c[n], qf[kk + 1][0], qf[kk + 1][1], qf[kk + 1][2], qf[kk + 1][3], b[2], b[3]);
        }
      }
      const int left = len - (st0 + i) * kSk - 16 * kw;  // keys of the sequence from the warp's first on
      const bool tail = left < 16;
      if (tail) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (8 * n + 2 * t + j >= left) c[n][j] = c[n][2 + j] = -INFINITY;
      }
      float x0 = fmaxf(fmaxf(c[0][0], c[0][1]), fmaxf(c[1][0], c[1][1]));
      float x1 = fmaxf(fmaxf(c[0][2], c[0][3]), fmaxf(c[1][2], c[1][3]));
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
      const float n0 = fmaxf(m0, x0 * a.sl2), n1 = fmaxf(m1, x1 * a.sl2);
      const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;  // no key yet: p = 0
      const float al0 = ex2(m0 - b0), al1 = ex2(m1 - b1);
      m0 = n0;
      m1 = n1;
      float p[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        p[n][0] = ex2(fmaf(c[n][0], a.sl2, -b0));
        p[n][1] = ex2(fmaf(c[n][1], a.sl2, -b0));
        p[n][2] = ex2(fmaf(c[n][2], a.sl2, -b1));
        p[n][3] = ex2(fmaf(c[n][3], a.sl2, -b1));
      }
      // l sums the unrounded p; P~ is bf16 as the PV operand, as everywhere in this library
      l0 = fmaf(al0, l0, (p[0][0] + p[0][1]) + (p[1][0] + p[1][1]));
      l1 = fmaf(al1, l1, (p[0][2] + p[0][3]) + (p[1][2] + p[1][3]));
      const uint32_t pa0 = pack_bf16(p[0][0], p[0][1]), pa1 = pack_bf16(p[0][2], p[0][3]);
      const uint32_t pa2 = pack_bf16(p[1][0], p[1][1]), pa3 = pack_bf16(p[1][2], p[1][3]);
      if (!__all_sync(0xffffffffu, al0 == 1.f && al1 == 1.f)) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          u[n][0] *= al0;
          u[n][1] *= al0;
          u[n][2] *= al1;
          u[n][3] *= al1;
        }
      }
      if (!rwait_all(BAR(C::B_VF + s), par, abort_flag, a.budget)) break;
      const uint32_t vb = sV + s * C::TB + vrow;
      // keys 2t, 2t + 1 (and 8 more) of a V fragment word: the halves behind the sequence are cleared
      const uint32_t keep0 = (2 * t < left ? 0xFFFFu : 0u) | (2 * t + 1 < left ? 0xFFFF0000u : 0u);
      const uint32_t keep1 = (8 + 2 * t < left ? 0xFFFFu : 0u) | (9 + 2 * t < left ? 0xFFFF0000u : 0u);
#pragma unroll
      for (int n = 0; n < D / 8; n += 2) {
        const uint32_t ch = static_cast<uint32_t>(n) + vchunk;
        uint32_t b[4];
        ldsm4t(vb + (ch >> 3) * C::BOX + (((ch & 7) ^ swz) << 4), b);
        if (tail) {
          b[0] &= keep0;
          b[1] &= keep1;
          b[2] &= keep0;
          b[3] &= keep1;
        }
        mma16816(u[n], pa0, pa1, pa2, pa3, b[0], b[1]);
        mma16816(u[n + 1], pa0, pa1, pa2, pa3, b[2], b[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::B_EMPTY + s));
    }
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    // The warps' partials take the ring's place once all of them (and the producer's copies) are done with it.
    named_bar_sync(1, C::THREADS);
    float* wm = reinterpret_cast<float*>(gbase);
    float* wl = wm + C::NW * 16;
    float* wu = wl + C::NW * 16 + warp * 16 * C::LDU;
    if (t == 0) {
      wm[warp * 16 + g] = m0;
      wm[warp * 16 + g + 8] = m1;
      wl[warp * 16 + g] = l0;
      wl[warp * 16 + g + 8] = l1;
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      *reinterpret_cast<float2*>(wu + g * C::LDU + 8 * n + 2 * t) = make_float2(u[n][0], u[n][1]);
      *reinterpret_cast<float2*>(wu + (g + 8) * C::LDU + 8 * n + 2 * t) = make_float2(u[n][2], u[n][3]);
    }
  }
  __syncthreads();

  // ------------------------------------------------------------ the block's partial: 4 columns a thread
  const float* wm = reinterpret_cast<const float*>(gbase);
  const float* wl = wm + C::NW * 16;
  const float* wu = wl + C::NW * 16;
  float* pm = reinterpret_cast<float*>(gbase + C::OFF_PART);
  float* pl = pm + C::ROWS;
  float* pu = pl + C::ROWS;
  for (int e = threadIdx.x; e < a.R * (D / 4); e += C::THREADS) {
    const int row = e / (D / 4), col = (e % (D / 4)) * 4;
    const int w0 = (row >> 4) * kKw, r = row & 15;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kKw; ++w) mm = fmaxf(mm, wm[(w0 + w) * 16 + r]);
    const float mb = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kKw; ++w) {
      const float f = ex2(wm[(w0 + w) * 16 + r] - mb);
      const float4 y = *reinterpret_cast<const float4*>(wu + ((w0 + w) * 16 + r) * C::LDU + col);
      ll = fmaf(f, wl[(w0 + w) * 16 + r], ll);
      x.x = fmaf(f, y.x, x.x);
      x.y = fmaf(f, y.y, x.y);
      x.z = fmaf(f, y.z, x.z);
      x.w = fmaf(f, y.w, x.w);
    }
    if constexpr (CLUSTER) {
      *reinterpret_cast<float4*>(pu + row * D + col) = x;
      if (col == 0) {
        pm[row] = mm;
        pl[row] = ll;
      }
    } else {
      const size_t slot = (static_cast<size_t>(bh) * a.R + row) * S + sp;
      *reinterpret_cast<float4*>(a.u_part + slot * D + col) = x;
      if (col == 0) {
        a.m_part[slot] = mm * kLn2;  // natural-log units; -inf stays -inf
        a.l_part[slot] = ll;
      }
    }
  }
  if constexpr (CLUSTER) {
    // ---------------------------------------------------------- O and lse: a share of the rows' vectors per block
    cluster_sync();
    const uint32_t spm = base + C::OFF_PART, spl = spm + 4u * C::ROWS, spu = spl + 4u * C::ROWS;
    const int total = a.R * (D / 4), rank = static_cast<int>(cluster_rank());
    for (int e = rank * C::THREADS + threadIdx.x; e < total; e += S * C::THREADS) {
      const int row = e / (D / 4), col = (e % (D / 4)) * 4;
      float mm = -INFINITY;
      for (int s = 0; s < S; ++s) mm = fmaxf(mm, peer_f32(spm + 4u * row, s));
      const float mb = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s = 0; s < S; ++s) {
        const float f = ex2(peer_f32(spm + 4u * row, s) - mb);
        const float4 y = peer_f32x4(spu + 4u * (row * D + col), s);
        ll = fmaf(f, peer_f32(spl + 4u * row, s), ll);
        x.x = fmaf(f, y.x, x.x);
        x.y = fmaf(f, y.y, x.y);
        x.z = fmaf(f, y.z, x.z);
        x.w = fmaf(f, y.w, x.w);
      }
      const float inv = ll > 0.f ? 1.f / ll : 0.f;
      const size_t row_off = static_cast<size_t>(bh) * a.R + row;
      if (a.o_fp32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.o) + row_off * D + col) =
            make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + row_off * D + col) =
            make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
      if (col == 0) a.lse[row_off] = ll > 0.f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
    }
    cluster_sync();  // no block leaves while another reads its partial
  }
#undef BAR
}

template <int D, int RB, bool CLUSTER>
cudaError_t launch_t(const CrossRowsLaunch& l, cudaStream_t stream) {
  using C = RowsCfg<D, RB>;
  const CrossRowsArgs& a = l.args;
  auto kern = cross_rows_kernel<D, RB, CLUSTER>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(a.S);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(l.BH) * static_cast<unsigned>(a.S));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, l.tk, l.tv, a);
}

}  // namespace

cudaError_t launch_cross_rows(const CrossRowsLaunch& a, cudaStream_t stream) {
  const bool two = a.args.R > 16, cluster = a.args.u_part == nullptr;
  if (a.d == 64) {
    if (cluster) return two ? launch_t<64, 2, true>(a, stream) : launch_t<64, 1, true>(a, stream);
    return two ? launch_t<64, 2, false>(a, stream) : launch_t<64, 1, false>(a, stream);
  }
  if (cluster) return two ? launch_t<128, 2, true>(a, stream) : launch_t<128, 1, true>(a, stream);
  return two ? launch_t<128, 2, false>(a, stream) : launch_t<128, 1, false>(a, stream);
}

cudaError_t cross_rows_status_word(unsigned int** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_rows_status);
}

}  // namespace fattn
