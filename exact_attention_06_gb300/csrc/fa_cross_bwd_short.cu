// Cross attention backward over at most 128 keys (fa_cross_bwd), for sm_103a: dQ, dK and dV of a text prompt of 77
// tokens or 64 latents in one pass over Q and dO.
//
// A block keeps K, V and the sums of its range of query tiles, dV [keys, d] and dK [keys, d] in TMEM, and streams the
// tiles past them.  Per tile of 128 query rows:
//   S = Q K^T, dP = dO V^T                  P = 2^(S c - lse), D = sum of P dP, dS = P (dP - D)
//   dV += P^T dO, dK += dS^T Q, dQ = dS K   P and dS as bf16 in shared memory, [query][key]: the first two take them
//                                           with the keys as rows (MN-major), the last as they lie
// A row's keys are all there, so D takes no pass over O (and no rounding of O).  Bound by HBM: Q and dO in, dQ out,
// 6 d + 4 bytes a row (8 x 64/16 heads, 4595 rows, 49 keys: 5.2 TB/s at d = 64, 5.7 at d = 128), where the chain of a
// tile, about 2 us, is hidden:
// - Two tiles in flight, a thread per row, where TMEM holds them (64 keys, and 96 at d = 64).
// - Else one (bound by that chain: 3.6-3.9 TB/s at d = 128), shortened: a row has two threads, one for each 64 keys,
//   which exchange their halves of D; the next tile's S is computed and its exponentials are taken while this one's
//   gradients are; Q and dO come and go apart, and dQ leaves through dO's place, which is the one needed later.
//   (2 x 16 heads, 8192 x 77, d = 128: 62 -> 51 us; with dQ in Q's place 62: the next loads then wait for the store.)
// - lse is read a tile ahead (8 x 64/16, 4595 x 49, d = 64: 197 -> 176 us).
// One thread issues S and dP, another the products with P and dS, whose sums want one order.  Several blocks of a key
// head leave fp32 partial sums, which cross_sum_kernel adds in their order.  Measured beside plan_cross_bwd.
//
// Padding behind the sequence: P and dS become 0 after the arithmetic and K's rows are cleared in shared memory, once.
#include "bwd_common.cuh"

namespace fattn {

namespace {

// KT: keys of the tile that are computed (64, 96 or 128).
template <int D, int KT>
struct BwdShortCfg {
  static constexpr int CH = KT == 64 || (D == 64 && KT == 96) ? 2 : 1;  // tiles in flight (chains)
  static constexpr int W = 2 / CH;                                      // threads per row
  // One chain: dQ is written over dP alone, the next tile's S comes early, and a stage's Q and dO come and go apart.
  static constexpr bool EARLY = CH == 1;
  static constexpr int NH = D / 64;
  static constexpr uint32_t KBOX = (KT == 64 ? 64u : 128u) * 128u;  // bytes of a box of K or V
  static constexpr uint32_t TK = NH * KBOX, TQ = NH * kBox;
  // dQ on its way out: in a place of its own, in that of the tile's dO, or in the chain's buffer, as shared memory allows
  // (a store warp, or, from the buffer, the chain's first thread).
  enum Out { kOwn, kInDO, kInBuf };
  static constexpr Out OUT = CH == 2 ? kInBuf : D == 64 ? kOwn : kInDO;
  static constexpr int ST = D == 64 ? 4 : 2;  // stages of dO and Q
  static constexpr uint32_t STAGE = 2 * TQ;
  // A chain's buffer: P, then dS over it when dV's product has read P (at 64 keys beside it).
  static constexpr uint32_t BUF = 2 * kBox, OFF_DS = KT == 64 ? kBox : 0;
  static constexpr uint32_t OFF_K = 0, OFF_V = TK, OFF_Q = 2 * TK, OFF_P = OFF_Q + ST * STAGE, OFF_O = OFF_P + CH * BUF,
                            OFF_BAR = OFF_O + (OUT == kOwn ? CH * TQ : 0);
  // TMEM: dV, dK, then per chain S and dP, over which dQ is written.
  static constexpr uint32_t COL_DK = D, COL_C = 2 * D, COL_DP = KT, COL_DQ = EARLY ? KT : 0;
  static constexpr uint32_t COLS = EARLY && D > KT ? KT + D : 2 * KT;
  static __device__ __forceinline__ uint32_t dq_place(uint32_t base, int c, int s) {
    return base + (OUT == kOwn ? OFF_O + c * TQ : OUT == kInDO ? OFF_Q + s * STAGE : OFF_P + c * BUF);
  }
  static constexpr int WARP_S = 4 * CH * W, WARP_O = WARP_S + 2, WARP_TMA = WARP_S + (OUT == kInBuf ? 2 : 3);
  static constexpr int THREADS = (WARP_TMA + 1) * 32;
  static constexpr int B_KV = 0, B_KC = 1, B_ACC = 2, B_DRAIN = 3, B_QF = 5, B_QE = B_QF + ST, B_DF = B_QE + ST,
                       B_DE = B_DF + ST, B_SF = B_DE + ST, B_SR = B_SF + CH, B_SP = B_SR + CH, B_PF = B_SP + CH,
                       B_DV = B_PF + CH, B_DS = B_DV + CH, B_GF = B_DS + CH, B_QR = B_GF + CH,
                       B_OW = B_QR + CH, B_OSF = B_OW + CH, B_DX = B_OSF + CH, NBAR = B_DX + 1;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 8u * NBAR, OFF_D = OFF_MISC + 16u;  // D's halves (two threads a row)
  static constexpr uint32_t SMEM = OFF_D + (W == 2 ? 2u * kTile * 4u : 0u) + 1024u;
  static_assert(SMEM <= 232448, "shared memory");
  static_assert(COL_C + CH * COLS <= kTmemCols && COL_DQ + D <= COLS && TQ <= BUF, "TMEM, dQ's places");
};

// p = 2^(s c - lse2) of 32 keys of this thread's row.  MASK here and below: keys from `valid` on count nothing,
// whatever is there.
template <bool MASK>
__device__ __forceinline__ void p_step(const uint32_t (&s)[32], uint64_t c2, uint64_t nl2, int valid, float* p) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, nl2), x0, x1);
    p[e] = MASK && e >= valid ? 0.f : ex2(x0);
    p[e + 1] = MASK && e + 1 >= valid ? 0.f : ex2(x1);
  }
}

// Sum of p dp over them.
template <bool MASK>
__device__ __forceinline__ float dot_step(const float* p, const uint32_t (&dp)[32], int valid) {
  uint64_t a = f2_pack(0.f, 0.f), b = a;
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float d0 = MASK && e >= valid ? 0.f : __uint_as_float(dp[e]);
    const float d1 = MASK && e + 1 >= valid ? 0.f : __uint_as_float(dp[e + 1]);
    if (e & 2) b = f2_fma(f2_pack(p[e], p[e + 1]), f2_pack(d0, d1), b);
    else a = f2_fma(f2_pack(p[e], p[e + 1]), f2_pack(d0, d1), a);
  }
  float s0, s1;
  f2_unpack(f2_add(a, b), s0, s1);
  return s0 + s1;
}

// dS = p (dp - D) of 32 keys, packed.
template <bool MASK>
__device__ __forceinline__ void ds_step(const float* p, const uint32_t (&dp)[32], uint64_t nd2, int valid,
                                        uint32_t* ds) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float s0, s1;
    f2_unpack(f2_mul(f2_pack(p[e], p[e + 1]),
                     f2_add(f2_pack(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])), nd2)),
              s0, s1);
    if (MASK) {
      if (e >= valid) s0 = 0.f;
      if (e + 1 >= valid) s1 = 0.f;
    }
    ds[e / 2] = pack_bf16(s0, s1);
  }
}

// Columns 32 c .. of row r as bf16 into its boxes of 64 columns (128-byte swizzle).
__device__ __forceinline__ void put_cols(uint32_t buf, int r, int c, const uint32_t* v) {
  const uint32_t row = buf + static_cast<uint32_t>(c >> 1) * kBox + static_cast<uint32_t>(r) * 128u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    sts128(row + ((static_cast<uint32_t>(4 * (c & 1) + i) ^ static_cast<uint32_t>(r & 7)) << 4), v[4 * i], v[4 * i + 1],
           v[4 * i + 2], v[4 * i + 3]);
}

// Columns [32 c0, 32 c1) of this thread's row of dQ out of TMEM: to global memory (fp32) or as bf16 into shared memory.
template <int D>
__device__ __forceinline__ void put_dq(void* out, size_t frow, bool valid, uint32_t buf, int r, uint32_t taddr,
                                       float scale, int c0, int c1, int fp32) {
#pragma unroll 2
  for (int c = c0; c < c1; ++c) {
    uint32_t u[32];
    tmem_ld_x32(taddr + 32u * c, u);
    if (!fp32) {
      uint32_t v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = pack_bf16(__uint_as_float(u[2 * i]) * scale, __uint_as_float(u[2 * i + 1]) * scale);
      put_cols(buf, r, c, v);
    } else if (valid) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + frow * D + 32 * c);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        dst[i] = make_float4(__uint_as_float(u[4 * i]) * scale, __uint_as_float(u[4 * i + 1]) * scale,
                             __uint_as_float(u[4 * i + 2]) * scale, __uint_as_float(u[4 * i + 3]) * scale);
    }
  }
}

// This thread's row of dV or dK out of TMEM; zeros where `zero`.
template <int D>
__device__ __forceinline__ void store_sum_row(void* out, size_t row, bool valid, bool zero, uint32_t taddr, float scale,
                                              int fp32) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint32_t u[32];
    tmem_ld_x32(taddr + 32u * c, u);
    if (!valid) continue;
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = zero ? 0.f : __uint_as_float(u[i]) * scale;
    if (fp32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + row * D + 32 * c);
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + row * D + 32 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dst[i] = make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                            pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7]));
    }
  }
}

struct BwdShortArgs {
  const float* lse;
  void *dq, *dk, *dv;  // dk, dv: this call's gradients, or partial sums, part_stride elements apart
  long long part_stride;
  const int* kv_lens;
  int kv_heads, R, Nk, tiles, q_fp32, kv_fp32;
  float sl2, scale;
  unsigned long long budget;
};

template <int D, int KT>
__global__ void __launch_bounds__(BwdShortCfg<D, KT>::THREADS, 1)
    cross_bwd_short_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                           const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                           const __grid_constant__ CUtensorMap tdq, const BwdShortArgs a) {
  using C = BwdShortCfg<D, KT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sK = base + C::OFF_K, sV = base + C::OFF_V, sQ = base + C::OFF_Q, sBar = base + C::OFF_BAR;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_MISC + 4);
#define BAR(i) (sBar + 8u * static_cast<uint32_t>(i))
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_launch();
  const int bh = static_cast<int>(blockIdx.x);
  const int row0 = static_cast<int>(blockIdx.y) * a.tiles * kTile;  // this block's rows
  const int rows = min(a.tiles * kTile, a.R - row0), n = (rows + kTile - 1) / kTile;
  const size_t frow0 = static_cast<size_t>(bh) * a.R + row0, fkey0 = static_cast<size_t>(bh) * a.Nk;
  const size_t part = static_cast<size_t>(blockIdx.y) * static_cast<size_t>(a.part_stride) * (a.kv_fp32 ? 4 : 2);
  uint8_t* dk = static_cast<uint8_t*>(a.dk) + part;
  uint8_t* dv = static_cast<uint8_t*>(a.dv) + part;
  int len = a.Nk;
  if (a.kv_lens) {  // (written, perhaps, by the previous kernel in the stream)
    grid_dep_wait();
    len = min(max(a.kv_lens[bh / a.kv_heads], 0), a.Nk);
  }
  if (len == 0) {  // gradients 0
    grid_dep_wait();
    auto zero = [&](uint8_t* p, size_t first, long long rows_, int fp32) {
      uint4* dst = reinterpret_cast<uint4*>(p + first * D * (fp32 ? 4 : 2));
      const long long vecs = rows_ * D * (fp32 ? 4 : 2) / 16;
      for (long long i = threadIdx.x; i < vecs; i += C::THREADS) dst[i] = make_uint4(0, 0, 0, 0);
    };
    zero(static_cast<uint8_t*>(a.dq), frow0, rows, a.q_fp32);
    zero(dk, fkey0, a.Nk, a.kv_fp32);
    zero(dv, fkey0, a.Nk, a.kv_fp32);
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(BAR(C::B_KV), 1);
    mbar_init(BAR(C::B_KC), 32);
    mbar_init(BAR(C::B_ACC), 1);
    mbar_init(BAR(C::B_DRAIN), 1);
    mbar_init(BAR(C::B_DRAIN + 1), 1);
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(BAR(C::B_QF + s), 1);
      mbar_init(BAR(C::B_QE + s), 1);
      mbar_init(BAR(C::B_DF + s), 1);
      mbar_init(BAR(C::B_DE + s), 1);
    }
    for (int c = 0; c < C::CH; ++c) {
      mbar_init(BAR(C::B_SF + c), 1);           // S computed (two chains: and dP)
      mbar_init(BAR(C::B_SR + c), 128 * C::W);  // S read
      mbar_init(BAR(C::B_SP + c), 1);           // dP computed
      mbar_init(BAR(C::B_PF + c), 128 * C::W);  // P in shared memory (more than 64 keys)
      mbar_init(BAR(C::B_DV + c), 1);           // P read (more than 64 keys)
      mbar_init(BAR(C::B_DS + c), 128 * C::W);  // dS in shared memory
      mbar_init(BAR(C::B_GF + c), 1);           // dQ computed, buffer read
      mbar_init(BAR(C::B_QR + c), 128 * C::W);  // dQ out of TMEM
      mbar_init(BAR(C::B_OW + c), 128 * C::W);  // dQ in shared memory
      mbar_init(BAR(C::B_OSF + c), 1);          // dQ's place free again
    }
    mbar_init(BAR(C::B_DX), 256);  // both halves of D written
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::WARP_S) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  grid_dep_wait();  // every global access below comes after the previous kernel in the stream
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

  if (warp == C::WARP_TMA) {
    // ------------------------------------------------------------ producer
    int issued = 0, q_only = 0;  // tiles asked for; 1: and one more without its dO (after a timeout)
    auto load_q = [&](int k) {
      const uint32_t full = BAR(C::B_QF + k % C::ST);
      mbar_arrive_expect_tx(full, C::EARLY ? C::TQ : C::STAGE);
      for (int h = 0; h < C::NH; ++h)
        tma_load_3d(sQ + (k % C::ST) * C::STAGE + C::TQ + h * kBox, &tq, full, h * 64, row0 + k * kTile, bh);
    };
    auto load_do = [&](int k) {
      const uint32_t full = BAR((C::EARLY ? C::B_DF : C::B_QF) + k % C::ST);
      if (C::EARLY) mbar_arrive_expect_tx(full, C::TQ);
      for (int h = 0; h < C::NH; ++h)
        tma_load_3d(sQ + (k % C::ST) * C::STAGE + h * kBox, &tdo, full, h * 64, row0 + k * kTile, bh);
    };
    if (lane == 0) {
      mbar_arrive_expect_tx(BAR(C::B_KV), 2 * C::TK);
      for (int h = 0; h < C::NH; ++h) {
        tma_load_3d(sK + h * C::KBOX, &tk, BAR(C::B_KV), h * 64, 0, bh);
        tma_load_3d(sV + h * C::KBOX, &tv, BAR(C::B_KV), h * 64, 0, bh);
      }
      for (; issued < min(C::ST, n); ++issued) {
        load_q(issued);
        load_do(issued);
      }
    }
    if (len < a.Nk) {  // K's rows behind the sequence
      __syncwarp();
      if (bwait_all(BAR(C::B_KV), 0, abort_flag, a.budget)) {
        for (int i = len * 8 + lane; i < static_cast<int>(C::KBOX / 16); i += 32)
          for (int h = 0; h < C::NH; ++h) sts128(sK + h * C::KBOX + i * 16, 0, 0, 0, 0);
        fence_proxy_async_smem();
        mbar_arrive(BAR(C::B_KC));
      }
    }
    if (lane == 0) {
      for (; issued < n; ++issued) {
        const int s = issued % C::ST, last = ((issued / C::ST) - 1) & 1;
        if (!bwait(BAR(C::B_QE + s), last, abort_flag, a.budget)) break;
        load_q(issued);
        if (C::EARLY && !bwait(BAR(C::B_DE + s), last, abort_flag, a.budget)) {
          q_only = 1;
          break;
        }
        load_do(issued);
      }
      // every copy lands before the shared memory is released
      bdrain(BAR(C::B_KV), 0, a.budget);
      const int q_end = issued + q_only;
      for (int k = max(0, q_end - C::ST); k < q_end; ++k) bdrain(BAR(C::B_QF + k % C::ST), (k / C::ST) & 1, a.budget);
      for (int k = max(0, issued - C::ST); C::EARLY && k < issued; ++k)
        bdrain(BAR(C::B_DF + k % C::ST), (k / C::ST) & 1, a.budget);
    }
  } else if (C::OUT != C::kInBuf && warp == C::WARP_O) {
    // ------------------------------------------------------------ dQ's stores (bf16; one chain)
    if (lane == 0 && !a.q_fp32) {
      for (int k = 0; k < n; ++k) {
        const int s = k % C::ST;
        if (!bwait(BAR(C::B_OW), k & 1, abort_flag, a.budget)) break;
        for (int h = 0; h < C::NH; ++h)
          tma_store_3d(&tdq, C::dq_place(base, 0, s) + h * kBox, h * 64, row0 + k * kTile, bh);
        bulk_commit();
        bulk_wait_read_all();
        mbar_arrive(BAR(C::OUT == C::kInDO ? C::B_DE + s : C::B_OSF));
      }
      bulk_wait_all();  // complete before the CTA exits
    }
  } else if (warp >= C::WARP_S) {
    // ------------------------------------------------------------ MMA issuers
    if (lane == 0) {
      const uint64_t dk_row = sdesc_sw128(sK, 16, 1024), dv_row = sdesc_sw128(sV, 16, 1024);
      const uint64_t dst_row = sdesc_sw128(sQ, 16, 1024), dst_col = sdesc_sw128(sQ, kBox, 1024);
      bool ok = bwait(BAR(C::B_KV), 0, abort_flag, a.budget) &&
                (len == a.Nk || bwait(BAR(C::B_KC), 0, abort_flag, a.budget));
      if (warp == C::WARP_S) {  // S = Q K^T, dP = dO V^T
        auto product = [&](uint32_t t, uint64_t x, uint64_t y) {
          constexpr uint32_t idesc = idesc_bf16_f32(kTile, KT, 0);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t ox = static_cast<uint32_t>(kk >> 2) * kBox + static_cast<uint32_t>(kk & 3) * 32u;
            const uint32_t oy = static_cast<uint32_t>(kk >> 2) * C::KBOX + static_cast<uint32_t>(kk & 3) * 32u;
            if (kk == 0) mma_ss_c<0>(t, sdesc_add(x, ox), sdesc_add(y, oy), idesc);
            else mma_ss_c<1>(t, sdesc_add(x, ox), sdesc_add(y, oy), idesc);
          }
        };
        for (int k = 0; ok && k < n; ++k) {
          const int c = k % C::CH, s = k % C::ST, last = ((k / C::CH) - 1) & 1;
          const uint32_t t = tmem + C::COL_C + C::COLS * c;
          const uint64_t d_do = sdesc_add(dst_row, s * C::STAGE);
          // the columns are free when the chain's last S is read, and its dQ
          ok = bwait(BAR(C::B_QF + s), (k / C::ST) & 1, abort_flag, a.budget) &&
               (k < C::CH || bwait(BAR((C::EARLY ? C::B_SR : C::B_QR) + c), last, abort_flag, a.budget));
          if (!ok) break;
          tc_fence_after();
          product(t, sdesc_add(d_do, C::TQ), dk_row);
          if (C::EARLY) {
            tc_commit(BAR(C::B_SF + c));
            ok = bwait(BAR(C::B_DF + s), (k / C::ST) & 1, abort_flag, a.budget) &&
                 (k < C::CH || bwait(BAR(C::B_QR + c), last, abort_flag, a.budget));
            if (!ok) break;
            tc_fence_after();
          }
          product(t + C::COL_DP, d_do, dv_row);
          tc_commit(BAR((C::EARLY ? C::B_SP : C::B_SF) + c));
        }
      } else {  // dV += P^T dO, dK += dS^T Q, dQ = dS K
        const uint64_t dk_col = sdesc_sw128(sK, C::KBOX, 1024);
        auto sum = [&](uint32_t acc, uint32_t buf, uint64_t rows_, uint32_t idesc, bool first) {  // 128 rows of queries
          const uint64_t keys = sdesc_sw128(buf, kBox, 1024);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk) {
            if (kk == 0 && first) mma_ss_c<0>(acc, keys, rows_, idesc);
            else mma_ss_c<1>(acc, sdesc_add(keys, 2048u * kk), sdesc_add(rows_, 2048u * kk), idesc);
          }
        };
        for (int k = 0; ok && k < n; ++k) {
          const int c = k % C::CH, s = k % C::ST, i = k / C::CH;
          const uint32_t buf = base + C::OFF_P + c * C::BUF, t_q = tmem + C::COL_C + C::COLS * c + C::COL_DQ;
          const uint64_t d_do = sdesc_add(dst_col, s * C::STAGE), d_q = sdesc_add(d_do, C::TQ);
          if constexpr (KT > 64) {
            ok = bwait(BAR(C::B_PF + c), i & 1, abort_flag, a.budget);
            if (!ok) break;
            tc_fence_after();
            sum(tmem, buf, d_do, idesc_bf16_f32(kTile, D, 1, 1), k == 0);
            tc_commit(BAR(C::B_DV + c));
            if (C::EARLY && (C::OUT != C::kInDO || a.q_fp32)) tc_commit(BAR(C::B_DE + s));
          }
          ok = bwait(BAR(C::B_DS + c), i & 1, abort_flag, a.budget);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ds = sdesc_sw128(buf + C::OFF_DS, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk) {
            const uint32_t off = static_cast<uint32_t>(kk >> 2) * kBox + static_cast<uint32_t>(kk & 3) * 32u;
            if (kk == 0) mma_ss_c<0>(t_q, ds, dk_col, idesc_bf16_f32(kTile, D, 1));
            else mma_ss_c<1>(t_q, sdesc_add(ds, off), sdesc_add(dk_col, 2048u * kk), idesc_bf16_f32(kTile, D, 1));
          }
          // At 64 keys [P dS]^T [dO Q] in one: dV is its upper left quarter and dK its lower right (the others would
          // be padding up to 128 rows).
          if constexpr (KT > 64) sum(tmem + C::COL_DK, buf, d_q, idesc_bf16_f32(kTile, D, 1, 1), k == 0);
          else sum(tmem, buf, d_do, idesc_bf16_f32(kTile, 2 * D, 1, 1), k == 0);
          tc_commit(BAR(C::B_GF + c));
          tc_commit(BAR(C::B_QE + s));
        }
        tc_commit(BAR(C::B_ACC));
      }
      tc_commit(BAR(C::B_DRAIN + (warp - C::WARP_S)));
      bdrain(BAR(C::B_DRAIN + (warp - C::WARP_S)), 0, a.budget);
    }
  } else {
    // ------------------------------------------------------------ elementwise warps
    // Group of four warps g: chain g, or (w) 64 keys of the one chain and half the columns of dQ.
    const int g = warp >> 2, c = g % C::CH, w = g / C::CH, r = 32 * (warp & 3) + lane;
    constexpr int QN = C::W == 2 ? 2 : KT / 32;  // 32-key steps of a thread (KT = 96: the second thread has one)
    const int q0 = 2 * w, qn = min(KT / 32 - q0, QN);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t t_s = lanes + C::COL_C + C::COLS * c, t_dp = t_s + C::COL_DP;
    const uint32_t buf = base + C::OFF_P + static_cast<uint32_t>(c) * C::BUF;
    float* halves = reinterpret_cast<float*>(gbase + C::OFF_D);
    const uint64_t c2 = f2_pack(a.sl2, a.sl2);
    const bool issuer = C::OUT == C::kInBuf && !a.q_fp32 && (warp & 3) == 0 && lane == 0;  // of a chain's stores
    float p[32 * QN];
    auto row_lse = [&](int k) {  // rows past the last: P = 0
      const int row = row0 + k * kTile + r;
      return row < a.R ? a.lse[static_cast<size_t>(bh) * a.R + row] : INFINITY;
    };
    auto masked = [&](int q) { return 32 * (q0 + q) + 32 > len; };
    auto p_of = [&](int q, float lse) {  // (this thread's step q)
      const int k0 = 32 * (q0 + q);
      const uint64_t nl2 = f2_pack(-lse * kLog2e, -lse * kLog2e);
      uint32_t s[32];
      tmem_ld_x32(t_s + k0, s);
      if (masked(q)) p_step<true>(s, c2, nl2, len - k0, p + 32 * q);
      else p_step<false>(s, c2, nl2, 32, p + 32 * q);
    };
    auto dot_of = [&](int q) {
      const int k0 = 32 * (q0 + q);
      uint32_t dp[32];
      tmem_ld_x32(t_dp + k0, dp);
      return masked(q) ? dot_step<true>(p + 32 * q, dp, len - k0) : dot_step<false>(p + 32 * q, dp, 32);
    };
    auto put_p = [&](int q) {
      uint32_t pp[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) pp[e] = pack_bf16(p[32 * q + 2 * e], p[32 * q + 2 * e + 1]);
      put_cols(buf, r, q0 + q, pp);
    };
    float lse = row_lse(c);  // of the chain's next tile, read a tile ahead
    auto take_p = [&](int k) -> bool {
      const float now = lse;
      lse = row_lse(k + 1);
      if (!bwait_all(BAR(C::B_SF), k & 1, abort_flag, a.budget)) return false;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < QN; ++q)
        if (q < qn) p_of(q, now);
      tc_fence_before();
      mbar_arrive(BAR(C::B_SR));
      return true;
    };
    bool ok = !C::EARLY || take_p(0);
    for (int k = c, i = 0; ok && k < n; k += C::CH, ++i) {
      const int row = row0 + k * kTile + r;
      const size_t frow = static_cast<size_t>(bh) * a.R + row;
      float dd = 0.f;
      if constexpr (C::EARLY) {
#pragma unroll
        for (int q = 0; q < QN; ++q)
          if (q < qn) put_p(q);
        fence_proxy_async_smem();
        ok = bwait_all(BAR(C::B_SP), k & 1, abort_flag, a.budget);
        if (!ok) break;
        tc_fence_after();
        // Only now: dP computed says that dO has landed, which dV's issuer does not wait for, and that it is read, before
        // dV's commit may give its place away.
        mbar_arrive(BAR(C::B_PF));
#pragma unroll
        for (int q = 0; q < QN; ++q)
          if (q < qn) dd += dot_of(q);
      } else {
        const float now = lse;
        lse = row_lse(k + C::CH);
        if (issuer) {  // the buffer is free once the last store has read it
          bulk_wait_read_all();
          mbar_arrive(BAR(C::B_OSF + c));
        }
        ok = bwait_all(BAR(C::B_SF + c), i & 1, abort_flag, a.budget);
        if (ok && !a.q_fp32) ok = bwait_all(BAR(C::B_OSF + c), i & 1, abort_flag, a.budget);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < QN; ++q) {
          p_of(q, now);
          dd += dot_of(q);
          put_p(q);
        }
        if constexpr (KT > 64) {
          fence_proxy_async_smem();
          mbar_arrive(BAR(C::B_PF + c));
        }
      }
      if constexpr (C::W == 2) {
        halves[w * kTile + r] = dd;
        mbar_arrive(BAR(C::B_DX));
        ok = bwait_all(BAR(C::B_DX), i & 1, abort_flag, a.budget);
        if (!ok) break;
        dd = halves[r] + halves[kTile + r];
      }
      const uint64_t nd2 = f2_pack(-dd, -dd);
      uint32_t ds[16 * QN];
#pragma unroll
      for (int q = 0; q < QN; ++q) {
        if (q >= qn) continue;
        const int k0 = 32 * (q0 + q);
        uint32_t dp[32];
        tmem_ld_x32(t_dp + k0, dp);
        if (masked(q)) ds_step<true>(p + 32 * q, dp, nd2, len - k0, ds + 16 * q);
        else ds_step<false>(p + 32 * q, dp, nd2, 32, ds + 16 * q);
      }
      if constexpr (KT > 64) {
        ok = bwait_all(BAR(C::B_DV + c), i & 1, abort_flag, a.budget);
        if (!ok) break;
      }
#pragma unroll
      for (int q = 0; q < QN; ++q)
        if (q < qn) put_cols(buf + C::OFF_DS, r, q0 + q, ds + 16 * q);
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(BAR(C::B_DS + c));
      if (C::EARLY && k + 1 < n && !(ok = take_p(k + 1))) break;
      ok = bwait_all(BAR(C::B_GF + c), i & 1, abort_flag, a.budget);
      if (ok && C::OUT == C::kOwn && !a.q_fp32 && i > 0)
        ok = bwait_all(BAR(C::B_OSF + c), (i - 1) & 1, abort_flag, a.budget);
      if (!ok) break;
      tc_fence_after();
      put_dq<D>(a.dq, frow, row < a.R, C::dq_place(base, c, k % C::ST), r, t_s + C::COL_DQ, a.scale,
                w * (D / 32 / C::W), (w + 1) * (D / 32 / C::W), a.q_fp32);
      tc_fence_before();
      mbar_arrive(BAR(C::B_QR + c));
      if (!a.q_fp32) {
        fence_proxy_async_smem();
        mbar_arrive(BAR(C::B_OW + c));
        if (issuer && bwait(BAR(C::B_OW + c), i & 1, abort_flag, a.budget)) {
          for (int h = 0; h < C::NH; ++h)
            tma_store_3d(&tdq, C::dq_place(base, c, k % C::ST) + h * kBox, h * 64, row0 + k * kTile, bh);
          bulk_commit();
        }
        __syncwarp();
      }
    }
    if (ok && (KT > 64 || g == 0) && bwait_all(BAR(C::B_ACC), 0, abort_flag, a.budget)) {
      tc_fence_after();
      const bool is_dk = KT > 64 ? g == 1 : r >= 64;  // (a group each, or its first two warps dV, the others dK)
      const int key = KT > 64 ? r : r & 63;
      store_sum_row<D>(is_dk ? dk : dv, fkey0 + key, key < a.Nk, key >= len, lanes + (is_dk ? C::COL_DK : 0u),
                       is_dk ? a.scale : 1.f, a.kv_fp32);
    }
    if (issuer) bulk_wait_all();  // the stores complete before the CTA exits
    tmem_wait_st();
  }
#undef BAR
  tc_fence_before();
  __syncthreads();
  if (warp == C::WARP_S) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int KT>
cudaError_t launch_t(const BwdLaunch& l, cudaStream_t stream) {
  using C = BwdShortCfg<D, KT>;
  auto kern = cross_bwd_short_kernel<D, KT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  const bool parts = l.kv_splits > 1;
  const long long elems = static_cast<long long>(l.BH) * l.Nk * D;
  float* dv_part = l.kv_part + l.kv_splits * elems;
  const BwdShortArgs args{l.lse, l.dq, parts ? static_cast<void*>(l.kv_part) : l.dk,
                          parts ? static_cast<void*>(dv_part) : l.dv, parts ? elems : 0, l.kv_lens, l.kv_heads, l.N, l.Nk,
                          l.q_tiles, l.grad_fp32, static_cast<int>(parts || l.grad_fp32), l.scale_log2, l.scale,
                          l.budget};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(l.BH), static_cast<unsigned>(l.kv_splits));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kern, l.tq, l.tk, l.tv, l.tdo, l.tdq, args)) != cudaSuccess) return e;
  return parts ? launch_cross_sum(l.kv_part, l.dk, l.dv, elems, l.kv_splits, l.grad_fp32, stream) : cudaSuccess;
}

}  // namespace

cudaError_t launch_cross_bwd_short(const BwdLaunch& l, cudaStream_t stream) {
  if (l.d == 64) {
    if (l.Nk <= 64) return launch_t<64, 64>(l, stream);
    return l.Nk <= 96 ? launch_t<64, 96>(l, stream) : launch_t<64, 128>(l, stream);
  }
  if (l.Nk <= 64) return launch_t<128, 64>(l, stream);
  return l.Nk <= 96 ? launch_t<128, 96>(l, stream) : launch_t<128, 128>(l, stream);
}

cudaError_t cross_bwd_short_status_word(unsigned int** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_bwd_status);
}

}  // namespace fattn
