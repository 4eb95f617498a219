// Cross attention forward over at most 128 keys (fa_cross_fwd with more than 16 rows per key head), for sm_103a: a text
// prompt of 77 tokens or 64 latents under thousands of queries.
//
// There is one tile of keys, so a block loads K and V once and streams query tiles past them: per tile
// S = Q K^T, a softmax with nothing carried over, O = P~ V / l.  Bound by HBM (Q in, O out, 4 d + 4 bytes a row for
// 4 d * keys flops), if the chain of a tile (about 2 us) is hidden: two or three tiles are in flight, each with its own
// S (P~ is packed into it) and U in TMEM, four softmax warps (one thread per row) and MMA-issuing thread.  Measured
// beside plan_short.
//
// Padding behind the sequence: its scores become -inf, and its rows of V are cleared in shared memory, once, since
// P~ = 0 times what they hold would reach U.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"
#include "softmax.cuh"
#include "tmem_io.cuh"

namespace fattn {

static __device__ unsigned int g_short_status = 0;

namespace {

constexpr int kTile = 128;              // query rows per tile
constexpr uint32_t kBox = 128u * 128u;  // bytes of a 128-row x 64-column bf16 box
constexpr uint32_t kTmemCols = 512;
constexpr float kLn2 = 0.6931471805599453f;

// KT: keys of the tile that are computed (64, 96 or 128).
template <int D, int KT>
struct ShortCfg {
  // Tiles in flight (chains): two, or three where TMEM (S and U of each), shared memory and registers hold them
  // (d = 64, 2 x 16 x 8192 rows: 64 keys 18.6 -> 15.7 us).
  static constexpr int CH = D == 64 && KT <= 96 ? 3 : 2;
  static constexpr uint32_t COLS = CH == 2 ? 256 : KT + D;  // TMEM columns of a chain: S (P~ is packed into it), then U
  static constexpr int WARP_MMA = 4 * CH, WARP_TMA = WARP_MMA + CH, THREADS = (WARP_TMA + 1) * 32;
  static constexpr int NH = D / 64;
  static constexpr uint32_t TB = NH * kBox;  // bytes of a 128 x d bf16 tile
  // Ring stages of Q: tile k is chain k % CH's and in stage k % ST, and ST is a multiple of CH, so that a stage is
  // always the same chain's, which then sees each of its phases.  (Otherwise a chain that waits for phase p of a
  // stage could find phase p - 2 when another chain's p - 1 has not landed: a wait by parity must not skip phases.)
  static constexpr int ST = D == 64 ? 2 * CH : CH;
  static constexpr uint32_t OFF_K = 0, OFF_V = TB, OFF_Q = 2 * TB, OFF_O = OFF_Q + ST * TB;  // O: one tile a chain
  static constexpr uint32_t OFF_BAR = OFF_O + CH * TB;
  static constexpr int B_KV = 0, B_VC = 1, B_QF = 2, B_QE = B_QF + ST, B_SF = B_QE + ST, B_PF = B_SF + CH,
                       B_OF = B_PF + CH, B_OSF = B_OF + CH, B_OW = B_OSF + CH, B_DRAIN = B_OW + CH, NBAR = B_DRAIN + CH;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 8u * NBAR;
  static constexpr uint32_t SMEM = OFF_MISC + 16u + 1024u;
  static_assert(SMEM <= 232448, "shared memory");
  static_assert(ST % CH == 0 && CH * COLS <= kTmemCols && KT + D <= COLS, "a stage belongs to one chain");
};

__device__ __forceinline__ bool swait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                      unsigned long long budget) {
  return mbar_wait(bar, parity, abort_flag, budget, &g_short_status);
}
__device__ __forceinline__ bool swait_all(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          unsigned long long budget) {
  return __all_sync(0xffffffffu, swait(bar, parity, abort_flag, budget));
}
__device__ __forceinline__ void sdrain(uint32_t bar, uint32_t parity, unsigned long long budget) {
  mbar_drain(bar, parity, budget, &g_short_status);
}

// N scores of this thread's row (raw fp32 bits); those from `valid` on become -inf.
template <int N>
__device__ __forceinline__ void load_scores(uint32_t taddr, int valid, uint32_t (&s)[N]) {
  if constexpr (N == 64) tmem_ld_x64(taddr, s);
  else tmem_ld_x32(taddr, s);
  if (valid < N) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i >= valid) s[i] = __float_as_uint(-INFINITY);
  }
}

template <int N>
__device__ __forceinline__ float max_of(const uint32_t (&s)[N]) {
  float a[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) a[k] = fmaxf(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1]));
#pragma unroll
  for (int i = 8; i < N; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      a[k] = fmax3(a[k], __uint_as_float(s[i + 2 * k]), __uint_as_float(s[i + 2 * k + 1]));
  return fmax3(a[0], a[1], fmaxf(a[2], a[3]));
}

template <int D, int KT>
__global__ void __launch_bounds__(ShortCfg<D, KT>::THREADS, 1)
    cross_short_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to,
                       const CrossShortArgs a) {
  using C = ShortCfg<D, KT>;
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
  const int n = (min(a.tiles * kTile, a.R - row0) + kTile - 1) / kTile;
  int len = a.Nk;
  if (a.kv_lens) {  // (written, perhaps, by the previous kernel in the stream)
    grid_dep_wait();
    len = min(max(a.kv_lens[bh / a.kv_heads], 0), a.Nk);
  }
  if (len == 0) {  // O = 0, lse = -inf
    grid_dep_wait();
    const size_t frow0 = static_cast<size_t>(bh) * a.R + row0;
    const int rows = min(a.tiles * kTile, a.R - row0), row_bytes = D * (a.o_fp32 ? 4 : 2);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.o) + frow0 * row_bytes);
    const long long vecs = static_cast<long long>(rows) * row_bytes / 16;
    for (long long i = threadIdx.x; i < vecs; i += C::THREADS) dst[i] = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < rows; i += C::THREADS) a.lse[frow0 + i] = -INFINITY;
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(BAR(C::B_KV), 1);
    mbar_init(BAR(C::B_VC), 32);
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(BAR(C::B_QF + s), 1);
      mbar_init(BAR(C::B_QE + s), 1);
    }
    for (int c = 0; c < C::CH; ++c) {
      mbar_init(BAR(C::B_SF + c), 1);
      mbar_init(BAR(C::B_PF + c), 128);
      mbar_init(BAR(C::B_OF + c), 1);
      mbar_init(BAR(C::B_OSF + c), 1);
      mbar_init(BAR(C::B_OW + c), 128);
      mbar_init(BAR(C::B_DRAIN + c), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::WARP_MMA) {
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
    int issued = 0;
    auto load = [&](int k) {
      const int s = k % C::ST;
      mbar_arrive_expect_tx(BAR(C::B_QF + s), C::TB);
      for (int h = 0; h < C::NH; ++h)
        tma_load_3d(sQ + s * C::TB + h * kBox, &tq, BAR(C::B_QF + s), h * 64, row0 + k * kTile, bh);
    };
    if (lane == 0) {
      mbar_arrive_expect_tx(BAR(C::B_KV), 2 * C::TB);
      for (int h = 0; h < C::NH; ++h) {
        tma_load_3d(sK + h * kBox, &tk, BAR(C::B_KV), h * 64, 0, bh);
        tma_load_3d(sV + h * kBox, &tv, BAR(C::B_KV), h * 64, 0, bh);
      }
      for (; issued < min(C::ST, n); ++issued) load(issued);
    }
    if (len < a.Nk) {  // V's rows behind the sequence
      __syncwarp();
      if (swait_all(BAR(C::B_KV), 0, abort_flag, a.budget)) {
        for (int i = len * 8 + lane; i < kTile * 8; i += 32)
          for (int h = 0; h < C::NH; ++h) sts128(sV + h * kBox + i * 16, 0, 0, 0, 0);
        fence_proxy_async_smem();
        mbar_arrive(BAR(C::B_VC));
      }
    }
    if (lane == 0) {
      for (; issued < n; ++issued) {
        if (!swait(BAR(C::B_QE + issued % C::ST), ((issued / C::ST) - 1) & 1, abort_flag, a.budget)) break;
        load(issued);
      }
      // every copy lands before the shared memory is released
      sdrain(BAR(C::B_KV), 0, a.budget);
      for (int k = max(0, issued - C::ST); k < issued; ++k) sdrain(BAR(C::B_QF + k % C::ST), (k / C::ST) & 1, a.budget);
    }
  } else if (warp >= C::WARP_MMA) {
    // ------------------------------------------------------------ MMA issuer of a chain: tiles c, c + CH, ..
    const int c = warp - C::WARP_MMA;
    if (lane == 0 && c < n) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(kTile, KT, 0), idesc_o = idesc_bf16_f32(kTile, D, 1);
      const uint64_t dq = sdesc_sw128(sQ, 16, 1024), dk = sdesc_sw128(sK, 16, 1024), dv = sdesc_sw128(sV, kBox, 1024);
      const uint32_t t_s = tmem + C::COLS * c, t_u = t_s + C::COLS - D;
      bool ok = swait(BAR(C::B_KV), 0, abort_flag, a.budget) &&
                (len == a.Nk || swait(BAR(C::B_VC), 0, abort_flag, a.budget));
      for (int k = c, i = 0; ok && k < n; k += C::CH, ++i) {
        ok = swait(BAR(C::B_QF + k % C::ST), (k / C::ST) & 1, abort_flag, a.budget);
        if (!ok) break;
        tc_fence_after();
        const uint64_t x = sdesc_add(dq, (k % C::ST) * C::TB);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {  // S = Q K^T (over the last P~, which PV below read: MMAs are in order)
          const uint32_t off = static_cast<uint32_t>(kk >> 2) * kBox + static_cast<uint32_t>(kk & 3) * 32u;
          if (kk == 0) mma_ss_c<0>(t_s, sdesc_add(x, off), sdesc_add(dk, off), idesc_s);
          else mma_ss_c<1>(t_s, sdesc_add(x, off), sdesc_add(dk, off), idesc_s);
        }
        tc_commit(BAR(C::B_SF + c));
        tc_commit(BAR(C::B_QE + k % C::ST));
        ok = swait(BAR(C::B_PF + c), i & 1, abort_flag, a.budget);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk) {  // U = P~ V
          if (kk == 0) mma_ts_c<0>(t_u, t_s, dv, idesc_o);
          else mma_ts_c<1>(t_u, t_s + 8u * kk, sdesc_add(dv, 2048u * kk), idesc_o);
        }
        tc_commit(BAR(C::B_OF + c));
      }
      tc_commit(BAR(C::B_DRAIN + c));
      sdrain(BAR(C::B_DRAIN + c), 0, a.budget);
    }
  } else {
    // ------------------------------------------------------------ softmax warps of a chain: thread = query row
    const int c = warp >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t t_s = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + C::COLS * c, t_u = t_s + C::COLS - D;
    const uint32_t stage = base + C::OFF_O + static_cast<uint32_t>(c) * C::TB;
    const uint64_t c2 = f2_pack(a.sl2, a.sl2);
    const bool issuer = (warp & 3) == 0 && lane == 0;  // of the chain's TMA stores
    bool ok = true;
    for (int k = c, i = 0; ok && k < n; k += C::CH, ++i) {
      if (issuer && !a.o_fp32) {  // the staging is free once the last store has read it
        bulk_wait_read_all();
        mbar_arrive(BAR(C::B_OSF + c));
      }
      ok = swait_all(BAR(C::B_SF + c), i & 1, abort_flag, a.budget);
      if (!ok) break;
      tc_fence_after();
      constexpr int N1 = KT == 64 ? 32 : KT - 64;  // scores behind the first 64 (none at KT = 64)
      uint32_t s0[64], s1[N1];
      load_scores(t_s, len, s0);
      float m = max_of(s0);
      if constexpr (KT > 64) {
        load_scores(t_s + 64, len - 64, s1);
        m = fmaxf(m, max_of(s1));
      }
      m *= a.sl2;
      const float mb = m == -INFINITY ? 0.f : m;  // every score -inf: p = 0
      uint64_t rs_a = f2_pack(0.f, 0.f), rs_b = rs_a;
      exp_pack_bf16(s0, c2, f2_pack(-mb, -mb), rs_a, rs_b);
      tmem_st_x32(t_s, *reinterpret_cast<const uint32_t(*)[32]>(s0));
      if constexpr (KT > 64) {
        exp_pack_bf16(s1, c2, f2_pack(-mb, -mb), rs_a, rs_b);
        if constexpr (N1 == 64) tmem_st_x32(t_s + 32, *reinterpret_cast<const uint32_t(*)[32]>(s1));
        else tmem_st_x16(t_s + 32, *reinterpret_cast<const uint32_t(*)[16]>(s1));
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(BAR(C::B_PF + c));
      float x0, x1, x2, x3;
      f2_unpack(rs_a, x0, x1);
      f2_unpack(rs_b, x2, x3);
      const float l = (x0 + x1) + (x2 + x3);  // of the unrounded p, as everywhere in this library
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int row = row0 + k * kTile + r;
      const size_t frow = static_cast<size_t>(bh) * a.R + row;
      if (row < a.R) a.lse[frow] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      ok = swait_all(BAR(C::B_OF + c), i & 1, abort_flag, a.budget);
      if (!ok) break;
      if (!a.o_fp32) ok = swait_all(BAR(C::B_OSF + c), i & 1, abort_flag, a.budget);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < C::NH; ++h) {
        uint32_t u[64];
        tmem_ld_x64(t_u + 64 * h, u);
        if (a.o_fp32) {
          if (row < a.R) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.o) + frow * D + 64 * h);
#pragma unroll
            for (int q = 0; q < 16; ++q)
              dst[q] = make_float4(__uint_as_float(u[4 * q]) * inv, __uint_as_float(u[4 * q + 1]) * inv,
                                   __uint_as_float(u[4 * q + 2]) * inv, __uint_as_float(u[4 * q + 3]) * inv);
          }
        } else {
          const uint32_t srow = stage + h * kBox + static_cast<uint32_t>(r) * 128u;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint32_t* x = u + 8 * q;
            sts128(srow + ((static_cast<uint32_t>(q) ^ static_cast<uint32_t>(r & 7)) << 4),
                   pack_bf16(__uint_as_float(x[0]) * inv, __uint_as_float(x[1]) * inv),
                   pack_bf16(__uint_as_float(x[2]) * inv, __uint_as_float(x[3]) * inv),
                   pack_bf16(__uint_as_float(x[4]) * inv, __uint_as_float(x[5]) * inv),
                   pack_bf16(__uint_as_float(x[6]) * inv, __uint_as_float(x[7]) * inv));
          }
        }
      }
      // (the U loads above complete before this thread's next P~-ready arrival, after which U is overwritten)
      if (!a.o_fp32) {
        fence_proxy_async_smem();
        mbar_arrive(BAR(C::B_OW + c));
        if (issuer) {
          ok = swait(BAR(C::B_OW + c), i & 1, abort_flag, a.budget);
          if (ok) {
            for (int h = 0; h < C::NH; ++h) tma_store_3d(&to, stage + h * kBox, h * 64, row0 + k * kTile, bh);
            bulk_commit();
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    if (issuer) bulk_wait_all();  // the stores complete before the CTA exits
    tmem_wait_st();
  }
#undef BAR
  tc_fence_before();
  __syncthreads();
  if (warp == C::WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int KT>
cudaError_t launch_t(const CrossShortLaunch& l, cudaStream_t stream) {
  using C = ShortCfg<D, KT>;
  auto kern = cross_short_kernel<D, KT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  const long long block_rows = static_cast<long long>(l.args.tiles) * kTile;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(l.BH), static_cast<unsigned>((l.args.R + block_rows - 1) / block_rows));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, l.tq, l.tk, l.tv, l.to, l.args);
}

}  // namespace

cudaError_t launch_cross_short(const CrossShortLaunch& l, cudaStream_t stream) {
  const int Nk = l.args.Nk;
  if (l.d == 64) {
    if (Nk <= 64) return launch_t<64, 64>(l, stream);
    return Nk <= 96 ? launch_t<64, 96>(l, stream) : launch_t<64, 128>(l, stream);
  }
  if (Nk <= 64) return launch_t<128, 64>(l, stream);
  return Nk <= 96 ? launch_t<128, 96>(l, stream) : launch_t<128, 128>(l, stream);
}

cudaError_t cross_short_status_word(unsigned int** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_short_status);
}

}  // namespace fattn
