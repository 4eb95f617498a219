// Backward of causal attention with a sliding window and sinks (fa_window_fwd.cu) for sm_103a: dK, dV (one CTA per key
// tile and range of its queries) and dQ (one per few query tiles, one after another), by the formulas of fa_bwd.cu, P
// recomputed from the forward's lse.  The scanned side is taken in halves of 64 rows, two or three in flight, as
// in fa_cross_bwd.cu.
//
// dK, dV.  The queries that see a key tile are the rows n0 .. of every query head that shares the key head, for each
// head the tile's window, W + 127 of them: the block takes them as one list of 128-row stages.  Key tile 0 holds
// the sinks (at most 128), which every later query sees: its list is all the queries, as long as many windows, and is
// cut into ranges of about a window's length whose fp32 partial sums a last kernel adds in their order.  So are
// the lists of all tiles where there are too few blocks to fill the SMs.
//
// dQ.  A query tile scans the sinks before its first row's window (through tensor maps that end behind the sinks), then
// the keys from that window's first, lo, up to its last row's own.
//
// Hidden pairs are cleared after the arithmetic, so that keys which no query sees get a gradient of 0 whatever
// they hold.
#include <cuda_bf16.h>

#include "bwd_halves.cuh"
#include "window.cuh"

namespace fattn {
namespace {

// Elementwise step of the dK/dV kernel on 32 query columns of one key row: P^T = 2^(S^T c - lse2),
// dS^T = P^T (dP^T - D) as bf16 pairs.  MASK: only the columns of `seen`.
template <bool MASK>
__device__ __forceinline__ void ew_window_dkdv(const uint32_t (&sv)[32], const uint32_t (&pv)[32], const float4* nv,
                                               uint64_t c2, int col0, uint32_t seen, uint32_t (&pp)[16],
                                               uint32_t (&dp)[16]) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float4 x = nv[(col0 + e) >> 1];
    float x0, x1, s0, s1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), c2, f2_pack(x.x, x.y)), x0, x1);
    float p0 = ex2(x0), p1 = ex2(x1);
    f2_unpack(f2_mul(f2_pack(p0, p1), f2_add(f2_pack(__uint_as_float(pv[e]), __uint_as_float(pv[e + 1])), f2_pack(x.z, x.w))),
              s0, s1);
    if (MASK) {
      if (!(seen & (1u << e))) p0 = s0 = 0.f;
      if (!(seen & (2u << e))) p1 = s1 = 0.f;
    }
    pp[e / 2] = pack_bf16(p0, p1);
    dp[e / 2] = pack_bf16(s0, s1);
  }
}

// The same of the dQ kernel on 32 key columns of one query row: dS alone.
template <bool MASK>
__device__ __forceinline__ void ew_window_dq(const uint32_t (&sv)[32], const uint32_t (&pv)[32], uint64_t c2,
                                             uint64_t nl2, uint64_t nd2, uint32_t seen, uint32_t (&dp)[16]) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float x0, x1, s0, s1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), c2, nl2), x0, x1);
    const float p0 = ex2(x0), p1 = ex2(x1);
    f2_unpack(f2_mul(f2_pack(p0, p1), f2_add(f2_pack(__uint_as_float(pv[e]), __uint_as_float(pv[e + 1])), nd2)), s0, s1);
    if (MASK) {
      if (!(seen & (1u << e))) s0 = 0.f;
      if (!(seen & (2u << e))) s1 = 0.f;
    }
    dp[e / 2] = pack_bf16(s0, s1);
  }
}

// One CTA per key tile of a key head and range of the tile's stages: blockIdx (x, y) in groups of heads, y the ranges
// of tile 0, then those of tile 1, ...  P^T and dS^T are packed into their S^T and dP^T.
template <int D>
__global__ void __launch_bounds__(CrossCfg<D, 2 * D>::THREADS, 1)
    window_dkdv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                       const __grid_constant__ CUtensorMap tdk, const __grid_constant__ CUtensorMap tdv,
                       const WindowBwdArgs a) {
  using C = CrossCfg<D, 2 * D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sK = base + C::OFF_A, sV = base + C::OFF_B, sRing = base + C::OFF_RING, sBar = base + C::OFF_BAR;
  float* vec = reinterpret_cast<float*>(gbase + C::OFF_VEC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_MISC + 4);
#define BAR(i) (sBar + 8u * static_cast<uint32_t>(i))
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, N = a.N;
  const unsigned long long budget = a.budget;
  int bh, rank;
  grouped_block(a.ng, bh, rank);
  const int kt = rank < a.splits0 ? 0 : 1 + (rank - a.splits0) / a.splits;
  const int z = kt == 0 ? rank : (rank - a.splits0) % a.splits;
  const bool part = (kt == 0 ? a.splits0 : a.splits) > 1;
  const bool grad_fp32 = part || a.grad_fp32;
  const int off = a.Nk - N, k0 = kt * kTile;
  // The tile's stages: per query head rows n0 + 128 i of the head, ns of them; this block's are s0 ..
  const int n0 = max(0, k0 - off);
  const int n1 = kt == 0 && a.sinks > 0 ? N - 1 : min(N - 1, k0 + kTile - 1 + a.window - 1 - off);
  const int ns = n1 < n0 ? 0 : (n1 - n0) / kTile + 1;
  const int each = kt == 0 ? a.stages0 : a.stages;
  const int s0 = z * each, n_i = min(each, ns * a.group - s0), n_h = 2 * n_i;
  // where its gradients go: the tensors (rows of key head bh), or its partial sums
  const size_t g0 = part && kt == 0 ? static_cast<size_t>(bh) * kTile : static_cast<size_t>(bh) * a.Nk + k0;
  float* pk = a.part0 + static_cast<size_t>(z) * a.stride0;
  float* pv_ = pk + static_cast<size_t>(a.splits0) * a.stride0;
  if (part && kt > 0) {
    pk = a.part + static_cast<size_t>(z) * a.stride;
    pv_ = pk + static_cast<size_t>(a.splits) * a.stride;
  }
  void* const dk = part ? pk : a.dk;
  void* const dv = part ? pv_ : a.dv;
  const int rows = min(kTile, a.Nk - k0);
  if (n_i <= 0) {  // no query sees the tile
    zero_rows<D>(dk, g0, rows, grad_fp32);
    zero_rows<D>(dv, g0, rows, grad_fp32);
    wait_as_last_block();
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(BAR(C::B_OWN), 1);
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(BAR(C::B_FULL + s), 1 + 32);  // TMA bytes + the producer warp's lse/D stores
      mbar_init(BAR(C::B_EMPTY + s), 2);      // dV and dK have read the stage
    }
    for (int g = 0; g < C::FLIGHT; ++g) {
      mbar_init(BAR(C::B_SF + g), 1);
      mbar_init(BAR(C::B_GD + g), 2);  // the pair's gradient MMAs are complete
    }
    for (int c = 0; c < 2 * C::FLIGHT; ++c) mbar_init(BAR(C::B_PF + c), 128);
    mbar_init(BAR(C::B_GF), 2);
    for (int i = 0; i < kIssuers; ++i) mbar_init(BAR(C::B_DRAIN + i), 1);
    mbar_init(BAR(C::B_OW), 128);
    mbar_init(BAR(C::B_OW + 1), 128);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::MMA) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  constexpr uint32_t kV = C::COL_ACC, kK = C::COL_ACC + D;

  if (warp == C::TMA) {
    // ------------------------------------------------------------ producer (whole warp)
    if (lane == 0) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tdo);
      mbar_arrive_expect_tx(BAR(C::B_OWN), 2 * C::TB);
      for (int h = 0; h < C::NH; ++h) {
        tma_load_3d(sK + h * kBox, &tk, BAR(C::B_OWN), h * 64, k0, bh);
        tma_load_3d(sV + h * kBox, &tv, BAR(C::B_OWN), h * 64, k0, bh);
      }
    }
    int issued = 0;
    for (int i = 0; i < n_i; ++i) {
      const int s = i % C::ST;
      const int qh = bh * a.group + (s0 + i) / ns, row = n0 + (s0 + i) % ns * kTile;
      if (i >= C::ST && !bwait_all(BAR(C::B_EMPTY + s), ((i / C::ST) - 1) & 1, abort_flag, budget)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(BAR(C::B_FULL + s), 2 * C::TB);
        const uint32_t st = sRing + s * C::STAGE;
        for (int h = 0; h < C::NH; ++h) {
          tma_load_3d(st + h * kBox, &tq, BAR(C::B_FULL + s), h * 64, row, qh);
          tma_load_3d(st + C::TB + h * kBox, &tdo, BAR(C::B_FULL + s), h * 64, row, qh);
        }
      }
      if (i == 0) {
        // Launched programmatically: D comes from the kernel before.  The dQ kernel, which reads it too, may then take
        // SMs as this grid's last round leaves them idle.
        grid_dep_wait();
        grid_dep_launch();
      }
      float* vs = vec + s * (2 * kTile);
#pragma unroll
      for (int c = 0; c < kTile / 32; ++c) {  // rows past N get -lse = -inf, so P = 0
        const int col = 32 * c + lane, r = row + col;
        const bool in = r < N;
        vs[4 * (col >> 1) + (col & 1)] = in ? -a.lse[static_cast<size_t>(qh) * N + r] * kLog2e : -INFINITY;
        vs[4 * (col >> 1) + 2 + (col & 1)] = in ? -a.delta[static_cast<size_t>(qh) * N + r] : 0.f;
      }
      mbar_arrive(BAR(C::B_FULL + s));
      issued = i + 1;
    }
    if (lane == 0) {
      bdrain(BAR(C::B_OWN), 0, budget);
      for (int i = max(0, issued - C::ST); i < issued; ++i) bdrain(BAR(C::B_FULL + i % C::ST), (i / C::ST) & 1, budget);
    }
  } else if (warp >= C::MMA) {
    // ------------------------------------------------------------ MMA issuers: the products, dV, dK
    if (elect_one()) {
      const int role = warp - C::MMA;
      bool ok = true;
      if (role == 0) {
        const uint64_t dK = sdesc_sw128(sK, 16, 1024), dV = sdesc_sw128(sV, 16, 1024), dR = sdesc_sw128(sRing, 16, 1024);
        ok = bwait(BAR(C::B_OWN), 0, abort_flag, budget);
        for (int hh = 0; ok && hh < n_h; ++hh) {
          const int i = hh >> 1, g = hh % C::FLIGHT;
          // the stage loaded, and the pair's last gradients done with its columns
          ok = bwait(BAR(C::B_FULL + i % C::ST), (i / C::ST) & 1, abort_flag, budget) &&
               (hh < C::FLIGHT || bwait(BAR(C::B_GD + g), ((hh / C::FLIGHT) - 1) & 1, abort_flag, budget));
          if (!ok) break;
          tc_fence_after();
          const uint32_t st = (i % C::ST) * C::STAGE, d = tmem + kPair * g;
          issue_half_product<D>(d, dK, sdesc_add(dR, st), hh & 1);               // S^T = K Q^T
          issue_half_product<D>(d + 64, dV, sdesc_add(dR, st + C::TB), hh & 1);  // dP^T = V dO^T
          tc_commit(BAR(C::B_SF + g));
        }
      } else {
        // dV += P^T dO (role 1), dK += dS^T Q (role 2)
        const uint64_t dY = sdesc_add(sdesc_sw128(sRing, kBox, 1024), role == 1 ? C::TB : 0u);
        const uint32_t acc = tmem + (role == 1 ? kV : kK), x0 = tmem + (role == 1 ? 0u : 64u);
        for (int hh = 0; ok && hh < n_h; ++hh) {
          const int g = hh % C::FLIGHT;
          const uint64_t dy = sdesc_add(dY, ((hh >> 1) % C::ST) * C::STAGE);
          for (int c = 0; ok && c < 2; ++c) {
            ok = bwait(BAR(C::B_PF + 2 * g + c), (hh / C::FLIGHT) & 1, abort_flag, budget);
            if (!ok) break;
            tc_fence_after();
            issue_half_chunk<D>(acc, x0 + kPair * g, dy, hh & 1, c, hh > 0 || c > 0);
          }
          if (!ok) break;
          tc_commit(BAR(C::B_GD + g));
          if (hh & 1) tc_commit(BAR(C::B_EMPTY + (hh >> 1) % C::ST));
        }
        tc_commit(BAR(C::B_GF));
      }
      tc_commit(BAR(C::B_DRAIN + role));
      bdrain(BAR(C::B_DRAIN + role), 0, budget);
    }
  } else {
    // ------------------------------------------------------------ elementwise warps: thread = key row
    const int g = warp >> 2, r = 32 * (warp & 3) + lane, key = k0 + r;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t tS = lanes + kPair * g, tP = tS + 64;
    const uint64_t c2 = f2_pack(a.sl2, a.sl2);
    bool ok = true;
    for (int hh = g; ok && hh < n_h; hh += C::FLIGHT) {
      const int i = hh >> 1, s = i % C::ST;
      const int pos = off + n0 + (s0 + i) % ns * kTile + kHalf * (hh & 1);  // of the half's first query
      ok = bwait_all(BAR(C::B_FULL + s), (i / C::ST) & 1, abort_flag, budget) &&
           bwait_all(BAR(C::B_SF + g), (hh / C::FLIGHT) & 1, abort_flag, budget);
      if (!ok) break;
      tc_fence_after();
      const float4* nv = reinterpret_cast<const float4*>(vec + s * (2 * kTile));
      const bool all = pos >= key && (key < a.sinks || pos + kHalf <= key + a.window);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t sv[32], pv[32];
        tmem_ld_x32(tS + 32 * c, sv);
        tmem_ld_x32(tP + 32 * c, pv);
        uint32_t pp[16], dp[16];
        const int col0 = kHalf * (hh & 1) + 32 * c;
        if (all) ew_window_dkdv<false>(sv, pv, nv, c2, col0, 0u, pp, dp);
        else ew_window_dkdv<true>(sv, pv, nv, c2, col0, visible_queries(pos + 32 * c, key, a.window, a.sinks), pp, dp);
        tmem_st_x16(tS + 16 * c, pp);
        tmem_st_x16(tP + 16 * c, dp);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(BAR(C::B_PF + 2 * g + c));
      }
    }
    if (ok) ok = bwait_all(BAR(C::B_GF), 0, abort_flag, budget);
    if (ok) {
      tc_fence_after();
      if (grad_fp32) {
        if (g == 0) store_grad_row<D>(dv, g0 + r, r < rows, lanes + kV, 1.f);
        if (g == 1) store_grad_row<D>(dk, g0 + r, r < rows, lanes + kK, a.scale);
      } else if (g < 2) {  // through shared memory: the V and K tiles have their shape and are no longer read
        const uint32_t tile = g == 0 ? sV : sK;
        stage_row_bf16<D>(tile, tile + kBox, r, lanes + (g == 0 ? kV : kK), g == 0 ? 1.f : a.scale);
        mbar_arrive(BAR(C::B_OW + g));
        if ((warp & 3) == 0 && lane == 0 && bwait(BAR(C::B_OW + g), 0, abort_flag, budget)) {
          for (int h = 0; h < C::NH; ++h) tma_store_3d(g == 0 ? &tdv : &tdk, tile + h * kBox, h * 64, k0, bh);
          bulk_commit();
          bulk_wait_all();  // complete before the CTA exits
        }
      }
    }
    tmem_wait_st();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// What the query tile from row `row` on scans, in halves of 64 keys: `hs` of the sinks before its first window (in a
// stage of their own), then those from key lo on.
struct DqTile {
  int lo, n_sink, hs, n_h, n_j;
  __device__ __forceinline__ DqTile(const WindowBwdArgs& a, int row) {
    const int off = a.Nk - a.N;
    lo = max(0, off + row - a.window + 1);
    n_sink = min(a.sinks, lo);
    hs = (n_sink + kHalf - 1) / kHalf;
    const int hw = (off + min(row + kTile, a.N) - lo + kHalf - 1) / kHalf;
    n_h = hs + hw;
    n_j = (hs > 0 ? 1 : 0) + (hw + 1) / 2;
  }
  __device__ __forceinline__ int stage(int hh) const { return hh < hs ? 0 : (hs > 0 ? 1 : 0) + (hh - hs) / 2; }
  __device__ __forceinline__ int half(int hh) const { return hh < hs ? hh : (hh - hs) & 1; }
  __device__ __forceinline__ bool ends_stage(int hh) const { return hh + 1 == hs || hh + 1 == n_h || (hh >= hs && half(hh)); }
};

// One CTA per a.own_tiles query tiles of a query head, scanned one after another, the next one's Q, dO and first keys
// on their way meanwhile.  Halves and stages are counted over all its tiles, so that their phases go on.  dS is
// packed into its dP.
template <int D>
__global__ void __launch_bounds__(CrossCfg<D, D>::THREADS, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tks,
                     const __grid_constant__ CUtensorMap tvs, const __grid_constant__ CUtensorMap tdo,
                     const __grid_constant__ CUtensorMap tdq, const WindowBwdArgs a) {
  using C = CrossCfg<D, D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sOwn = base + C::OFF_A, sRing = base + C::OFF_RING, sBar = base + C::OFF_BAR;  // own: Q, dO
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, N = a.N;
  const unsigned long long budget = a.budget;
  int bh, qb;
  grouped_block(a.ng_q, bh, qb);
  qb = static_cast<int>(gridDim.y) - 1 - qb;  // the rows with whole windows first
  const int t0 = qb * a.own_tiles, nt = min(a.own_tiles, (N + kTile - 1) / kTile - t0), kh = bh / a.group;
  const bool producer = threadIdx.x == C::TMA * 32;
  auto keys_of = [&](int t) { return DqTile(a, (t0 + t) * kTile); };
  if (producer) {
    for (int b = 0; b < C::NB; ++b) {
      mbar_init(BAR(C::B_OWN + b), 1);
      mbar_init(BAR(C::B_GF + b), 1);    // the tile's dQ is complete
      mbar_init(BAR(C::B_OW + b), 128);  // and out of TMEM (bf16: in Q's place)
    }
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(BAR(C::B_FULL + s), 1);
      mbar_init(BAR(C::B_EMPTY + s), 1);
    }
    for (int g = 0; g < C::FLIGHT; ++g) {
      mbar_init(BAR(C::B_SF + g), 2);  // S and dP
      mbar_init(BAR(C::B_GD + g), 1);  // the pair's dQ MMAs are complete
    }
    for (int c = 0; c < 2 * C::FLIGHT; ++c) mbar_init(BAR(C::B_PF + c), 128);
    for (int i = 0; i < kIssuers; ++i) mbar_init(BAR(C::B_DRAIN + i), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  auto load = [&](int jj, const DqTile& k, int j) {  // stage j of a tile as the block's stage jj
    const int s = jj % C::ST;
    const bool sink = k.hs > 0 && j == 0;
    const int key = sink ? 0 : k.lo + (j - (k.hs > 0 ? 1 : 0)) * kTile;
    const uint32_t st = sRing + s * C::STAGE;
    mbar_arrive_expect_tx(BAR(C::B_FULL + s), 2 * C::TB);
    for (int h = 0; h < C::NH; ++h) {
      tma_load_3d(st + h * kBox, sink ? &tks : &tk, BAR(C::B_FULL + s), h * 64, key, kh);
      tma_load_3d(st + C::TB + h * kBox, sink ? &tvs : &tv, BAR(C::B_FULL + s), h * 64, key, kh);
    }
  };
  auto load_own = [&](int t) {  // Q, dO of the block's tile t
    const uint32_t full = BAR(C::B_OWN + t % C::NB), own = sOwn + t % C::NB * (2 * C::TB);
    mbar_arrive_expect_tx(full, 2 * C::TB);
    for (int h = 0; h < C::NH; ++h) {
      tma_load_3d(own + h * kBox, &tq, full, h * 64, (t0 + t) * kTile, bh);
      tma_load_3d(own + C::OFF_B + h * kBox, &tdo, full, h * 64, (t0 + t) * kTile, bh);
    }
  };
  const int first = min(C::ST, keys_of(0).n_j);  // stages asked for at once
  if (producer) {
    const DqTile k = keys_of(0);
    load_own(0);
    for (int j = 0; j < first; ++j) load(j, k, j);
    if (C::NB > 1 && nt > 1) load_own(1);
  }
  if (warp == C::MMA) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

  if (warp == C::TMA) {
    if (lane == 0) {
      int issued = first, owned = min(C::NB, nt), before = 0;  // stages, tiles, stages of the tiles before
      bool ok = true;
      auto finish = [&](int t) {  // tile t's dQ: stored from Q's place, which is then free, as dO's
        ok = bwait(BAR(C::B_OW + t % C::NB), (t / C::NB) & 1, abort_flag, budget);
        if (!ok || a.grad_fp32) return;
        for (int h = 0; h < C::NH; ++h)
          tma_store_3d(&tdq, sOwn + t % C::NB * (2 * C::TB) + h * kBox, h * 64, (t0 + t) * kTile, bh);
        bulk_commit();
        bulk_wait_read_all();
      };
      int done = 0;  // tiles finished
      for (int t = 0; ok && t < nt; ++t) {
        const DqTile k = keys_of(t);
        auto take = [&](int end) {  // the tile's stages before `end`
          for (; ok && issued < before + end; ++issued) {
            const int s = issued % C::ST;
            if (issued >= C::ST) ok = bwait(BAR(C::B_EMPTY + s), ((issued / C::ST) - 1) & 1, abort_flag, budget);
            if (!ok) return;
            load(issued, k, issued - before);
          }
        };
        take(min(C::ST, k.n_j));
        if (ok && t > 0) {
          finish(done++);
          if (ok && owned < nt) load_own(owned++);
        }
        take(k.n_j);
        before += k.n_j;
      }
      // every copy lands before the shared memory is released
      for (int t = max(0, owned - C::NB); t < owned; ++t) bdrain(BAR(C::B_OWN + t % C::NB), (t / C::NB) & 1, budget);
      for (int j = max(0, issued - C::ST); j < issued; ++j) bdrain(BAR(C::B_FULL + j % C::ST), (j / C::ST) & 1, budget);
      while (ok && done < nt) finish(done++);
      bulk_wait_all();  // the stores complete before the CTA exits
    }
  } else if (warp >= C::MMA) {
    // ------------------------------------------------------------ MMA issuers: S, dP, dQ
    if (elect_one()) {
      const int role = warp - C::MMA;
      bool ok = true;
      int H = 0, jc = 0;  // halves so far, stages of the tiles before
      if (role < 2) {     // S = Q K^T, dP = dO V^T
        const uint64_t dA = sdesc_add(sdesc_sw128(sOwn, 16, 1024), role == 0 ? 0u : C::OFF_B);
        const uint64_t dR = sdesc_add(sdesc_sw128(sRing, 16, 1024), role == 0 ? 0u : C::TB);
        for (int t = 0; ok && t < nt; ++t) {
          const DqTile k = keys_of(t);
          ok = bwait(BAR(C::B_OWN + t % C::NB), (t / C::NB) & 1, abort_flag, budget);
          for (int hh = 0; ok && hh < k.n_h; ++hh, ++H) {
            const int J = jc + k.stage(hh), g = H % C::FLIGHT, s = J % C::ST;
            // the stage loaded, and the pair's last dQ MMAs done with its columns
            ok = bwait(BAR(C::B_FULL + s), (J / C::ST) & 1, abort_flag, budget) &&
                 (H < C::FLIGHT || bwait(BAR(C::B_GD + g), ((H / C::FLIGHT) - 1) & 1, abort_flag, budget));
            if (!ok) break;
            tc_fence_after();
            issue_half_product<D>(tmem + kPair * g + 64 * role, sdesc_add(dA, t % C::NB * (2 * C::TB)),
                                  sdesc_add(dR, s * C::STAGE), k.half(hh));
            tc_commit(BAR(C::B_SF + g));
          }
          jc += k.n_j;
        }
      } else {  // dQ += dS K
        const uint64_t dRmn = sdesc_sw128(sRing, kBox, 1024);
        for (int t = 0; ok && t < nt; ++t) {
          const DqTile k = keys_of(t);
          const int b = t % C::NB;
          if (t >= C::NB) {  // the accumulator's last tile is out
            ok = bwait(BAR(C::B_OW + b), ((t / C::NB) - 1) & 1, abort_flag, budget);
            if (!ok) break;
          }
          for (int hh = 0; ok && hh < k.n_h; ++hh, ++H) {
            const int s = (jc + k.stage(hh)) % C::ST, g = H % C::FLIGHT;
            for (int c = 0; ok && c < 2; ++c) {
              ok = bwait(BAR(C::B_PF + 2 * g + c), (H / C::FLIGHT) & 1, abort_flag, budget);
              if (!ok) break;
              tc_fence_after();
              issue_half_chunk<D>(tmem + C::COL_ACC + b * D, tmem + kPair * g + 64, sdesc_add(dRmn, s * C::STAGE),
                                  k.half(hh), c, hh > 0 || c > 0);
            }
            if (!ok) break;
            tc_commit(BAR(C::B_GD + g));
            if (k.ends_stage(hh)) tc_commit(BAR(C::B_EMPTY + s));
          }
          if (ok) tc_commit(BAR(C::B_GF + b));
          jc += k.n_j;
        }
      }
      tc_commit(BAR(C::B_DRAIN + role));
      bdrain(BAR(C::B_DRAIN + role), 0, budget);
    }
  } else {
    // ------------------------------------------------------------ elementwise warps: thread = query row
    const int g = warp >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t tS = lanes + kPair * g, tP = tS + 64;
    const uint64_t c2 = f2_pack(a.sl2, a.sl2);
    bool ok = true;
    int out = 0;  // tiles whose dQ is out (the first four warps take them out of TMEM)
    auto put_out = [&](int t) {
      const int b = t % C::NB, row = (t0 + t) * kTile + r;
      ok = bwait_all(BAR(C::B_GF + b), (t / C::NB) & 1, abort_flag, budget);
      if (!ok) return;
      tc_fence_after();
      const uint32_t acc = lanes + C::COL_ACC + b * D, place = sOwn + b * (2 * C::TB);
      if (a.grad_fp32) store_grad_row<D>(a.dq, static_cast<size_t>(bh) * N + row, row < N, acc, a.scale);
      else stage_row_bf16<D>(place, place + kBox, r, acc, a.scale);  // (its Q is no longer read)
      tc_fence_before();
      mbar_arrive(BAR(C::B_OW + b));
    };
    auto row_of = [&](const float* v, int t, float past) {
      const int row = (t0 + t) * kTile + r;
      return row < N ? v[static_cast<size_t>(bh) * N + row] : past;
    };
    DqTile k = keys_of(0);
    float lse_n = row_of(a.lse, 0, INFINITY), dd_n = row_of(a.delta, 0, 0.f);  // of tile t + 1, read a tile ahead
    int t = -1, hh = g, i = 0;
    uint64_t nl2 = 0, nd2 = 0;
    for (int tile = 0; ok; hh += C::FLIGHT, ++i) {
      while (tile < nt && hh >= k.n_h) {
        hh -= k.n_h;
        if (++tile < nt) k = keys_of(tile);
      }
      if (g == 0)
        while (ok && out < tile) put_out(out++);
      if (!ok || tile >= nt) break;
      if (tile != t) {
        const bool next = tile == t + 1;
        t = tile;
        const float lse2 = (next ? lse_n : row_of(a.lse, t, INFINITY)) * kLog2e;
        const float dd = next ? dd_n : row_of(a.delta, t, 0.f);
        nl2 = f2_pack(-lse2, -lse2);
        nd2 = f2_pack(-dd, -dd);
        if (t + 1 < nt) {
          lse_n = row_of(a.lse, t + 1, INFINITY);
          dd_n = row_of(a.delta, t + 1, 0.f);
        }
      }
      ok = bwait_all(BAR(C::B_SF + g), i & 1, abort_flag, budget);
      if (!ok) break;
      tc_fence_after();
      // the half's keys and what the row sees of them; the sinks' halves show their n_sink keys to every row
      const bool sink = hh < k.hs;
      const int key0 = sink ? hh * kHalf : k.lo + (hh - k.hs) * kHalf;
      const int upto = sink ? k.n_sink - 1 : a.Nk - N + (t0 + t) * kTile + r, sinks = sink ? kTile : a.sinks;
      const bool all = key0 + kHalf - 1 <= upto && (key0 > upto - a.window || key0 + kHalf <= sinks);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t sv[32], pv[32];
        tmem_ld_x32(tS + 32 * c, sv);
        tmem_ld_x32(tP + 32 * c, pv);
        uint32_t dp[16];
        if (all) ew_window_dq<false>(sv, pv, c2, nl2, nd2, 0u, dp);
        else ew_window_dq<true>(sv, pv, c2, nl2, nd2, visible_keys(key0 + 32 * c, upto, a.window, sinks), dp);
        tmem_st_x16(tP + 16 * c, dp);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(BAR(C::B_PF + 2 * g + c));
      }
    }
    tmem_wait_st();
  }
#undef BAR
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  wait_as_last_block();
}

// dK (blockIdx.y = 0) and dV (1) from the partial sums, in their order; 4 elements a thread, rows first .. last - 1 of
// each key head.
template <int D>
__global__ void __launch_bounds__(256) window_sum_kernel(const WindowBwdArgs a, int first, int last) {
  const long long e = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * 4;
  const int per_head = (last - first) * D;
  grid_dep_wait();  // launched programmatically after the kernels that leave the partial sums
  const long long bh = e / per_head;
  const int in_head = static_cast<int>(e - bh * per_head), row = first + in_head / D, col = in_head % D;
  if (bh >= a.kv_heads) return;
  const bool tile0 = row < kTile;
  const int S = tile0 ? a.splits0 : a.splits;
  const size_t out = (static_cast<size_t>(bh) * a.Nk + row) * D + col;
  const size_t stride = static_cast<size_t>(tile0 ? a.stride0 : a.stride);
  const float* p = (tile0 ? a.part0 + (static_cast<size_t>(bh) * kTile + row) * D + col : a.part + out) + blockIdx.y * S * stride;
  if (S < 2) return;  // (those rows are written already)
  float4 acc = *reinterpret_cast<const float4*>(p);
  for (int s = 1; s < S; ++s) {
    const float4 y = *reinterpret_cast<const float4*>(p + s * stride);
    acc.x += y.x;
    acc.y += y.y;
    acc.z += y.z;
    acc.w += y.w;
  }
  void* const dst = blockIdx.y ? a.dv : a.dk;
  if (a.grad_fp32)
    *reinterpret_cast<float4*>(static_cast<float*>(dst) + out) = acc;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(dst) + out) =
        make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
}

template <int D>
cudaError_t launch_t(const WindowBwdLaunch& l, cudaStream_t stream) {
  using KV = CrossCfg<D, 2 * D>;
  using Q = CrossCfg<D, D>;
  WindowBwdArgs a = l.args;
  auto k1 = window_dkdv_kernel<D>;
  auto k2 = window_dq_kernel<D>;
  auto k3 = window_sum_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, KV::SMEM);
  if (e != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(k2, cudaFuncAttributeMaxDynamicSharedMemorySize, Q::SMEM)) != cudaSuccess) return e;
  const int k_blocks = a.splits0 + ((a.Nk + kTile - 1) / kTile - 1) * a.splits;
  const int q_blocks = ((a.N + kTile - 1) / kTile + a.own_tiles - 1) / a.own_tiles;
  const int q_heads = a.kv_heads * a.group;
  a.ng = head_groups(a.kv_heads, k_blocks, false, l.sms);
  a.ng_q = head_groups(q_heads, q_blocks, false, l.sms);
  e = launch_delta(l.o, l.dout, l.delta, static_cast<long long>(q_heads) * a.N, D, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(a.kv_heads), static_cast<unsigned>(k_blocks));
  cfg.blockDim = dim3(KV::THREADS);
  cfg.dynamicSmemBytes = KV::SMEM;
  if ((e = cudaLaunchKernelEx(&cfg, k1, l.tq, l.tk, l.tv, l.tdo, l.tdk, l.tdv, a)) != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(q_heads), static_cast<unsigned>(q_blocks));
  cfg.blockDim = dim3(Q::THREADS);
  cfg.dynamicSmemBytes = Q::SMEM;
  if ((e = cudaLaunchKernelEx(&cfg, k2, l.tq, l.tk, l.tv, l.tks, l.tvs, l.tdo, l.tdq, a)) != cudaSuccess) return e;
  if (a.splits0 < 2 && a.splits < 2) return cudaSuccess;
  const int first = a.splits0 > 1 ? 0 : kTile, last = a.splits > 1 ? a.Nk : (a.Nk < kTile ? a.Nk : kTile);
  if (last <= first) return cudaSuccess;
  const long long elems = static_cast<long long>(a.kv_heads) * (last - first) * D;
  cfg.gridDim = dim3(static_cast<unsigned>((elems / 4 + 255) / 256), 2);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, k3, a, first, last);
}

}  // namespace

cudaError_t launch_window_bwd(const WindowBwdLaunch& l, cudaStream_t stream) {
  return l.d == 64 ? launch_t<64>(l, stream) : launch_t<128>(l, stream);
}

cudaError_t window_bwd_status_word(unsigned int** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_bwd_status);
}

}  // namespace fattn
