// Cross attention backward over more than 128 keys for sm_103a: dK, dV (one CTA per key tile and range of query
// tiles) and dQ (one per few query tiles, one after another, and range of key tiles), by the formulas of fa_bwd.cu,
// P recomputed from the forward's lse.
//
// A step -- products, their way through TMEM, exponentials, P and dS back, gradients -- is a chain several times
// as long as its work on the tensor core, so these kernels keep several in flight.  The scanned side is taken
// in halves of 64 rows; a half's S and dP are 64 TMEM columns each (a "pair"), and the columns that the
// accumulators leave of 512 hold two pairs (dK, dV at d = 128) or three.  Each pair has four elementwise warps
// (one thread per row, two chunks of 32 columns).  Three threads issue the MMAs, since one thread's issue keeps only
// about a batch in flight: the products, dV's and dK's (S's, dP's and dQ's in the dQ kernel).  A commit of
// each gradient batch tells the product issuers that its pair's columns may be overwritten.
//
// Ranges.  Few key tiles under many queries (or the reverse) leave SMs idle: the scan is cut into ranges whose fp32
// partial sums a last kernel adds in their order, so the gradients are repeatable.
//
// Padding.  Keys behind the sequence are rows of the dK/dV kernel's tile: their P^T and dS^T are cleared after the
// arithmetic.  In the dQ kernel their dS is cleared, and so are their rows of K in shared memory, since
// 0 times what the padding holds would reach dQ.
#include <cuda_bf16.h>

#include "bwd_halves.cuh"

namespace fattn {
namespace {

// Cross attention, by value: see BwdLaunch.  n_keys: keys of the k, v tensors; tiles: tiles of the
// scanned side per block (blockIdx.z takes tiles z * tiles ..); part_stride: elements from one
// partial sum to the next (0: the gradient itself is written).
struct CrossArgs {
  const int* kv_lens;
  int kv_heads, n_keys, tiles;
  int own_tiles;  // dQ kernel: query tiles per block, one after another
  long long part_stride;
  __device__ __forceinline__ int keys(int bh) const {
    return kv_lens ? min(max(kv_lens[bh / kv_heads], 0), n_keys) : n_keys;
  }
};

// One CTA per key tile and range of query tiles.  P^T and dS^T are packed into their S^T and dP^T.
template <int D>
__global__ void __launch_bounds__(CrossCfg<D, 2 * D>::THREADS, 1)
    cross_dkdv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                        const float* __restrict__ lse, const float* __restrict__ delta, void* __restrict__ dk,
                        void* __restrict__ dv, int N, float sl2, float scale, int grad_fp32, unsigned long long budget,
                        const __grid_constant__ CUtensorMap tdk, const __grid_constant__ CUtensorMap tdv, int ng,
                        const CrossArgs x) {
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
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int bh, kt;
  grouped_block(ng, bh, kt);
  const int row0 = static_cast<int>(blockIdx.z) * x.tiles * kTile;  // this block's query rows
  const int n_h = (min(x.tiles * kTile, N - row0) + kHalf - 1) / kHalf, n_i = (n_h + 1) / 2;
  if (x.part_stride) {
    dk = static_cast<float*>(dk) + blockIdx.z * x.part_stride;
    dv = static_cast<float*>(dv) + blockIdx.z * x.part_stride;
  }
  const int lim = x.keys(bh);
  if (kt * kTile >= lim) {  // padding only
    const size_t k0 = static_cast<size_t>(bh) * x.n_keys + kt * kTile;
    const int rows = min(kTile, x.n_keys - kt * kTile);
    zero_rows<D>(dk, k0, rows, grad_fp32);
    zero_rows<D>(dv, k0, rows, grad_fp32);
    wait_as_last_block();
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(BAR(C::B_OWN), 1);
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(BAR(C::B_FULL + s), 1 + 32);  // TMA bytes + the producer warp's lse/D stores
      mbar_init(BAR(C::B_EMPTY + s), 2);  // dV and dK have read the stage
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
        tma_load_3d(sK + h * kBox, &tk, BAR(C::B_OWN), h * 64, kt * kTile, bh);
        tma_load_3d(sV + h * kBox, &tv, BAR(C::B_OWN), h * 64, kt * kTile, bh);
      }
    }
    int issued = 0;
    for (int i = 0; i < n_i; ++i) {
      const int s = i % C::ST;
      if (i >= C::ST && !bwait_all(BAR(C::B_EMPTY + s), ((i / C::ST) - 1) & 1, abort_flag, budget)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(BAR(C::B_FULL + s), 2 * C::TB);
        const uint32_t st = sRing + s * C::STAGE;
        for (int h = 0; h < C::NH; ++h) {
          tma_load_3d(st + h * kBox, &tq, BAR(C::B_FULL + s), h * 64, row0 + i * kTile, bh);
          tma_load_3d(st + C::TB + h * kBox, &tdo, BAR(C::B_FULL + s), h * 64, row0 + i * kTile, bh);
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
        const int col = 32 * c + lane, r = row0 + i * kTile + col;
        const bool in = r < N;
        vs[4 * (col >> 1) + (col & 1)] = in ? -lse[static_cast<size_t>(bh) * N + r] * kLog2e : -INFINITY;
        vs[4 * (col >> 1) + 2 + (col & 1)] = in ? -delta[static_cast<size_t>(bh) * N + r] : 0.f;
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
    if (lane == 0) {
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
          issue_half_product<D>(d, dK, sdesc_add(dR, st), hh & 1);                 // S^T = K Q^T
          issue_half_product<D>(d + 64, dV, sdesc_add(dR, st + C::TB), hh & 1);     // dP^T = V dO^T
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
    const int g = warp >> 2, r = 32 * (warp & 3) + lane, key = kt * kTile + r;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t tS = lanes + kPair * g, tP = tS + 64;
    const uint64_t c2 = f2_pack(sl2, sl2);
    bool ok = true;
    for (int hh = g; ok && hh < n_h; hh += C::FLIGHT) {
      const int i = hh >> 1, s = i % C::ST;
      ok = bwait_all(BAR(C::B_FULL + s), (i / C::ST) & 1, abort_flag, budget) &&
           bwait_all(BAR(C::B_SF + g), (hh / C::FLIGHT) & 1, abort_flag, budget);
      if (!ok) break;
      tc_fence_after();
      const float4* nv = reinterpret_cast<const float4*>(vec + s * (2 * kTile));
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t sv[32], pv[32];
        tmem_ld_x32(tS + 32 * c, sv);
        tmem_ld_x32(tP + 32 * c, pv);
        uint32_t pp[16], dp[16];
        ew_pairs_dkdv<false>(sv, pv, nv, c2, kHalf * (hh & 1) + 32 * c, 0, 0, pp, dp);
        if (key >= lim) clear_pairs(pp, dp);
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
      const size_t row_off = static_cast<size_t>(bh) * x.n_keys + key;
      if (grad_fp32) {
        if (g == 0) store_grad_row<D>(dv, row_off, key < x.n_keys, lanes + kV, 1.f);
        if (g == 1) store_grad_row<D>(dk, row_off, key < x.n_keys, lanes + kK, scale);
      } else if (g < 2) {  // through shared memory: the V and K tiles have their shape and are no longer read
        const uint32_t tile = g == 0 ? sV : sK;
        stage_row_bf16<D>(tile, tile + kBox, r, lanes + (g == 0 ? kV : kK), g == 0 ? 1.f : scale);
        mbar_arrive(BAR(C::B_OW + g));
        if ((warp & 3) == 0 && lane == 0 && bwait(BAR(C::B_OW + g), 0, abort_flag, budget)) {
          for (int h = 0; h < C::NH; ++h)
            tma_store_3d(g == 0 ? &tdv : &tdk, tile + h * kBox, h * 64, kt * kTile, bh);
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

// One CTA per x.own_tiles query tiles and range of key tiles: it scans the keys for one tile after another, the next
// one's Q, dO and first keys on their way meanwhile.  Halves (and stages) are counted over all its tiles, so that their
// phases go on.  dS is packed into its dP.
template <int D>
__global__ void __launch_bounds__(CrossCfg<D, D>::THREADS, 1)
    cross_dq_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                      const float* __restrict__ lse, const float* __restrict__ delta, void* __restrict__ dq, int N,
                      float sl2, float scale, int grad_fp32, unsigned long long budget,
                      const __grid_constant__ CUtensorMap tdq, int ng, const CrossArgs x) {
  using C = CrossCfg<D, D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sOwn = base + C::OFF_A, sRing = base + C::OFF_RING, sBar = base + C::OFF_BAR;  // own: Q, dO
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int bh, qb;
  grouped_block(ng, bh, qb);
  const int t0 = qb * x.own_tiles, nt = min(x.own_tiles, (N + kTile - 1) / kTile - t0);
  const int key0 = static_cast<int>(blockIdx.z) * x.tiles * kTile;  // this block's keys
  const int n_keys = x.keys(bh);
  const int mine = min(x.tiles * kTile, n_keys - key0);
  if (x.part_stride) dq = static_cast<float*>(dq) + blockIdx.z * x.part_stride;
  // One thread sets the barriers up while the length is on its way, and starts the copies before TMEM is allocated.
  // (Measured 92 -> 89 us at d = 64; the dK/dV kernel, whose blocks are longer, was slower with it.)
  const bool producer = threadIdx.x == C::TMA * 32;
  if (producer) {
    for (int b = 0; b < C::NB; ++b) {
      mbar_init(BAR(C::B_OWN + b), 1);
      mbar_init(BAR(C::B_GF + b), 1);    // the tile's dQ is complete
      mbar_init(BAR(C::B_OW + b), 128);  // and out of TMEM (bf16: in Q's place)
    }
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(BAR(C::B_FULL + s), 1);
      mbar_init(BAR(C::B_EMPTY + s), 1);
      mbar_init(BAR(C::B_KC + s), 32);  // K's last tile cleared behind the sequence
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
  if (mine <= 0) {  // no key in this range
    zero_rows<D>(dq, static_cast<size_t>(bh) * N + t0 * kTile, min(nt * kTile, N - t0 * kTile), grad_fp32);
    wait_as_last_block();
    return;
  }
  const int n_h = (mine + kHalf - 1) / kHalf, n_j = (n_h + 1) / 2;  // per query tile
  const bool k_tail = mine % kTile != 0 && n_keys < x.n_keys;  // rows behind the sequence in K's last tile
  auto load = [&](int jj, int j) {  // K_j, V_j as the block's stage jj
    const int s = jj % C::ST, row = key0 + j * kTile;
    const uint32_t st = sRing + s * C::STAGE;
    mbar_arrive_expect_tx(BAR(C::B_FULL + s), 2 * C::TB);
    for (int h = 0; h < C::NH; ++h) {
      tma_load_3d(st + h * kBox, &tk, BAR(C::B_FULL + s), h * 64, row, bh);
      tma_load_3d(st + C::TB + h * kBox, &tv, BAR(C::B_FULL + s), h * 64, row, bh);
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
  const int first = min(C::ST, n_j);  // stages asked for at once
  if (producer) {
    load_own(0);
    for (int j = 0; j < first; ++j) load(j, j);
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
    int issued = first, owned = min(C::NB, nt);  // stages, tiles
    bool ok = true;
    auto take = [&](int before, int end) {  // stages up to before + end, of which `before` are of earlier tiles
      if (lane == 0)
        for (; ok && issued < before + end; ++issued) {
          const int s = issued % C::ST;
          if (issued >= C::ST) ok = bwait(BAR(C::B_EMPTY + s), ((issued / C::ST) - 1) & 1, abort_flag, budget);
          if (!ok) break;
          load(issued, issued - before);
        }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    };
    // dQ = dS K multiplies the last tile's K rows behind the sequence by dS = 0: clear what the
    // caller's padding holds there (0 times an infinity or NaN).
    auto clear = [&](int t) {
      const int last = t * n_j + n_j - 1, s = last % C::ST;
      ok = ok && bwait_all(BAR(C::B_FULL + s), (last / C::ST) & 1, abort_flag, budget);
      if (!ok) return;
      for (int i = (mine - (n_j - 1) * kTile) * 8 + lane; i < kTile * 8; i += 32)
        for (int h = 0; h < C::NH; ++h) sts128(sRing + s * C::STAGE + h * kBox + i * 16, 0, 0, 0, 0);
      fence_proxy_async_smem();
      mbar_arrive(BAR(C::B_KC + s));
    };
    auto finish = [&](int t) {  // tile t's dQ: stored from Q's place, which is then free, as dO's
      ok = bwait(BAR(C::B_OW + t % C::NB), (t / C::NB) & 1, abort_flag, budget);
      if (!ok || grad_fp32) return;
      for (int h = 0; h < C::NH; ++h)
        tma_store_3d(&tdq, sOwn + t % C::NB * (2 * C::TB) + h * kBox, h * 64, (t0 + t) * kTile, bh);
      bulk_commit();
      bulk_wait_read_all();
    };
    int done = 0;  // tiles finished
    for (int t = 0; ok && t < nt; ++t) {
      take(t * n_j, first);
      if (k_tail && first == n_j) clear(t);
      if (lane == 0 && ok && t > 0) {
        finish(done++);
        if (ok && owned < nt) load_own(owned++);
      }
      take(t * n_j, n_j);
      if (k_tail && first < n_j) clear(t);
    }
    if (lane == 0) {
      // every copy lands before the shared memory is released
      for (int t = max(0, owned - C::NB); t < owned; ++t) bdrain(BAR(C::B_OWN + t % C::NB), (t / C::NB) & 1, budget);
      for (int j = max(0, issued - C::ST); j < issued; ++j) bdrain(BAR(C::B_FULL + j % C::ST), (j / C::ST) & 1, budget);
      while (ok && done < nt) finish(done++);
      bulk_wait_all();  // the stores complete before the CTA exits
    }
  } else if (warp >= C::MMA) {
    // ------------------------------------------------------------ MMA issuers: S, dP, dQ
    if (lane == 0) {
      const int role = warp - C::MMA;
      bool ok = true;
      int hc = 0, jc = 0;  // halves and stages of the tiles before
      if (role < 2) {  // S = Q K^T, dP = dO V^T
        const uint64_t dA = sdesc_add(sdesc_sw128(sOwn, 16, 1024), role == 0 ? 0u : C::OFF_B);
        const uint64_t dR = sdesc_add(sdesc_sw128(sRing, 16, 1024), role == 0 ? 0u : C::TB);
        uint32_t cleared = 0;  // parity of each stage's next clearing
        for (int t = 0; ok && t < nt; ++t, hc += n_h, jc += n_j) {
          ok = bwait(BAR(C::B_OWN + t % C::NB), (t / C::NB) & 1, abort_flag, budget);
          for (int hh = 0; ok && hh < n_h; ++hh) {
            const int H = hc + hh, J = jc + (hh >> 1), g = H % C::FLIGHT, s = J % C::ST;
            // the stage loaded (and cleared behind the sequence), and the pair's last dQ MMAs done with its columns
            ok = bwait(BAR(C::B_FULL + s), (J / C::ST) & 1, abort_flag, budget) &&
                 (!k_tail || (hh >> 1) + 1 < n_j || bwait(BAR(C::B_KC + s), (cleared >> s) & 1, abort_flag, budget)) &&
                 (H < C::FLIGHT || bwait(BAR(C::B_GD + g), ((H / C::FLIGHT) - 1) & 1, abort_flag, budget));
            if (!ok) break;
            tc_fence_after();
            issue_half_product<D>(tmem + kPair * g + 64 * role, sdesc_add(dA, t % C::NB * (2 * C::TB)),
                                  sdesc_add(dR, s * C::STAGE), hh & 1);
            tc_commit(BAR(C::B_SF + g));
          }
          cleared ^= 1u << ((jc + n_j - 1) % C::ST);
        }
      } else {  // dQ += dS K
        const uint64_t dRmn = sdesc_sw128(sRing, kBox, 1024);
        for (int t = 0; ok && t < nt; ++t, hc += n_h, jc += n_j) {
          const int b = t % C::NB;
          if (t >= C::NB) {  // the accumulator's last tile is out
            ok = bwait(BAR(C::B_OW + b), ((t / C::NB) - 1) & 1, abort_flag, budget);
            if (!ok) break;
          }
          for (int hh = 0; ok && hh < n_h; ++hh) {
            const int H = hc + hh, s = (jc + (hh >> 1)) % C::ST, g = H % C::FLIGHT;
            for (int c = 0; ok && c < 2; ++c) {
              ok = bwait(BAR(C::B_PF + 2 * g + c), (H / C::FLIGHT) & 1, abort_flag, budget);
              if (!ok) break;
              tc_fence_after();
              issue_half_chunk<D>(tmem + C::COL_ACC + b * D, tmem + kPair * g + 64, sdesc_add(dRmn, s * C::STAGE),
                                  hh & 1, c, hh > 0 || c > 0);
            }
            if (!ok) break;
            tc_commit(BAR(C::B_GD + g));
            if ((hh & 1) || hh + 1 == n_h) tc_commit(BAR(C::B_EMPTY + s));
          }
          if (ok) tc_commit(BAR(C::B_GF + b));
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
    const uint64_t c2 = f2_pack(sl2, sl2);
    bool ok = true;
    int out = 0;  // tiles whose dQ is out (the first four warps take them out of TMEM)
    auto put_out = [&](int t) {
      const int b = t % C::NB, row = (t0 + t) * kTile + r;
      ok = bwait_all(BAR(C::B_GF + b), (t / C::NB) & 1, abort_flag, budget);
      if (!ok) return;
      tc_fence_after();
      const uint32_t acc = lanes + C::COL_ACC + b * D, place = sOwn + b * (2 * C::TB);
      if (grad_fp32) store_grad_row<D>(dq, static_cast<size_t>(bh) * N + row, row < N, acc, scale);
      else stage_row_bf16<D>(place, place + kBox, r, acc, scale);  // (its Q is no longer read)
      tc_fence_before();
      mbar_arrive(BAR(C::B_OW + b));
    };
    auto row_of = [&](const float* v, int t, float past) {
      const int row = (t0 + t) * kTile + r;
      return row < N ? v[static_cast<size_t>(bh) * N + row] : past;
    };
    float lse_n = row_of(lse, 0, INFINITY), dd_n = row_of(delta, 0, 0.f);  // of tile t + 1, read a tile ahead
    int t = -1, hh = g, i = 0;
    uint64_t nl2 = 0, nd2 = 0;
    for (int tile = 0; ok; hh += C::FLIGHT, ++i) {
      while (hh >= n_h) {
        hh -= n_h;
        ++tile;
      }
      if (g == 0)
        while (ok && out < min(tile, nt)) put_out(out++);
      if (!ok || tile >= nt) break;
      if (tile != t) {
        const bool next = tile == t + 1;
        t = tile;
        const float lse2 = (next ? lse_n : row_of(lse, t, INFINITY)) * kLog2e, dd = next ? dd_n : row_of(delta, t, 0.f);
        nl2 = f2_pack(-lse2, -lse2);
        nd2 = f2_pack(-dd, -dd);
        if (t + 1 < nt) {
          lse_n = row_of(lse, t + 1, INFINITY);
          dd_n = row_of(delta, t + 1, 0.f);
        }
      }
      ok = bwait_all(BAR(C::B_SF + g), i & 1, abort_flag, budget);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t sv[32], pv[32];
        tmem_ld_x32(tS + 32 * c, sv);
        tmem_ld_x32(tP + 32 * c, pv);
        uint32_t dp[16];
        const int k0 = hh * kHalf + 32 * c;
        if (k0 + 32 > mine) ew_pairs_dq<true, true>(sv, pv, c2, nl2, nd2, k0, mine - 1, dp);
        else ew_pairs_dq<false>(sv, pv, c2, nl2, nd2, k0, mine - 1, dp);
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

// out = sum of S partial sums of n elements each, in their order; 4 elements a thread.  blockIdx.y = 1: out2 from
// the S after those.
__global__ void __launch_bounds__(256) cross_sum_kernel(const float* __restrict__ part, void* __restrict__ out,
                                                        void* __restrict__ out2, long long n, int S, int fp32) {
  const long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * 4;
  grid_dep_wait();  // launched programmatically after the kernel that leaves the partial sums
  if (i >= n) return;
  if (blockIdx.y) {
    part += S * n;
    out = out2;
  }
  float4 acc = *reinterpret_cast<const float4*>(part + i);
  for (int s = 1; s < S; ++s) {
    const float4 y = *reinterpret_cast<const float4*>(part + s * n + i);
    acc.x += y.x;
    acc.y += y.y;
    acc.z += y.z;
    acc.w += y.w;
  }
  if (fp32)
    *reinterpret_cast<float4*>(static_cast<float*>(out) + i) = acc;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + i) =
        make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
}

template <int D>
cudaError_t launch_t(const BwdLaunch& a, cudaStream_t stream) {
  using KV = CrossCfg<D, 2 * D>;
  using Q = CrossCfg<D, D>;
  const long long kv_elems = static_cast<long long>(a.BH) * a.Nk * D, q_elems = static_cast<long long>(a.BH) * a.N * D;
  const int k_tiles = (a.Nk + kTile - 1) / kTile;
  const int q_blocks = ((a.N + kTile - 1) / kTile + a.own_tiles - 1) / a.own_tiles;
  const bool kv_part = a.kv_splits > 1, q_part = a.q_splits > 1;
  auto k1 = cross_dkdv_kernel<D>;
  auto k2 = cross_dq_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, KV::SMEM);
  if (e != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(k2, cudaFuncAttributeMaxDynamicSharedMemorySize, Q::SMEM)) != cudaSuccess) return e;
  float* dv_part = a.kv_part + a.kv_splits * kv_elems;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto dkdv = [&]() -> cudaError_t {
    cfg.gridDim = dim3(static_cast<unsigned>(a.BH), static_cast<unsigned>(k_tiles), static_cast<unsigned>(a.kv_splits));
    cfg.blockDim = dim3(KV::THREADS);
    cfg.dynamicSmemBytes = KV::SMEM;
    return cudaLaunchKernelEx(
        &cfg, k1, a.tq, a.tk, a.tv, a.tdo, a.lse, static_cast<const float*>(a.delta),
        kv_part ? static_cast<void*>(a.kv_part) : a.dk, kv_part ? static_cast<void*>(dv_part) : a.dv, a.N, a.scale_log2,
        a.scale, static_cast<int>(kv_part || a.grad_fp32), a.budget, a.tdk, a.tdv,
        head_groups(a.BH, k_tiles, false, a.sms),
        CrossArgs{a.kv_lens, a.kv_heads, a.Nk, a.q_tiles, 0, kv_part ? kv_elems : 0});
  };
  auto dq = [&]() -> cudaError_t {
    cfg.gridDim = dim3(static_cast<unsigned>(a.BH), static_cast<unsigned>(q_blocks), static_cast<unsigned>(a.q_splits));
    cfg.blockDim = dim3(Q::THREADS);
    cfg.dynamicSmemBytes = Q::SMEM;
    return cudaLaunchKernelEx(
        &cfg, k2, a.tq, a.tk, a.tv, a.tdo, a.lse, static_cast<const float*>(a.delta),
        q_part ? static_cast<void*>(a.q_part) : a.dq, a.N, a.scale_log2, a.scale,
        static_cast<int>(q_part || a.grad_fp32), a.budget, a.tdq, head_groups(a.BH, q_blocks, false, a.sms),
        CrossArgs{a.kv_lens, a.kv_heads, a.Nk, a.k_tiles, a.own_tiles, q_part ? q_elems : 0});
  };
  e = launch_delta(a.o, a.dout, a.delta, static_cast<long long>(a.BH) * a.N, D, stream);
  if (e != cudaSuccess || (e = dkdv()) != cudaSuccess || (e = dq()) != cudaSuccess) return e;
  if (kv_part && (e = launch_cross_sum(a.kv_part, a.dk, a.dv, kv_elems, a.kv_splits, a.grad_fp32, stream)) != cudaSuccess)
    return e;
  if (q_part) return launch_cross_sum(a.q_part, a.dq, nullptr, q_elems, a.q_splits, a.grad_fp32, stream);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_cross_sum(const float* part, void* out, void* out2, long long n, int S, int fp32,
                             cudaStream_t stream) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((n / 4 + 255) / 256), out2 ? 2 : 1);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cross_sum_kernel, part, out, out2, n, S, fp32);
}

cudaError_t launch_cross_bwd(const BwdLaunch& a, cudaStream_t stream) {
  return a.d == 64 ? launch_t<64>(a, stream) : launch_t<128>(a, stream);
}

cudaError_t cross_bwd_status_word(unsigned int** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_bwd_status);
}

}  // namespace fattn
