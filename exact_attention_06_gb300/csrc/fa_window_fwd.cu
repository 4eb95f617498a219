// Causal attention with a sliding window and sinks for sm_103a: query i of N stands at position p = Nk - N + i and
// sees the `window` keys up to its own and the first `sinks` keys.
//
// A CTA owns two 128-row query tiles of one query head and runs the schedules of fwd_kernel (fa_fwd.cu) over the keys
// that its rows see.  Those are at most two ranges: the sinks before the window of its first row, one step of at most
// 128 keys, and the keys from that window's first, lo, up to its last row's own.  Tiles are counted from lo, not from
// a multiple of 128, so that a block of 256 rows scans ceil((window + 255) / 128) tiles, and keys before lo
// are never read (whatever they hold has no influence).  The second query tile starts a step later, since
// its windows start 128 keys later, and the first ends a step sooner.
//
// Masks are needed in the steps at both ends of the window only; a thread builds them as four words of bits from
// three comparisons (window.cuh).
//
// The sinks' step reads K and V through tensor maps that end after `sinks` rows: the rows behind them arrive
// as zeros, whatever the cache holds there.
#include "fwd_common.cuh"
#include "window.cuh"

namespace fattn {
namespace {

template <int D>
__global__ void __launch_bounds__(FwdCfg<D>::THREADS, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tks,
                      const __grid_constant__ CUtensorMap tvs, const __grid_constant__ CUtensorMap to,
                      const WindowFwdArgs a) {
  using C = FwdCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sQ = base + C::OFF_Q, sK = base + C::OFF_K, sV = base + C::OFF_V;
  const uint32_t sBar = base + C::OFF_BAR;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_MISC + 4);
#define BAR(i) (sBar + 8u * static_cast<uint32_t>(i))
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned long long budget = a.budget;
  grid_dep_launch();  // a dependent kernel may launch once every CTA has started
  int bh, pair;
  grouped_block(a.ng, bh, pair);
  pair = static_cast<int>(gridDim.y) - 1 - pair;  // the rows with whole windows first
  const int row0 = pair * kRowsPerCta, off = a.Nk - a.N;
  // Steps: the sinks (if any come before lo), then key tiles from lo.  Tile t takes the steps before end(t), but tile 1
  // not the first of lo when that holds nothing it sees.
  const int lo = max(0, off + row0 - a.window + 1), n_sink = min(a.sinks, lo), ws = n_sink > 0 ? 1 : 0;
  auto end_of = [&](int t) {
    const int r = row0 + t * kBr;
    return r < a.N ? ws + (off + min(r + kBr, a.N) - lo + kBc - 1) / kBc : 0;
  };
  const int end0 = end_of(0), end1 = end_of(1), n_max = max(end0, end1);
  const bool skip = end1 > 0 && off + row0 - a.window + 1 >= 0 && lo >= a.sinks;
  // a tile's own steps, counted: step_of(t, i) is its i-th, count(t) of them
  auto step_of = [&](int t, int i) { return i + (t == 1 && skip && i >= ws ? 1 : 0); };
  auto count = [&](int t) { return t == 0 ? end0 : end1 - (skip ? 1 : 0); };
  const int cnt0 = count(0), cnt1 = end1 > 0 ? count(1) : 0;

  if (threadIdx.x == 0) {
    mbar_init(BAR(C::B_Q), 1);
    // With an MMA warp per tile, each K (V) stage is released once by every tile.
    const uint32_t users = C::TWO_ISSUERS ? 1u + (cnt1 > 0 ? 1u : 0u) : 1u;
    for (int s = 0; s < C::KST; ++s) {
      mbar_init(BAR(C::B_KF + s), 1);
      mbar_init(BAR(C::B_KE + s), users);
    }
    for (int s = 0; s < C::VST; ++s) {
      mbar_init(BAR(C::B_VF + s), 1);
      mbar_init(BAR(C::B_VE + s), users);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(BAR(C::B_SF + t), 1);
      mbar_init(BAR(C::B_PF + t), C::SMW * 32);
      mbar_init(BAR(C::B_SC + t), C::SMW * 32);
      mbar_init(BAR(C::B_OF + t), 1);
      mbar_init(BAR(C::B_DRAIN + t), 1);
      mbar_init(BAR(C::B_OW + t), C::SMW * 32);  // O of tile t staged (bf16 O)
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
  auto wait = [&](uint32_t bar, uint32_t parity) { return mbar_wait(bar, parity, abort_flag, budget, &g_fwd_status); };

  if (warp == C::WARP_TMA) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
      const int kh = bh / a.group;  // key head
      int k_issued = 0, v_issued = 0;
      mbar_arrive_expect_tx(BAR(C::B_Q), 2 * C::QB);
      for (int t = 0; t < 2; ++t)
        for (int h = 0; h < C::NH; ++h)
          tma_load_3d(sQ + t * C::QB + h * kBox, &tq, BAR(C::B_Q), h * 64, row0 + t * kBr, bh);
      for (int j = 0; j < n_max; ++j) {
        const int key = j < ws ? 0 : lo + (j - ws) * kBc;
        const int ks = j % C::KST;
        if (j >= C::KST && !wait(BAR(C::B_KE + ks), ((j / C::KST) - 1) & 1)) break;
        mbar_arrive_expect_tx(BAR(C::B_KF + ks), C::KVB);
        for (int h = 0; h < C::NH; ++h)
          tma_load_3d(sK + ks * C::KVB + h * kBox, j < ws ? &tks : &tk, BAR(C::B_KF + ks), h * 64, key, kh);
        k_issued = j + 1;
        const int vs = j % C::VST;
        if (j >= C::VST && !wait(BAR(C::B_VE + vs), ((j / C::VST) - 1) & 1)) break;
        mbar_arrive_expect_tx(BAR(C::B_VF + vs), C::KVB);
        for (int h = 0; h < C::NH; ++h)
          tma_load_3d(sV + vs * C::KVB + h * kBox, j < ws ? &tvs : &tv, BAR(C::B_VF + vs), h * 64, key, kh);
        v_issued = j + 1;
      }
      // Every copy this CTA started must land before its shared memory is released.
      drain_wait(BAR(C::B_Q), 0, budget);
      for (int j = max(0, k_issued - C::KST); j < k_issued; ++j)
        drain_wait(BAR(C::B_KF + j % C::KST), (j / C::KST) & 1, budget);
      for (int j = max(0, v_issued - C::VST); j < v_issued; ++j)
        drain_wait(BAR(C::B_VF + j % C::VST), (j / C::VST) & 1, budget);
    }
  } else if (warp >= C::WARP_MMA) {
    // ------------------------------------------------------------ MMA issuers
    constexpr uint32_t idesc_s = idesc_bf16_f32(kBr, kBc, 0);
    constexpr uint32_t idesc_o = idesc_bf16_f32(kBr, D, 1);
    const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024);
    const uint64_t dk0 = sdesc_sw128(sK, 16, 1024);
    const uint64_t dv0 = sdesc_sw128(sV, kBox, 1024);
    auto issue_s = [&](int t, int j) {
      const uint64_t dq = sdesc_add(dq0, t * C::QB), dk = sdesc_add(dk0, (j % C::KST) * C::KVB);
      const uint32_t d_s = tmem + t * kBc;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {  // 32 bytes of K per MMA
        const uint32_t o32 = static_cast<uint32_t>(kk >> 2) * kBox + static_cast<uint32_t>(kk & 3) * 32u;
        if (kk == 0) mma_ss_c<0>(d_s, sdesc_add(dq, o32), sdesc_add(dk, o32), idesc_s);
        else mma_ss_c<1>(d_s, sdesc_add(dq, o32), sdesc_add(dk, o32), idesc_s);
      }
    };
    auto issue_pv = [&](int t, int j, bool first) {
      const uint64_t dv = sdesc_add(dv0, (j % C::VST) * C::KVB);
      const uint32_t a_p = tmem + (C::SEP ? C::COL_P + 64u * t : static_cast<uint32_t>(t * kBc));
      const uint32_t d_o = tmem + kColO + t * D;
#pragma unroll
      for (int kk = 0; kk < kBc / 16; ++kk) {  // 16 keys per MMA: 8 TMEM columns of P~
        const uint64_t b = sdesc_add(dv, static_cast<uint32_t>(kk) * 2048u);
        if (!first || kk > 0) mma_ts_c<1>(d_o, a_p + 8u * kk, b, idesc_o);
        else mma_ts_c<0>(d_o, a_p + 8u * kk, b, idesc_o);
      }
    };
    if (lane == 0) {
      if constexpr (C::TWO_ISSUERS) {
        const int t = warp - C::WARP_MMA, n = t ? cnt1 : cnt0;
        if (t == 1 && skip) {  // (its first use of both rings: nothing to wait for)
          mbar_arrive(BAR(C::B_KE + ws));
          mbar_arrive(BAR(C::B_VE + ws));
        }
        auto start_s = [&](int j) {
          if (!wait(BAR(C::B_KF + j % C::KST), (j / C::KST) & 1)) return false;
          tc_fence_after();
          issue_s(t, j);
          tc_commit(BAR(C::B_SF + t));
          tc_commit(BAR(C::B_KE + j % C::KST));
          return true;
        };
        bool ok = n > 0 && wait(BAR(C::B_Q), 0) && start_s(step_of(t, 0));
        for (int i = 0; ok && i < n; ++i) {
          if (i + 1 < n && !(wait(BAR(C::B_SC + t), i & 1) && start_s(step_of(t, i + 1)))) break;
          const int j = step_of(t, i);
          ok = wait(BAR(C::B_PF + t), i & 1) && wait(BAR(C::B_VF + j % C::VST), (j / C::VST) & 1);
          if (!ok) break;
          tc_fence_after();
          issue_pv(t, j, i == 0);
          tc_commit(BAR(C::B_OF + t));
          tc_commit(BAR(C::B_VE + j % C::VST));
        }
        if (n > 0) {  // all MMAs complete before TMEM is released
          tc_commit(BAR(C::B_DRAIN + t));
          drain_wait(BAR(C::B_DRAIN + t), 0, budget);
        }
      } else {
        auto has = [&](int t, int j) { return j < (t ? end1 : end0) && !(t == 1 && skip && j == ws); };
        auto nth = [&](int t, int j) { return j - (t == 1 && skip && j > ws ? 1 : 0); };  // step j as the tile counts it
        bool ok = wait(BAR(C::B_Q), 0) && wait(BAR(C::B_KF), 0);
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (has(t, 0)) {
              issue_s(t, 0);
              tc_commit(BAR(C::B_SF + t));
            }
          tc_commit(BAR(C::B_KE));
        }
        for (int j = 1; ok && j <= n_max; ++j) {
          // this iteration's operands first, so that a tile's MMAs issue back to back once its P~ is ready
          ok = wait(BAR(C::B_VF + (j - 1) % C::VST), ((j - 1) / C::VST) & 1) &&
               (j >= n_max || wait(BAR(C::B_KF + j % C::KST), (j / C::KST) & 1));
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const bool pv = has(t, j - 1), s = has(t, j);
            if (!ok || (!pv && !s)) continue;
            if (pv && !wait(BAR(C::B_PF + t), nth(t, j - 1) & 1)) {
              ok = false;
              continue;
            }
            tc_fence_after();
            if (pv) issue_pv(t, j - 1, nth(t, j - 1) == 0);
            if (s) issue_s(t, j);
            // S_t(j) ready and the PV before it done: U_t may be rescaled.  (Not between the sinks and a skipped step.)
            if (s || j == (t ? end1 : end0)) tc_commit(BAR(C::B_SF + t));
          }
          if (!ok) break;
          tc_commit(BAR(C::B_VE + (j - 1) % C::VST));
          if (j < n_max) tc_commit(BAR(C::B_KE + j % C::KST));
        }
        tc_commit(BAR(C::B_DRAIN));  // all MMAs complete before TMEM is released
        drain_wait(BAR(C::B_DRAIN), 0, budget);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax warps
    const int t = warp / C::SMW;
    const int quarter = warp & 3;                       // TMEM lane quarter this warp may access
    const int sub = C::ONE ? 0 : (warp % C::SMW) >> 2;  // which 16 lanes of the quarter (two threads a row)
    const int h = C::ONE ? 0 : lane >> 4;               // which half of the row's columns (two threads a row)
    const int r = C::ONE ? 32 * quarter + lane : 32 * quarter + 16 * sub + (lane & 15);  // TMEM lane = row
    const int row = row0 + t * kBr + r, p = off + row;
    const int n = t ? cnt1 : cnt0;
    const uint32_t lane_addr = static_cast<uint32_t>(C::ONE ? 32 * quarter : 32 * quarter + 16 * sub) << 16;
    const uint32_t t_s = tmem + lane_addr + static_cast<uint32_t>(t * kBc);
    const uint32_t t_o = tmem + lane_addr + kColO + static_cast<uint32_t>(t * D);
    const uint32_t t_p = tmem + lane_addr + C::COL_P + 64u * t;  // separate P~ columns (d = 64)
    const uint64_t c2 = f2_pack(a.sl2, a.sl2);
    float m2 = -INFINITY, l = 0.f;  // l: this thread's part of the row sum (all of it, one thread a row)
    bool ok = n > 0;
    for (int i = 0; ok && i < n; ++i) {
      const int j = step_of(t, i);
      // this step's first key; the sinks' step shows its first n_sink keys to every row
      const bool sink = j < ws;
      const int key0 = (sink ? 0 : lo + (j - ws) * kBc) + 64 * h;
      const int upto = sink ? n_sink - 1 : p, sinks = sink ? kBc : a.sinks;
      ok = wait_all(BAR(C::B_SF + t), i & 1, abort_flag, budget);
      if (!ok) break;
      tc_fence_after();
      uint32_t sr[64], sr2[C::ONE ? 64 : 1];  // one thread a row: columns 0..63 in sr, 64..127 in sr2
      if constexpr (C::ONE) {
        tmem_ld_x64(t_s, sr);
        tmem_ld_x64(t_s + 64, sr2);
      } else {
        tmem_ld2_x64<64>(t_s, sr);  // columns 64h .. 64h+63 of the row
      }
      if constexpr (C::SEP) {
        tc_fence_before();
        mbar_arrive(BAR(C::B_SC + t));  // S_t is in registers: the MMA may overwrite it
      }
      constexpr int kMine = C::ONE ? kBc : kBc / 2;
      if (key0 + kMine - 1 > upto || (key0 <= upto - a.window && key0 + kMine > sinks)) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          hide(sr + 32 * w, visible_keys(key0 + 32 * w, upto, a.window, sinks));
          if constexpr (C::ONE) hide(sr2 + 32 * w, visible_keys(key0 + 64 + 32 * w, upto, a.window, sinks));
        }
      }
      float m_new;
      if constexpr (C::ONE) m_new = row_max_full(sr, sr2, kBc, m2, a.sl2);
      else m_new = row_max_update(sr, 64, m2, a.sl2);
      const float mb = (m_new == -INFINITY) ? 0.f : m_new;  // no key seen yet: alpha = p = 0
      const float alpha = ex2(m2 - mb);
      const uint64_t nmb2 = f2_pack(-mb, -mb);
      uint64_t rs_a = f2_pack(0.f, 0.f), rs_b = rs_a;
      exp_pack_bf16(sr, c2, nmb2, rs_a, rs_b);  // P~ packed in place into sr[0..31]
      if constexpr (C::SEP) {
        // PV_t of the step before must be done before P~_t and U_t are overwritten.
        if (i > 0) {
          ok = wait_all(BAR(C::B_OF + t), (i - 1) & 1, abort_flag, budget);
          if (!ok) break;
          tc_fence_after();
          if (!__all_sync(0xffffffffu, alpha == 1.f)) rescale_half_row<D>(t_o, alpha);
        }
        uint32_t pr[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) pr[k] = sr[k];
        tmem_st2_x32<32>(t_p, pr);
      } else {
        exp_pack_bf16(sr2, c2, nmb2, rs_a, rs_b);
        tmem_st_x32(t_s, *reinterpret_cast<const uint32_t(*)[32]>(sr));        // keys 0..63
        tmem_st_x32(t_s + 32, *reinterpret_cast<const uint32_t(*)[32]>(sr2));  // keys 64..127
      }
      float s0, s1, s2, s3;
      f2_unpack(rs_a, s0, s1);
      f2_unpack(rs_b, s2, s3);
      l = fmaf(alpha, l, (s0 + s1) + (s2 + s3));
      if constexpr (!C::SEP) {
        // (the commit that announced this S covers the PV before it)
        if (i > 0 && !__all_sync(0xffffffffu, alpha == 1.f)) rescale_row128(t_o, alpha);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(BAR(C::B_PF + t));
      m2 = m_new;
    }
    if (ok) {  // U_t final
      if constexpr (C::SEP) ok = wait_all(BAR(C::B_OF + t), (n - 1) & 1, abort_flag, budget);
      else ok = wait_all(BAR(C::B_SF + t), n & 1, abort_flag, budget);
    }
    if (ok) {
      tc_fence_after();
      const float l_row = C::ONE ? l : l + __shfl_xor_sync(0xffffffffu, l, 16);
      const size_t at = static_cast<size_t>(bh) * a.N + row;
      if (!a.o_fp32) {
        // bf16 O through shared memory, in Q_t's place (its S MMAs are complete), and one TMA store per tile
        const uint32_t box0 = sQ + static_cast<uint32_t>(t) * C::QB, box1 = box0 + kBox;
        store_lse(a.lse, at, h, row < a.N, l_row, m2);
        const float o_mul = (l_row > 0.f) ? 1.f / l_row : 0.f;
        if constexpr (C::ONE) stage_full_row_bf16(box0, box1, r, t_o, o_mul);
        else stage_half_row_bf16<D>(box0, box1, r, h, t_o, o_mul);
        mbar_arrive(BAR(C::B_OW + t));
        if ((warp % C::SMW) == 0 && lane == 0 && wait(BAR(C::B_OW + t), 0)) {
          for (int hb = 0; hb < C::NH; ++hb) tma_store_3d(&to, hb ? box1 : box0, hb * 64, row0 + t * kBr, bh);
          bulk_commit();
          bulk_wait_all();  // complete before the CTA exits
        }
      } else {
        if constexpr (C::ONE) store_full_row(a.o, a.lse, at, row < a.N, true, t_o, l_row, m2, 1.f);
        else store_half_row<D>(a.o, a.lse, at, h, row < a.N, true, t_o, l_row, m2, 1.f);
      }
    }
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

template <int D>
cudaError_t launch_t(const WindowFwdLaunch& l, cudaStream_t stream) {
  using C = FwdCfg<D>;
  auto kern = window_fwd_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  const int n_pairs = (l.args.N + kRowsPerCta - 1) / kRowsPerCta;
  WindowFwdArgs a = l.args;
  a.ng = head_groups(l.BH, n_pairs, false, l.sms);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(l.BH), static_cast<unsigned>(n_pairs));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, l.tq, l.tk, l.tv, l.tks, l.tvs, l.to, a);
}

}  // namespace

cudaError_t launch_window_fwd(const WindowFwdLaunch& l, cudaStream_t stream) {
  return l.d == 64 ? launch_t<64>(l, stream) : launch_t<128>(l, stream);
}

cudaError_t window_fwd_status_word(unsigned int** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_fwd_status);
}

}  // namespace fattn
