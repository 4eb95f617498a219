// Causal attention with a sliding window and sinks for sm_103a: query i of N stands at position p = Nk - N + i and
// sees the `window` keys up to its own and the first `sinks` keys.
//
// One CTA per SM walks a list of items: two 128-row query tiles against the keys that their rows see, by the steps of
// fa_fwd.cu's schedules.  A tile's rows are the query heads that share a key head side by side, 128 / G positions of G
// heads, so that they see few keys more than one position's window (one TMA box of a 4-D map brings them in
// that order); or 128 positions of one head.  The keys are at most two ranges: the sinks before the window of the item's
// first position, one step, and the keys from that window's first, lo, up to its last position's own.  Tiles are counted from
// lo, not from a multiple of 128, and keys before lo are never read (whatever they hold has no influence).  With one
// head the second query tile starts a step later, since its windows start 128 keys later.
//
// Persistent, because an item of a narrow window is short (a window of 256: four steps): TMEM, barriers and the K/V ring
// stay between items, the next item's Q and keys are on their way and its first S is computed under the epilogue of the
// last.
//
// Masks are needed in the steps at both ends of the window only; a thread builds them as words of bits from
// three comparisons (window.cuh).  The sinks' step reads K and V through tensor maps that end after `sinks` rows, so that
// the rows behind them arrive as zeros, whatever the cache holds there; its products take no more than the sinks' groups of
// 16 keys, and its softmax 32 columns where they suffice.
//
// Bound by the tensor cores and the softmax's chains in a long window, by an item's begin and end in a narrow one.  Measured
// (GB300): 32/8 heads x 16381, d = 128, window 4096: 598 us in a short burst (2070 MHz; 1610 TFLOP/s of the visible pairs, 0.85 of
// the library's largest product), 645 in a long run (1935 MHz under the power cap; 0.88 of that product there); 2 x 16/4 x 8192,
// window 1024: 114 us; 4 x 16 x 2048, d = 64, window 256: 26 us (the tiles' keys are 1.5 times the window's); 4 x 16/4 x 517
// behind 1500 keys, window 333: 10.2 us.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "fwd_common.cuh"
#include "window.cuh"

namespace fattn {
namespace {

// The w-th item of the list: two tiles of a.tile positions each from n0 on, of unit u.  Steps: `ws` of the sinks (0 or 1),
// then key tiles from lo.  Tile t takes the steps before end(t), but tile 1 not the first of lo where that holds nothing it
// sees.
struct Item {
  int u, n0, lo, n_sink, ws, end0, end1, n;
  bool skip;
  __device__ __forceinline__ Item(const WindowFwdArgs& a, int w) {
    const int pairs = (a.N + 2 * a.tile - 1) / (2 * a.tile);
    int rank;
    grouped_item(w, a.units, pairs, a.ng, u, rank);
    n0 = (pairs - 1 - rank) * 2 * a.tile;  // the last positions first
    const int off = a.Nk - a.N;
    lo = max(0, off + n0 - a.window + 1);
    n_sink = min(a.sinks, lo);
    ws = n_sink > 0 ? 1 : 0;
    auto end_of = [&](int first) { return first < a.N ? ws + (off + min(first + a.tile, a.N) - lo + kBc - 1) / kBc : 0; };
    end0 = end_of(n0);
    end1 = end_of(n0 + a.tile);
    n = max(end0, end1);
    skip = end1 > 0 && a.tile == kBr && off + n0 - a.window + 1 >= 0 && lo >= a.sinks;
  }
  __device__ __forceinline__ bool has(int t, int j) const { return j < (t ? end1 : end0) && !(t == 1 && skip && j == ws); }
  __device__ __forceinline__ int steps(int t) const { return t ? end1 - (skip ? 1 : 0) : end0; }  // of tile t
  __device__ __forceinline__ int step_of(int t, int i) const { return i + (t == 1 && skip && i >= ws ? 1 : 0); }
  __device__ __forceinline__ int key(int j) const { return j < ws ? 0 : lo + (j - ws) * kBc; }
  // groups of 16 keys in the sinks' step
  __device__ __forceinline__ int k16() const { return (n_sink + 15) / 16; }
};

// S_t = Q_t K^T and U_t (+)= P~_t V for a ring stage of 128 keys, or (SINK) its first 16 * k16.  Whole stages have
// code of their own: an issuing thread that branches between its MMAs leaves the tensor core waiting.
template <int D, bool SINK>
__device__ __forceinline__ void issue_scores(uint32_t d_s, uint64_t dq, uint64_t dk, int k16) {
  const uint32_t idesc = idesc_bf16_f32(kBr, SINK ? 16 * k16 : kBc, 0);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {  // 32 bytes of K per MMA
    const uint32_t o32 = static_cast<uint32_t>(kk >> 2) * kBox + static_cast<uint32_t>(kk & 3) * 32u;
    if (kk == 0) mma_ss_c<0>(d_s, sdesc_add(dq, o32), sdesc_add(dk, o32), idesc);
    else mma_ss_c<1>(d_s, sdesc_add(dq, o32), sdesc_add(dk, o32), idesc);
  }
}
template <int D, bool SINK>
__device__ __forceinline__ void issue_values(uint32_t d_o, uint32_t a_p, uint64_t dv, int k16, bool first) {
  constexpr uint32_t idesc = idesc_bf16_f32(kBr, D, 1);
  if (first) mma_ts_c<0>(d_o, a_p, dv, idesc);  // 16 keys per MMA: 8 TMEM columns of P~
  else mma_ts_c<1>(d_o, a_p, dv, idesc);
  if constexpr (SINK) {
#pragma unroll 1
    for (int kk = 1; kk < k16; ++kk) mma_ts_c<1>(d_o, a_p + 8u * kk, sdesc_add(dv, static_cast<uint32_t>(kk) * 2048u), idesc);
  } else {
#pragma unroll
    for (int kk = 1; kk < kBc / 16; ++kk)
      mma_ts_c<1>(d_o, a_p + 8u * kk, sdesc_add(dv, static_cast<uint32_t>(kk) * 2048u), idesc);
  }
}

// Row r of tile t: its position among the N, and where its output goes.
struct Row {
  int n;
  bool in;
  size_t at;
  __device__ __forceinline__ Row(const Item& I, const WindowFwdArgs& a, int t, int r) {
    const int i = r / a.pack;
    n = I.n0 + t * a.tile + i;
    in = i < a.tile && n < a.N;
    at = (static_cast<size_t>(I.u) * a.pack + (r - i * a.pack)) * a.N + n;
  }
};

// Q's rows behind the packed ones, which no copy writes: zeros.
template <int NH>
__device__ __forceinline__ void clear_unused_rows(uint32_t sQ, uint32_t tile_bytes, int rows) {
  for (int i = threadIdx.x; i < (kBr - rows) * 8; i += blockDim.x)
    for (int b = 0; b < 2 * NH; ++b)
      sts128(sQ + (b / NH) * tile_bytes + (b % NH) * kBox + static_cast<uint32_t>(rows) * 128u + i * 16u, 0, 0, 0, 0);
  fence_proxy_async_smem();
}

// What a row sees of step j: keys key0 .. , up to `upto`, by the window and the first `sinks`; the sinks' step shows its
// n_sink keys to every row.
struct Seen {
  int key0, upto, sinks;
  __device__ __forceinline__ Seen(const Item& I, const WindowFwdArgs& a, int j, int p, int col) {
    const bool sink = j < I.ws;
    key0 = I.key(j) + col;
    upto = sink ? I.n_sink - 1 : p;
    sinks = sink ? kBc : a.sinks;
  }
  __device__ __forceinline__ bool all(int n, int window) const {
    return key0 + n - 1 <= upto && (key0 > upto - window || key0 + n <= sinks);
  }
  __device__ __forceinline__ uint32_t word(int i, int window) const { return visible_keys(key0 + 32 * i, upto, window, sinks); }
};

// The maximum that a row's exponents refer to, from the last one and the row's maximum so far (in log2 units): it moves only
// when it has been passed by more than 8, so that U_t is hardly ever rescaled (with 32 rows a warp, some row's maximum
// moves in most steps).  P~ is then at most 2^8, with the same relative rounding, and sums of it stay in fp32.  Without
// a key seen yet: 0, and p = 0.  Measured, moving it always: 725 instead of 673 us at 32 heads x 16381,
// d = 128, window 4096.
__device__ __forceinline__ float reference_max(float last, float now) {
  if (now == -INFINITY) return 0.f;
  return now > last + 8.f ? now : last;
}

__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
  float a0 = __uint_as_float(s[0]), a1 = __uint_as_float(s[1]);
#pragma unroll
  for (int i = 2; i < 30; i += 4) {
    a0 = fmax3(a0, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
    a1 = fmax3(a1, __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
  }
  return fmax3(fmaxf(a0, a1), __uint_as_float(s[30]), __uint_as_float(s[31]));
}

// ---------------------------------------------------------------------------------------------------------------------
// d = 128: P~ aliases S (fa_fwd.cu's schedule for d = 128), one issuing thread.  Per tile the SF barrier completes once a
// step (S ready, and the PV before it done) and once more at an item's end (U final); the issuer starts the tile's next
// item only after its threads have U in registers (SC), so the barrier is never two phases ahead of them.  O goes
// straight from registers to memory, as far as it has no room of its own: Q's place is the next item's.
// STAGED, for tiles of several heads: two K stages, and in place of the third half of each tile's O on its way to memory.
// Straight to memory a warp's rows are a line each, which keeps the load-store unit busy for 11 of 118 us at 2 x 16/4 x 8192,
// window 1024 (by whole sectors; 15 of 122 by halves of them; put together by shuffles it takes 138).  Where both tiles of an
// item end together, half of the columns go through shared memory: 118 -> 114 us, at window 256 66 -> 59; tiles of one
// head, a step apart: 55 -> 58 (2 x 16 x 8192, window 64).
template <bool STAGED>
struct Cfg128 : FwdCfg<128> {
  static constexpr int KST = STAGED ? 2 : 3;
  static constexpr uint32_t OFF_V = OFF_K + KST * KVB, OFF_O = OFF_V + VST * KVB, OFF_BAR = OFF_O + (STAGED ? 2 * kBox : 0);
  static constexpr int B_Q = 0, B_QE = 2, B_KF = 4, B_KE = B_KF + KST, B_VF = B_KE + KST, B_VE = B_VF + VST, B_SF = B_VE + VST,
                       B_PF = B_SF + 2, B_SC = B_PF + 2, B_OSF = B_SC + 2, B_OW = B_OSF + 2, B_DRAIN = B_OW + 2,
                       NBAR = B_DRAIN + 1;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 8u * NBAR;
  static constexpr uint32_t SMEM = OFF_MISC + 16u + 1024u;
};

template <bool STAGED>
__global__ void __launch_bounds__(Cfg128<STAGED>::THREADS, 1)
    window_fwd128_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tks,
                         const __grid_constant__ CUtensorMap tvs, const __grid_constant__ CUtensorMap to,
                         const WindowFwdArgs a) {
  using C = Cfg128<STAGED>;
  constexpr int D = 128;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sQ = base + C::OFF_Q, sK = base + C::OFF_K, sV = base + C::OFF_V, sBar = base + C::OFF_BAR;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_MISC + 4);
#define BAR(i) (sBar + 8u * static_cast<uint32_t>(i))
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned long long budget = a.budget;
  const int w0 = static_cast<int>(blockIdx.x), w_step = static_cast<int>(gridDim.x);
  grid_dep_launch();  // a dependent kernel may launch once every CTA has started
  clear_unused_rows<C::NH>(sQ, C::QB, a.pack * a.tile);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::KST; ++s) {
      mbar_init(BAR(C::B_KF + s), 1);
      mbar_init(BAR(C::B_KE + s), 1);
    }
    for (int s = 0; s < C::VST; ++s) {
      mbar_init(BAR(C::B_VF + s), 1);
      mbar_init(BAR(C::B_VE + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(BAR(C::B_Q + t), 1);
      mbar_init(BAR(C::B_QE + t), 1);
      mbar_init(BAR(C::B_SF + t), 1);
      mbar_init(BAR(C::B_PF + t), C::SMW * 32);
      mbar_init(BAR(C::B_SC + t), C::SMW * 32);
      mbar_init(BAR(C::B_OSF + t), 1);            // the last item's staged O has been read
      mbar_init(BAR(C::B_OW + t), C::SMW * 32);   // this one's is there
    }
    mbar_init(BAR(C::B_DRAIN), 1);
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
      int k_issued = 0, v_issued = 0, q_issued = 0, kc = 0;  // kc: ring steps of the items before
      bool ok = true;
      for (int w = w0, it = 0; ok && w < a.n_items; w += w_step, ++it) {
        const Item I(a, w);
        const int kh = I.u / a.share;  // key head
        auto load = [&](int j, bool is_v, uint32_t dst, uint32_t bar) {
          const bool sink = j < I.ws;
          mbar_arrive_expect_tx(bar, C::KVB);
          for (int h = 0; h < C::NH; ++h)
            tma_load_3d(dst + h * kBox, is_v ? (sink ? &tvs : &tv) : (sink ? &tks : &tk), bar, h * 64, I.key(j), kh);
        };
        auto load_q = [&] {
          for (int t = 0; t < 2; ++t) {
            // The last item's Q is free once the tile's last S MMA has completed (when both tiles' have, 2 x 16 heads x 8192 at
            // windows of 64 / 256 / 1024: 62.8 / 71.7 / 122.6 instead of 57.9 / 67.0 / 120.4 us).
            if (it > 0 && !wait(BAR(C::B_QE + t), (it - 1) & 1)) return false;
            mbar_arrive_expect_tx(BAR(C::B_Q + t), C::NH * static_cast<uint32_t>(a.pack * a.tile) * 128u);
            for (int h = 0; h < C::NH; ++h)
              tma_load_4d(sQ + t * C::QB + h * kBox, &tq, BAR(C::B_Q + t), h * 64, 0, I.n0 + t * a.tile, I.u);
            ++q_issued;
          }
          return true;
        };
        for (int j = 0; ok && j < I.n; ++j) {
          const int g = kc + j, ks = g % C::KST, vs = g % C::VST;
          ok = g < C::KST || wait(BAR(C::B_KE + ks), ((g / C::KST) - 1) & 1);
          if (!ok) break;
          load(j, false, sK + ks * C::KVB, BAR(C::B_KF + ks));
          k_issued = g + 1;
          if (j == 0) ok = load_q();
          ok = ok && (g < C::VST || wait(BAR(C::B_VE + vs), ((g / C::VST) - 1) & 1));
          if (!ok) break;
          load(j, true, sV + vs * C::KVB, BAR(C::B_VF + vs));
          v_issued = g + 1;
        }
        kc += I.n;
      }
      // Every copy this CTA started must land before its shared memory is released.
      for (int t = 0; t < 2; ++t) {
        const int n = (q_issued + 1 - t) / 2;
        if (n > 0) drain_wait(BAR(C::B_Q + t), (n - 1) & 1, budget);
      }
      for (int g = max(0, k_issued - C::KST); g < k_issued; ++g)
        drain_wait(BAR(C::B_KF + g % C::KST), (g / C::KST) & 1, budget);
      for (int g = max(0, v_issued - C::VST); g < v_issued; ++g)
        drain_wait(BAR(C::B_VF + g % C::VST), (g / C::VST) & 1, budget);
    }
  } else if (warp == C::WARP_MMA) {
    // ------------------------------------------------------------ MMA issuer of both tiles
    if (elect_one()) {
      const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024), dk0 = sdesc_sw128(sK, 16, 1024), dv0 = sdesc_sw128(sV, kBox, 1024);
      int ks = 0, vs = 0, kp = 0, vp = 0;          // the rings' next stages and their phases
      int g0 = 0, g1 = 0, e0 = 0, e1 = 0, it = 0;  // each tile's PVs and finished items so far, items
      auto next_k = [&] {
        if (++ks == C::KST) ks = 0, kp ^= 1;
      };
      auto next_v = [&] {
        if (++vs == C::VST) vs = 0, vp ^= 1;
      };
      bool ok = true;
      for (int w = w0; ok && w < a.n_items; w += w_step, ++it) {
        const Item I(a, w);
        // Iteration j: PV of step j - 1, then S of step j, for one tile and the other, this iteration's operands first, so
        // that a tile's MMAs issue back to back once its P~ is ready.  MID: iterations in which both tiles have both and
        // neither begins or ends; the issuing thread's own work between a P~ and its MMAs is on the steps' chain
        // (measured with one code for all iterations: 915 instead of 771 us at 32 heads x 16381, d = 128, window 4096).
        auto iterate = [&](auto mid, int j) {
          constexpr bool MID = decltype(mid)::value;
          const bool has_k = MID || j < I.n, has_v = MID || j > 0;
          const uint64_t dk = sdesc_add(dk0, ks * C::KVB), dv = sdesc_add(dv0, vs * C::KVB);
          if (has_v && !wait(BAR(C::B_VF + vs), vp)) return false;
          if (has_k && !wait(BAR(C::B_KF + ks), kp)) return false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t d_s = tmem + static_cast<uint32_t>(t * kBc), d_o = tmem + kColO + t * D;
            const uint64_t dq = sdesc_add(dq0, t * C::QB);
            int &g = t ? g1 : g0, &e = t ? e1 : e0;
            if constexpr (MID) {
              if (!wait(BAR(C::B_PF + t), g & 1)) return false;
              tc_fence_after();
              issue_values<D, false>(d_o, d_s, dv, 8, false);
              issue_scores<D, false>(d_s, dq, dk, 8);
              tc_commit(BAR(C::B_SF + t));
              ++g;
            } else {
              const int end = t ? I.end1 : I.end0, begin = I.step_of(t, 0);
              const bool pv = j > 0 && I.has(t, j - 1), sc = I.has(t, j), last = j == end;
              if (!pv && !sc) continue;
              if (pv && !wait(BAR(C::B_PF + t), g & 1)) return false;
              if (sc && j == begin && e > 0 && !wait(BAR(C::B_SC + t), (e - 1) & 1)) return false;  // its last U is out
              if (sc && j == begin && !wait(BAR(C::B_Q + t), it & 1)) return false;
              tc_fence_after();
              if (pv) {
                if (j > I.ws) issue_values<D, false>(d_o, d_s, dv, 8, j - 1 == begin);
                else issue_values<D, true>(d_o, d_s, dv, I.k16(), true);
                ++g;
              }
              if (sc) {
                if (j >= I.ws) issue_scores<D, false>(d_s, dq, dk, 8);
                else issue_scores<D, true>(d_s, dq, dk, I.k16());
              }
              // S_t ready and the PV before it done: U_t may be rescaled (not between the sinks and a skipped step); or
              // U final.
              if (sc || last) tc_commit(BAR(C::B_SF + t));
              if (sc && j + 1 == end) tc_commit(BAR(C::B_QE + t));
              if (last) ++e;
            }
          }
          if (has_v) {
            tc_commit(BAR(C::B_VE + vs));
            next_v();
          }
          if (has_k) {
            tc_commit(BAR(C::B_KE + ks));
            next_k();
          }
          return true;
        };
        const int mid0 = I.ws + 3, mid1 = I.end1 > 0 ? I.end0 - 1 : 0;
        int j = 0;
        for (; ok && j < min(mid0, I.n + 1); ++j) ok = iterate(std::false_type{}, j);
        for (; ok && j < mid1; ++j) ok = iterate(std::true_type{}, j);
        for (; ok && j <= I.n; ++j) ok = iterate(std::false_type{}, j);
        if (ok && I.end1 == 0) {  // no second tile
          ok = wait(BAR(C::B_Q + 1), it & 1);
          mbar_arrive(BAR(C::B_QE + 1));
        }
      }
      tc_commit(BAR(C::B_DRAIN));  // all MMAs complete before TMEM is released
      drain_wait(BAR(C::B_DRAIN), 0, budget);
    }
  } else {
    // ------------------------------------------------------------ softmax warps: one thread a row
    const int t = warp / C::SMW, quarter = warp & 3, r = 32 * quarter + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t t_s = tmem + lane_addr + static_cast<uint32_t>(t * kBc);
    const uint32_t t_o = tmem + lane_addr + kColO + static_cast<uint32_t>(t * D);
    const uint64_t c2 = f2_pack(a.sl2, a.sl2);
    const bool o_issuer = warp % C::SMW == 0 && lane == 0;
    const uint32_t o_stage = base + C::OFF_O + static_cast<uint32_t>(t) * kBox;
    int ph = 0, gi = 0;  // phases of SF so far, O tiles staged
    bool ok = true;
    for (int w = w0; ok && w < a.n_items; w += w_step) {
      const Item I(a, w);
      const int n = I.steps(t), p = a.Nk - a.N + Row(I, a, t, r).n;
      if (n <= 0) continue;  // the tile is past N
      float m2 = -INFINITY, l = 0.f;
      for (int i = 0; i < n; ++i) {
        const int j = I.step_of(t, i);
        const Seen see(I, a, j, p, 0);
        ok = wait_all(BAR(C::B_SF + t), ph & 1, abort_flag, budget);
        if (!ok) break;
        ++ph;
        tc_fence_after();
        float alpha;
        uint64_t rs_a = f2_pack(0.f, 0.f), rs_b = rs_a;
        auto begin = [&](float m_new) {
          const float mb = reference_max(m2, m_new);
          alpha = ex2(m2 - mb);
          m2 = m_new == -INFINITY ? m_new : mb;
          return f2_pack(-mb, -mb);
        };
        if (j < I.ws && I.n_sink <= 32) {
          uint32_t sr[32];
          tmem_ld_x32(t_s, sr);
          hide(sr, see.word(0, a.window));
          const uint64_t nmb2 = begin(fmaxf(m2, max32(sr) * a.sl2));
          exp_pack_bf16(sr, c2, nmb2, rs_a, rs_b);
          tmem_st_x16(t_s, *reinterpret_cast<const uint32_t(*)[16]>(sr));
        } else {
          uint32_t sr[64], sr2[64];
          tmem_ld_x64(t_s, sr);
          tmem_ld_x64(t_s + 64, sr2);
          if (!see.all(kBc, a.window)) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              hide(sr + 32 * q, see.word(q, a.window));
              hide(sr2 + 32 * q, see.word(2 + q, a.window));
            }
          }
          const uint64_t nmb2 = begin(row_max_full(sr, sr2, kBc, m2, a.sl2));
          exp_pack_bf16(sr, c2, nmb2, rs_a, rs_b);  // P~ packed in place into sr[0..31]
          exp_pack_bf16(sr2, c2, nmb2, rs_a, rs_b);
          tmem_st_x32(t_s, *reinterpret_cast<const uint32_t(*)[32]>(sr));        // keys 0..63
          tmem_st_x32(t_s + 32, *reinterpret_cast<const uint32_t(*)[32]>(sr2));  // keys 64..127
        }
        float s0, s1, s2, s3;
        f2_unpack(rs_a, s0, s1);
        f2_unpack(rs_b, s2, s3);
        l = fmaf(alpha, l, (s0 + s1) + (s2 + s3));
        // (the commit that announced this S covers the PV before it)
        if (i > 0 && !__all_sync(0xffffffffu, alpha == 1.f)) rescale_row128(t_o, alpha);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(BAR(C::B_PF + t));
      }
      if (!ok) break;
      ok = wait_all(BAR(C::B_SF + t), ph & 1, abort_flag, budget);  // U_t final
      if (!ok) break;
      ++ph;
      tc_fence_after();
      uint32_t u[2][64];
      tmem_ld_x64(t_o, u[0]);
      tmem_ld_x64(t_o + 64, u[1]);
      tc_fence_before();
      mbar_arrive(BAR(C::B_SC + t));  // U_t is in registers
      const Row row(I, a, t, r);
      const float inv = l > 0.f ? 1.f / l : 0.f;
      if (row.in) a.lse[row.at] = l > 0.f ? (m2 + log2f(l)) * kLn2 : -INFINITY;
      if (a.o_fp32) {
        if (row.in) {
          float* const dst = static_cast<float*>(a.o) + row.at * D;
#pragma unroll
          for (int i = 0; i < D / 4; ++i) {
            const uint32_t* x = &u[i / 16][4 * (i % 16)];
            reinterpret_cast<float4*>(dst)[i] = make_float4(__uint_as_float(x[0]) * inv, __uint_as_float(x[1]) * inv,
                                                            __uint_as_float(x[2]) * inv, __uint_as_float(x[3]) * inv);
          }
        }
        __syncwarp();
        continue;
      }
      auto pieces = [&](int i, uint32_t (&w)[8]) {  // columns 16 i ..
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = pack_bf16(__uint_as_float(u[i / 4][16 * (i % 4) + 2 * e]) * inv,
                           __uint_as_float(u[i / 4][16 * (i % 4) + 2 * e + 1]) * inv);
      };
      if constexpr (STAGED) {
        if (gi > 0) {
          if (o_issuer) {
            bulk_wait_read_all();
            mbar_arrive(BAR(C::B_OSF + t));
          }
          ok = wait_all(BAR(C::B_OSF + t), (gi - 1) & 1, abort_flag, budget);
          if (!ok) break;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[8];
          pieces(i, w);
          const uint32_t at = o_stage + static_cast<uint32_t>(r) * 128u, x = static_cast<uint32_t>(r & 7);
          sts128(at + (((2u * i) ^ x) << 4), w[0], w[1], w[2], w[3]);
          sts128(at + (((2u * i + 1u) ^ x) << 4), w[4], w[5], w[6], w[7]);
        }
        fence_proxy_async_smem();
        mbar_arrive(BAR(C::B_OW + t));
      }
      if (row.in) {
        __nv_bfloat16* const dst = static_cast<__nv_bfloat16*>(a.o) + row.at * D;
        const bool whole = (reinterpret_cast<uintptr_t>(a.o) & 31) == 0;
#pragma unroll
        for (int i = STAGED ? 4 : 0; i < 8; ++i) {
          uint32_t w[8];
          pieces(i, w);
          store_bf16x16(dst + 16 * i, w, whole);
        }
      }
      // (One lane's wait does not end the loop: the next item's waits are the whole warp's, and see that it ran out.)
      if (STAGED && o_issuer && wait(BAR(C::B_OW + t), gi & 1)) {
        tma_store_4d(&to, o_stage, 0, 0, I.n0 + t * a.tile, I.u);
        bulk_commit();
      }
      ++gi;
      __syncwarp();
    }
    if (o_issuer) bulk_wait_all();  // the stores complete before the CTA exits
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

// ---------------------------------------------------------------------------------------------------------------------
// d = 64: P~ in columns of its own, three issuing threads (the S products of both tiles, the PV products of tile 0, those
// of tile 1), two threads a row, as fwd_persist_kernel in fa_fwd.cu.
struct Cfg64 : FwdCfg<64> {
  static constexpr int N_ISSUERS = 3;
  static constexpr int WARP_TMA = kWarpMma + N_ISSUERS, THREADS = (WARP_TMA + 1) * 32;
  static constexpr int B_Q = 0, B_QE = 1, B_KF = 2, B_KE = B_KF + KST, B_VF = B_KE + KST, B_VE = B_VF + VST, B_SF = B_VE + VST,
                       B_PF = B_SF + 2, B_SC = B_PF + 2, B_OF = B_SC + 2, B_DRAIN = B_OF + 2, B_OSF = B_DRAIN + N_ISSUERS,
                       B_OW = B_OSF + 2, NBAR = B_OW + 2;
  static constexpr uint32_t OFF_BAR = OFF_V + VST * KVB;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 8u * NBAR;
  static constexpr uint32_t OFF_O = (OFF_MISC + 16u + 1023u) & ~1023u;
  static constexpr uint32_t SMEM = OFF_O + 2u * kBr * 128u + 1024u;
};
static_assert(Cfg128<true>::SMEM <= 232448 && Cfg128<false>::SMEM <= 232448 && Cfg64::SMEM <= 232448,
              "shared memory of the window kernels exceeds 227 KB");

__global__ void __launch_bounds__(Cfg64::THREADS, 1)
    window_fwd64_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tks,
                        const __grid_constant__ CUtensorMap tvs, const __grid_constant__ CUtensorMap to,
                        const WindowFwdArgs a) {
  using C = Cfg64;
  constexpr int D = 64;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sQ = base + C::OFF_Q, sK = base + C::OFF_K, sV = base + C::OFF_V, sBar = base + C::OFF_BAR;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_MISC + 4);
#define BAR(i) (sBar + 8u * static_cast<uint32_t>(i))
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned long long budget = a.budget;
  const int w0 = static_cast<int>(blockIdx.x), w_step = static_cast<int>(gridDim.x);
  grid_dep_launch();
  clear_unused_rows<C::NH>(sQ, C::QB, a.pack * a.tile);
  if (threadIdx.x == 0) {
    mbar_init(BAR(C::B_Q), 1);
    mbar_init(BAR(C::B_QE), 2);
    // Each K (V) stage is released once per tile; for a step that a tile does not take its issuer releases it unread.
    for (int s = 0; s < C::KST; ++s) {
      mbar_init(BAR(C::B_KF + s), 1);
      mbar_init(BAR(C::B_KE + s), 2);
    }
    for (int s = 0; s < C::VST; ++s) {
      mbar_init(BAR(C::B_VF + s), 1);
      mbar_init(BAR(C::B_VE + s), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(BAR(C::B_SF + t), 1);
      mbar_init(BAR(C::B_PF + t), kSoftmaxWarps * 32);
      mbar_init(BAR(C::B_SC + t), kSoftmaxWarps * 32);
      mbar_init(BAR(C::B_OF + t), 1);
      mbar_init(BAR(C::B_OSF + t), 1);                  // O staging of tile t free again
      mbar_init(BAR(C::B_OW + t), kSoftmaxWarps * 32);  // O staging of tile t written
    }
    for (int i = 0; i < C::N_ISSUERS; ++i) mbar_init(BAR(C::B_DRAIN + i), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  grid_dep_wait();
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
      int k_issued = 0, v_issued = 0, q_issued = 0, kc = 0;
      bool ok = true;
      for (int w = w0, it = 0; ok && w < a.n_items; w += w_step, ++it) {
        const Item I(a, w);
        const int kh = I.u / a.share;
        if (it > 0 && !wait(BAR(C::B_QE), (it - 1) & 1)) break;
        mbar_arrive_expect_tx(BAR(C::B_Q), 2 * static_cast<uint32_t>(a.pack * a.tile) * 128u);
        for (int t = 0; t < 2; ++t) tma_load_4d(sQ + t * C::QB, &tq, BAR(C::B_Q), 0, 0, I.n0 + t * a.tile, I.u);
        q_issued = it + 1;
        for (int j = 0; j < I.n; ++j) {
          const int g = kc + j, ks = g % C::KST, vs = g % C::VST;
          ok = g < C::KST || wait(BAR(C::B_KE + ks), ((g / C::KST) - 1) & 1);
          if (!ok) break;
          mbar_arrive_expect_tx(BAR(C::B_KF + ks), C::KVB);
          tma_load_3d(sK + ks * C::KVB, j < I.ws ? &tks : &tk, BAR(C::B_KF + ks), 0, I.key(j), kh);
          k_issued = g + 1;
          ok = g < C::VST || wait(BAR(C::B_VE + vs), ((g / C::VST) - 1) & 1);
          if (!ok) break;
          mbar_arrive_expect_tx(BAR(C::B_VF + vs), C::KVB);
          tma_load_3d(sV + vs * C::KVB, j < I.ws ? &tvs : &tv, BAR(C::B_VF + vs), 0, I.key(j), kh);
          v_issued = g + 1;
        }
        kc += I.n;
      }
      if (q_issued > 0) drain_wait(BAR(C::B_Q), (q_issued - 1) & 1, budget);
      for (int g = max(0, k_issued - C::KST); g < k_issued; ++g)
        drain_wait(BAR(C::B_KF + g % C::KST), (g / C::KST) & 1, budget);
      for (int g = max(0, v_issued - C::VST); g < v_issued; ++g)
        drain_wait(BAR(C::B_VF + g % C::VST), (g / C::VST) & 1, budget);
    }
  } else if (warp >= kWarpMma && warp < kWarpMma + C::N_ISSUERS) {
    // ------------------------------------------------------------ MMA issuers
    if (elect_one()) {
      const int role = warp - kWarpMma, t_pv = role - 1;
      const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024), dk0 = sdesc_sw128(sK, 16, 1024), dv0 = sdesc_sw128(sV, kBox, 1024);
      int g0 = 0, g1 = 0, kc = 0;  // each tile's steps and the ring's over the items so far
      bool ok = true, issued = false;
      for (int w = w0, it = 0; ok && w < a.n_items; w += w_step, ++it) {
        const Item I(a, w);
        if (role == 0) {
          ok = wait(BAR(C::B_Q), it & 1);
          if (!ok) break;
          if (I.end1 == 0) mbar_arrive(BAR(C::B_QE));
          for (int j = 0; ok && j < I.n; ++j) {
            const int gk = kc + j;
            ok = wait(BAR(C::B_KF + gk % C::KST), (gk / C::KST) & 1);
            for (int t = 0; ok && t < 2; ++t) {
              if (!I.has(t, j)) {
                mbar_arrive(BAR(C::B_KE + gk % C::KST));
                continue;
              }
              int& g = t ? g1 : g0;
              ok = g == 0 || wait(BAR(C::B_SC + t), (g - 1) & 1);  // the tile's last S is in registers
              if (!ok) break;
              tc_fence_after();
              const uint64_t dq = sdesc_add(dq0, t * C::QB), dk = sdesc_add(dk0, (gk % C::KST) * C::KVB);
              if (j >= I.ws) issue_scores<D, false>(tmem + t * kBc, dq, dk, 8);
              else issue_scores<D, true>(tmem + t * kBc, dq, dk, I.k16());
              issued = true;
              ++g;
              tc_commit(BAR(C::B_SF + t));
              tc_commit(BAR(C::B_KE + gk % C::KST));
              if (j + 1 == (t ? I.end1 : I.end0)) tc_commit(BAR(C::B_QE));  // the tile's last S of the item
            }
          }
        } else {
          const int t = t_pv;
          for (int j = 0; ok && j < I.n; ++j) {
            const int gv = kc + j;
            ok = wait(BAR(C::B_VF + gv % C::VST), (gv / C::VST) & 1);
            if (!ok) break;
            if (!I.has(t, j)) {
              mbar_arrive(BAR(C::B_VE + gv % C::VST));
              continue;
            }
            ok = wait(BAR(C::B_PF + t), g0 & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dv = sdesc_add(dv0, (gv % C::VST) * C::KVB);
            const uint32_t d_o = tmem + kColO + t * D, a_p = tmem + C::COL_P + 64u * t;
            if (j >= I.ws) issue_values<D, false>(d_o, a_p, dv, 8, I.step_of(t, 0) == j);
            else issue_values<D, true>(d_o, a_p, dv, I.k16(), true);
            issued = true;
            ++g0;  // (this thread's only tile)
            tc_commit(BAR(C::B_OF + t));
            tc_commit(BAR(C::B_VE + gv % C::VST));
          }
        }
        kc += I.n;
      }
      if (issued) {  // all MMAs complete before TMEM is released
        tc_commit(BAR(C::B_DRAIN + role));
        drain_wait(BAR(C::B_DRAIN + role), 0, budget);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax warps: two threads a row
    const int t = warp / kSoftmaxWarps;
    const int quarter = warp & 3, sub = (warp % kSoftmaxWarps) >> 2, h = lane >> 4;
    const int r = 32 * quarter + 16 * sub + (lane & 15);
    const uint32_t lane_addr = static_cast<uint32_t>(32 * quarter + 16 * sub) << 16;
    const uint32_t t_s = tmem + lane_addr + static_cast<uint32_t>(t * kBc);
    const uint32_t t_o = tmem + lane_addr + kColO + static_cast<uint32_t>(t * D);
    const uint32_t t_p = tmem + lane_addr + C::COL_P + 64u * t;
    const uint64_t c2 = f2_pack(a.sl2, a.sl2);
    const bool o_issuer = (warp % kSoftmaxWarps) == 0 && lane == 0;
    const uint32_t o_stage = base + C::OFF_O + static_cast<uint32_t>(t) * (kBr * 128u);
    int g = 0, gi = 0;  // this tile's steps over the items so far (phases of SF and OF), its O tiles staged (OSF, OW)
    bool ok = true;
    for (int w = w0; ok && w < a.n_items; w += w_step) {
      const Item I(a, w);
      const int n = I.steps(t);
      const Row row(I, a, t, r);
      const int p = a.Nk - a.N + row.n;
      if (n <= 0) continue;  // the tile is past N
      if (o_issuer && !a.o_fp32) {  // the staging is free once the last store has read it (long done by now)
        bulk_wait_read_all();
        mbar_arrive(BAR(C::B_OSF + t));
      }
      float m2 = -INFINITY, l = 0.f;  // l: this thread's half of the row
      for (int i = 0; i < n; ++i, ++g) {
        const int j = I.step_of(t, i);
        ok = wait_all(BAR(C::B_SF + t), g & 1, abort_flag, budget);
        if (!ok) break;
        tc_fence_after();
        float alpha;
        uint64_t rs_a = f2_pack(0.f, 0.f), rs_b = rs_a;
        auto begin = [&](float m_new) {
          const float mb = reference_max(m2, m_new);
          alpha = ex2(m2 - mb);
          m2 = m_new == -INFINITY ? m_new : mb;
          return f2_pack(-mb, -mb);
        };
        // PV_t of the step before must be done before P~_t and U_t are overwritten (at an item's first step: the
        // epilogue waited for it).
        auto turn = [&] {
          if (i == 0) return true;
          if (!wait_all(BAR(C::B_OF + t), (g - 1) & 1, abort_flag, budget)) return false;
          tc_fence_after();
          if (!__all_sync(0xffffffffu, alpha == 1.f)) rescale_half_row<D>(t_o, alpha);
          return true;
        };
        if (j < I.ws && I.n_sink <= 32) {
          const Seen see(I, a, j, p, 0);
          uint32_t sr[16];
          tmem_ld2_x16<16>(t_s, sr);  // columns 16h .. 16h + 15
          tc_fence_before();
          mbar_arrive(BAR(C::B_SC + t));
          const uint32_t seen = see.word(0, a.window) >> (16 * h);
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (!(seen & (1u << k))) sr[k] = 0xff800000u;
          float mx = __uint_as_float(sr[0]);
#pragma unroll
          for (int k = 1; k < 16; ++k) mx = fmaxf(mx, __uint_as_float(sr[k]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const uint64_t nmb2 = begin(fmaxf(m2, mx * a.sl2));
          exp_pack_bf16(sr, c2, nmb2, rs_a, rs_b);
          ok = turn();
          if (!ok) break;
          tmem_st2_x8<8>(t_p, *reinterpret_cast<const uint32_t(*)[8]>(sr));
        } else {
          const Seen see(I, a, j, p, 64 * h);
          uint32_t sr[64];
          tmem_ld2_x64<64>(t_s, sr);  // columns 64h .. 64h + 63 of the row
          tc_fence_before();
          mbar_arrive(BAR(C::B_SC + t));  // S_t is in registers: the MMA may overwrite it
          if (!see.all(64, a.window)) {
            hide(sr, see.word(0, a.window));
            hide(sr + 32, see.word(1, a.window));
          }
          const uint64_t nmb2 = begin(row_max_update(sr, 64, m2, a.sl2));
          exp_pack_bf16(sr, c2, nmb2, rs_a, rs_b);  // P~ packed in place into sr[0..31]
          ok = turn();
          if (!ok) break;
          uint32_t pr[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) pr[k] = sr[k];
          tmem_st2_x32<32>(t_p, pr);
        }
        float s0, s1, s2, s3;
        f2_unpack(rs_a, s0, s1);
        f2_unpack(rs_b, s2, s3);
        l = fmaf(alpha, l, (s0 + s1) + (s2 + s3));
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(BAR(C::B_PF + t));
      }
      if (!ok) break;
      ok = wait_all(BAR(C::B_OF + t), (g - 1) & 1, abort_flag, budget);  // U_t final
      if (!ok) break;
      tc_fence_after();
      const float l_row = l + __shfl_xor_sync(0xffffffffu, l, 16);
      if (a.o_fp32) {
        store_half_row<D>(a.o, a.lse, row.at, h, row.in, true, t_o, l_row, m2, 1.f);
      } else {
        ok = wait_all(BAR(C::B_OSF + t), gi & 1, abort_flag, budget);
        if (!ok) break;
        store_lse(a.lse, row.at, h, row.in, l_row, m2);
        stage_half_row_bf16<D>(o_stage, o_stage, r, h, t_o, (l_row > 0.f) ? 1.f / l_row : 0.f);
        mbar_arrive(BAR(C::B_OW + t));
        // (One lane's wait does not end the loop: the next item's waits are the whole warp's, and see that it ran out.)
        if (o_issuer && wait(BAR(C::B_OW + t), gi & 1)) {
          tma_store_4d(&to, o_stage, 0, 0, I.n0 + t * a.tile, I.u);
          bulk_commit();
        }
        ++gi;
      }
      // The U_t loads above complete (tcgen05.wait::ld) before this thread's first P~-ready arrival of the next item,
      // after which PV_t of that item may overwrite U_t.
    }
    if (o_issuer) bulk_wait_all();  // the stores complete before the CTA exits
  }
#undef BAR
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <typename Kern, typename... Args>
cudaError_t launch_kernel(Kern kern, int grid, int threads, uint32_t smem, cudaStream_t stream, Args... args) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

cudaError_t launch_window_fwd(const WindowFwdLaunch& l, cudaStream_t stream) {
  WindowFwdArgs a = l.args;
  const long long items = static_cast<long long>(a.units) * ((a.N + 2 * a.tile - 1) / (2 * a.tile));
  if (items > INT_MAX) return cudaErrorInvalidValue;
  a.n_items = static_cast<int>(items);
  // Items run in the order of their positions, last first, over all units of a group: a group is as many as have their
  // windows' K and V in half of L2 together.  (Measured with 1 / 2 / 4 / 10 / 32 groups of 32 heads x 16381, window 4096: 918
  // / 934 / 927 / 962 / 991 us of an earlier kernel.)
  const long long window_bytes = (static_cast<long long>(a.window) + kRowsPerCta) * l.d * 4;
  const long long group = std::max<long long>(1, (64ll << 20) / window_bytes) * a.share;
  a.ng = static_cast<int>((a.units + group - 1) / group);
  const int grid = static_cast<int>(std::min<long long>(items, l.sms));
  if (l.d == 64)
    return launch_kernel(window_fwd64_kernel, grid, Cfg64::THREADS, Cfg64::SMEM, stream, l.tq, l.tk, l.tv, l.tks, l.tvs, l.to, a);
  auto launch128 = [&](auto kern, int threads, uint32_t smem) {
    return launch_kernel(kern, grid, threads, smem, stream, l.tq, l.tk, l.tv, l.tks, l.tvs, l.to, a);
  };
  return a.pack > 1 ? launch128(window_fwd128_kernel<true>, Cfg128<true>::THREADS, Cfg128<true>::SMEM)
                    : launch128(window_fwd128_kernel<false>, Cfg128<false>::THREADS, Cfg128<false>::SMEM);
}

cudaError_t window_fwd_status_word(unsigned int** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_fwd_status);
}

}  // namespace fattn
