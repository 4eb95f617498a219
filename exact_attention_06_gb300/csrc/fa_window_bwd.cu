// Backward of causal attention with a sliding window and sinks (fa_window_fwd.cu) for sm_103a: dK, dV (a CTA takes a few key
// tiles one after another) and dQ (a few query tiles), by the formulas of fa_bwd.cu, P recomputed from the forward's lse.  The
// scanned side is taken in halves of 64 rows, two or three in flight, as in fa_cross_bwd.cu.  Bound by the products whose
// operands both come from shared memory (N = 64) at d = 128, by the halves' chains at d = 64.  Measured (GB300, us, the
// kernels one at a time): 2 x 16/4 x 8192, d = 128, window 1024: D 23, dK/dV 257, dQ 206, sums 5; 4 x 16 x 2048, d = 64,
// window 256: 10, 53, 33, 6.
//
// dK, dV.  The queries that see a key tile are, in every query head that shares the key head, the tile's window, W + 127 of
// them: one list of 128-row stages.  Key tile 0 holds the sinks (at most 128), which every later query sees: those
// queries are a list of their own, as long as many windows, cut into ranges of about a window's length whose fp32 partial
// sums (of the sinks' rows alone) a last kernel adds in their order.  So are the lists of all tiles where there are
// too few of them to fill the SMs.  What the sinks cost (the whole backward, none / 4 / 16): 420 / 454 / 454 and 72.2 / 91 /
// 90.8 us at the sizes above.
//
// dQ.  A query tile scans the sinks before its first row's window (through tensor maps that end behind the sinks), then
// the keys from that window's first, lo, up to its last row's own.
//
// Hidden pairs are cleared after the arithmetic, so that keys which no query sees get a gradient of 0 whatever
// they hold.
#include <cuda_bf16.h>

#include <algorithm>

#include "bwd_halves.cuh"
#include "window.cuh"

namespace fattn {
namespace {

// --------------------------------------------------------------------- D
// D_i = rowsum(O_i * dO_i) = sum_j P_ij dP_ij, for 16 query rows a warp.  The first form reads O as the forward rounded it to
// bf16, and its error, 2^-9 |O_i| |dO_i|, goes into every dS_ij = P_ij (dP_ij - D_i) of the row.  Where a row sees few keys,
// dP_ij - D_i is small beside it: measured over rows of 2 / 4 / 12 / 64 keys (d = 128, norms of dQ's error
// over dQ) 0.0038 / 0.0030 / 0.0026 / 0.0024, of which rounding dQ itself is 0.0017; in the second form 0.0024 throughout.  So
// rows of at most kFewKeys keys (all of a narrow window's, the first of any sequence) take the second form, with warp-level
// products of their 16 rows and the keys that they see, bound by their loads' latency.  (Rows of up to 32 / 48 / 64 keys:
// dQ's error 0.00250 / 0.00246 / 0.00237 at most; us of backward: 64 x 8 x 128, d = 128, window 64 47 / 49 / 58, 4 x 16 x 2048,
// d = 64, window 256 90 / 91 / 92; 2 x 16 x 8192, d = 128, window 64, whose rows are all the second form's with 64 only: 180
// instead of 228.)  The first form is
// bound by memory, and a kernel of its own, whose few registers leave room for the warps that keep loads in flight (one kernel
// of both: 25 instead of 20 us for 262144 rows at d = 128, 6.7 TB/s).
//
// D goes with the rows' lse into one array, for each pair of rows {-lse2, -lse2, -D, -D} (lse2 = lse * log2(e)), so that the
// dK/dV kernel has those of a stage by one bulk copy; a head's rows are row_stride(N) apart, those from N on
// {-inf, 0}: their P is 0.
__host__ __device__ constexpr int row_stride(int N) { return (N + kTile) & ~1; }
constexpr int kFewKeys = 48;
constexpr int kDeltaThreads = 128;

// Leading groups of 16 rows whose first row, which sees the fewest keys, sees at most kFewKeys.
inline int few_groups(const WindowBwdArgs& a) {
  const int groups = (a.N + 15) / 16;
  auto few = [&](int i) {
    const long long seen = static_cast<long long>(a.Nk) - a.N + 16ll * i + 1;  // with its own
    return std::min<long long>(seen, a.window) + std::min<long long>(a.sinks, std::max(seen - a.window, 0ll)) <= kFewKeys;
  };
  int n = 0, end = groups;  // (the number of keys grows with the row)
  while (n < end) {
    const int mid = (n + end) / 2;
    if (few(mid)) n = mid + 1;
    else end = mid;
  }
  return n;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c (16 rows x 8 keys) = A B^T over D columns.  Which column stands at which place of the product's inner dimension does not
// matter as long as both operands agree: lane t of a row's four takes columns 32 m + 8 t .. + 7 as one 16-byte load.
template <int D>
__device__ __forceinline__ void row_products(float (&c)[4], const uint4 (&lo)[D / 32], const uint4 (&hi)[D / 32],
                                             const __nv_bfloat16* key) {
  uint4 b[D / 32];
#pragma unroll
  for (int m = 0; m < D / 32; ++m) b[m] = *reinterpret_cast<const uint4*>(key + 32 * m);
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = 0.f;
#pragma unroll
  for (int m = 0; m < D / 32; ++m) {
    mma16816(c, lo[m].x, hi[m].x, lo[m].y, hi[m].y, b[m].x, b[m].y);
    mma16816(c, lo[m].z, hi[m].z, lo[m].w, hi[m].w, b[m].z, b[m].w);
  }
}

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) s = fmaf(bf16hi(x[i]), bf16hi(y[i]), fmaf(bf16lo(x[i]), bf16lo(y[i]), s));
  return s;
}

// Groups of 16 rows from group0 on, per_head of each query head.  `first`: of the backward's kernels, the one that waits for
// those before; another starts once that one has begun, and ends after it.
template <int D, bool FEW>
__global__ void __launch_bounds__(kDeltaThreads)
    window_delta_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                        const __nv_bfloat16* __restrict__ v, const __nv_bfloat16* __restrict__ o,
                        const __nv_bfloat16* __restrict__ dout, const float* __restrict__ lse, float* __restrict__ rows_out,
                        const WindowBwdArgs a, int group0, int per_head, bool first) {
  if (first) grid_dep_wait();
  grid_dep_launch();  // (not before: the next kernel reads q, k, v and dout without waiting for this one)
  const int lane = threadIdx.x & 31, stride = row_stride(a.N);
  if (!first) wait_as_last_block();
  const long long unit = static_cast<long long>(blockIdx.x) * (kDeltaThreads / 32) + (threadIdx.x >> 5);
  const long long bh = unit / per_head;
  if (bh >= static_cast<long long>(a.kv_heads) * a.group) return;
  const int n0 = (group0 + static_cast<int>(unit - bh * per_head)) * 16, rows = min(16, a.N - n0), p0 = a.Nk - a.N + n0;
  const size_t row0 = static_cast<size_t>(bh) * a.N + n0;
  float* const out = rows_out + static_cast<size_t>(bh) * stride * 2;
  const float lse_row = lane < rows ? lse[row0 + lane] : INFINITY;
  auto put_lse = [&] {  // (last: nothing else waits for lse)
    const int r = n0 + lane;
    if (lane >= 16 || r >= stride) return;
    float* const to = out + (r >> 1) * 4 + (r & 1);
    to[0] = -lse_row * kLog2e;
    if (lane >= rows) to[2] = 0.f;
  };
  if (rows <= 0) return put_lse();
  auto put = [&](int r, float d) { out[(n0 + r >> 1) * 4 + 2 + (r & 1)] = -d; };  // (n0 is even)
  if constexpr (!FEW) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kPasses = 16 / kRows;
    const int r0 = lane / kLanes, col = (lane % kLanes) * 8;
    uint4 x[kPasses], y[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const size_t at = (row0 + min(r0 + i * kRows, rows - 1)) * D + col;
      x[i] = *reinterpret_cast<const uint4*>(o + at);
      y[i] = *reinterpret_cast<const uint4*>(dout + at);
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      float s = dot8(x[i], y[i]);
#pragma unroll
      for (int w = kLanes / 2; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      if (col == 0 && r0 + i * kRows < rows) put(r0 + i * kRows, s);
    }
    put_lse();
  } else {
    const int g = lane >> 2, t = lane & 3;  // rows g, g + 8 and (of 8 keys) key g; columns 8 t .., keys 2 t, 2 t + 1
    const size_t r_lo = (row0 + min(g, rows - 1)) * D + 8 * t, r_hi = (row0 + min(g + 8, rows - 1)) * D + 8 * t;
    uint4 q_lo[D / 32], q_hi[D / 32], d_lo[D / 32], d_hi[D / 32];
#pragma unroll
    for (int m = 0; m < D / 32; ++m) {
      q_lo[m] = *reinterpret_cast<const uint4*>(q + r_lo + 32 * m);
      q_hi[m] = *reinterpret_cast<const uint4*>(q + r_hi + 32 * m);
      d_lo[m] = *reinterpret_cast<const uint4*>(dout + r_lo + 32 * m);
      d_hi[m] = *reinterpret_cast<const uint4*>(dout + r_hi + 32 * m);
    }
    const float l_lo = __shfl_sync(0xffffffffu, lse_row, min(g, rows - 1)) * kLog2e;
    const float l_hi = __shfl_sync(0xffffffffu, lse_row, min(g + 8, rows - 1)) * kLog2e;
    const size_t kv0 = static_cast<size_t>(bh / a.group) * a.Nk;
    const int lo = max(0, p0 - a.window + 1), n_sink = min(a.sinks, lo), last = p0 + rows - 1;
    float s_lo = 0.f, s_hi = 0.f;
    for (int key0 = n_sink > 0 ? 0 : lo; key0 <= last; key0 = key0 < n_sink && key0 + 8 >= n_sink ? lo : key0 + 8) {
      const size_t at = (kv0 + min(key0 + g, a.Nk - 1)) * D + 8 * t;
      float s[4], dp[4];
      row_products<D>(s, q_lo, q_hi, k + at);
      row_products<D>(dp, d_lo, d_hi, v + at);
      // (keys from n_sink on that the last of the sinks' eights holds too count with the window's)
      const uint32_t mine = low_bits(key0 < n_sink ? n_sink - key0 : 32) >> (2 * t);
      const uint32_t see_lo = visible_keys(key0, p0 + g, a.window, a.sinks) >> (2 * t) & mine;
      const uint32_t see_hi = visible_keys(key0, p0 + g + 8, a.window, a.sinks) >> (2 * t) & mine;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (see_lo >> j & 1u) s_lo = fmaf(ex2(fmaf(s[j], a.sl2, -l_lo)), dp[j], s_lo);
        if (see_hi >> j & 1u) s_hi = fmaf(ex2(fmaf(s[2 + j], a.sl2, -l_hi)), dp[2 + j], s_hi);
      }
    }
#pragma unroll
    for (int w = 1; w < 4; w <<= 1) {
      s_lo += __shfl_xor_sync(0xffffffffu, s_lo, w);
      s_hi += __shfl_xor_sync(0xffffffffu, s_hi, w);
    }
    if (t == 0 && g < rows) put(g, s_lo);
    if (t == 0 && g + 8 < rows) put(g + 8, s_hi);
    put_lse();
  }
}

// --------------------------------------------------------------------- dK, dV and dQ
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

// A row of a gradient from TMEM to memory, rounded to bf16; whole sectors where `out` is 32-byte aligned.
template <int D>
__device__ __forceinline__ void store_row_bf16(__nv_bfloat16* out, size_t row, bool valid, uint32_t taddr, float scale) {
  const bool whole = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
#pragma unroll
  for (int q = 0; q < D / 32; ++q) {
    uint32_t u[32];
    tmem_ld_x32(taddr + 32u * q, u);
    if (!valid) continue;
    __nv_bfloat16* const dst = out + row * D + 32 * q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j] = pack_bf16(__uint_as_float(u[16 * i + 2 * j]) * scale, __uint_as_float(u[16 * i + 2 * j + 1]) * scale);
      store_bf16x16(dst + 16 * i, w, whole);
    }
  }
}

// The items of a block: n of the list of all heads' items, from rank `rank` of `head` on.  FLAT (one row of blocks): every `own` of
// the list, over the heads' ends; else `own` of one head, heads and ranks in the order of grouped_block, the last ranks first if
// `reversed`.
struct BlockItems {
  int head, rank, n, per_head;
  __device__ __forceinline__ BlockItems(bool flat, int heads, int per, int own, int ng, bool reversed) : per_head(per) {
    if (flat) {
      const int at = static_cast<int>(blockIdx.x) * own;  // (the host keeps the list within an int)
      head = at / per_head;
      rank = at - head * per_head;
      n = min(own, heads * per_head - at);
    } else {
      grouped_block(ng, head, rank);
      rank = (reversed ? static_cast<int>(gridDim.y) - 1 - rank : rank) * own;
      n = min(own, per_head - rank);
    }
  }
  __device__ __forceinline__ void place(int t, int& h, int& r) const {
    h = head;
    for (r = rank + t; r >= per_head; r -= per_head) ++h;
  }
};

// Layout of the dK/dV kernel: CrossCfg's, with room for two tiles' K and V at d = 64.
template <int D>
struct DkdvCfg : CrossCfg<D, 2 * D> {
  using B = CrossCfg<D, 2 * D>;
  static constexpr int NB = D == 64 ? 2 : 1;
  static constexpr uint32_t OFF_RING = NB * 2 * B::TB;
  static constexpr uint32_t OFF_VEC = OFF_RING + B::ST * B::STAGE, OFF_BAR = OFF_VEC + B::ST * B::VEC;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 8u * B::NBAR;
  static constexpr uint32_t SMEM = OFF_MISC + 16u + 1024u;
  static_assert(SMEM <= 232448, "shared memory");
};

// One item of the dK/dV kernel: a key tile of key head bh, and stages of 128 query rows that see it: of the list of the tile's
// stages, ns of each query head from row `first` on, n_i from the s0-th on.  Per key head:
// the ranges of the queries behind tile 0's window, which see its sinks, then `splits` ranges of every tile's window.
struct KeyItem {
  int bh, kt, first, ns, s0, n_i;
  int slot;  // of the partial sums
  bool sink;
  __device__ __forceinline__ KeyItem(const WindowBwdArgs& a, int head, int rank) : bh(head) {
    sink = rank < a.sink_items;
    kt = sink ? 0 : (rank - a.sink_items) / a.splits;
    slot = sink ? rank : rank - a.sink_items - kt * a.splits;
    const int off = a.Nk - a.N, k0 = kt * kTile;
    first = max(0, k0 - off) & ~1;  // (a stage's rows are pairs of the array of lse and D)
    const int last = min(a.N - 1, k0 + kTile - 1 + a.window - 1 - off);
    ns = last < first ? 0 : (last - first) / kTile + 1;
    int each = a.stages;
    if (sink) {
      first = ns * kTile;  // (off >= 0, so tile 0's window starts at row 0)
      ns = (a.N + kTile - 1) / kTile - ns;
      each = a.sink_stages;
    }
    s0 = slot * each;
    n_i = max(0, min(each, ns * a.group - s0));
  }
  __device__ __forceinline__ bool part(const WindowBwdArgs& a) const { return a.splits > 1 || (kt == 0 && a.sink_items > 0); }
  // Where its dK (dV: which = 1) goes, as fp32 partial sums: row 0, and how many rows.
  __device__ __forceinline__ float* part_at(const WindowBwdArgs& a, int which, int d) const {
    if (sink)
      return a.sink_part + ((static_cast<size_t>(which) * a.sink_items + slot) * a.kv_heads + bh) * a.sink_rows * d;
    if (a.splits == 1) return a.part0 + (static_cast<size_t>(which) * a.kv_heads + bh) * kTile * d;
    return a.part + (((static_cast<size_t>(which) * a.splits + slot) * a.kv_heads + bh) * a.Nk + kt * kTile) * d;
  }
  __device__ __forceinline__ int rows(const WindowBwdArgs& a) const { return sink ? a.sink_rows : min(kTile, a.Nk - kt * kTile); }
};

// One CTA per a.own_items items, one after another, the next one's K, V and first stages on their way meanwhile: into a place of their
// own (d = 64), or into the last one's once its last products with them are complete (d = 128; its gradients then go straight to
// memory, not through K's and V's place).
// Halves and stages are counted over all its items, so that their phases go on.  P^T and dS^T are packed into their
// S^T and dP^T.
template <int D>
__global__ void __launch_bounds__(CrossCfg<D, 2 * D>::THREADS, 1)
    window_dkdv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                       const __grid_constant__ CUtensorMap tdk, const __grid_constant__ CUtensorMap tdv,
                       const WindowBwdArgs a) {
  using C = DkdvCfg<D>;
  constexpr int kOwnRead = C::B_OW + 1;  // (free with one place)
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sRing = base + C::OFF_RING, sBar = base + C::OFF_BAR;  // own tiles: K, V from base on
  float* vec = reinterpret_cast<float*>(gbase + C::OFF_VEC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_MISC + 4);
#define BAR(i) (sBar + 8u * static_cast<uint32_t>(i))
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, N = a.N;
  const unsigned long long budget = a.budget;
  const BlockItems mine(a.flat, a.kv_heads, a.per_head, a.own_items, a.ng, false);  // (the last key tiles have the fewest queries)
  const int nt = mine.n;
  auto item = [&](int t) {
    int head, rank;
    mine.place(t, head, rank);
    return KeyItem(a, head, rank);
  };
  if (threadIdx.x == 0) {
    mbar_init(BAR(C::B_OWN), 1);
    mbar_init(BAR(C::B_OWN + 1), 1);
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(BAR(C::B_FULL + s), 1);
      mbar_init(BAR(C::B_EMPTY + s), 2);      // dV and dK have read the stage
    }
    for (int g = 0; g < C::FLIGHT; ++g) {
      mbar_init(BAR(C::B_SF + g), 1);
      mbar_init(BAR(C::B_GD + g), 2);  // the pair's gradient MMAs are complete
    }
    for (int c = 0; c < 2 * C::FLIGHT; ++c) mbar_init(BAR(C::B_PF + c), 128);
    mbar_init(BAR(C::B_GF), 2);    // an item's gradients are complete
    // and out of TMEM (two places, bf16: in K's and V's).  A barrier for each place, so that it is never two phases ahead of a
    // waiting thread: an item that takes the place again starts with the copies that follow this one's store.
    mbar_init(BAR(C::B_OW), 256);
    mbar_init(BAR(C::B_OW + 1), C::NB > 1 ? 256 : 1);  // (one place: the item's products with K and V are complete)
    for (int i = 0; i < kIssuers; ++i) mbar_init(BAR(C::B_DRAIN + i), 1);
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
    // ------------------------------------------------------------ producer
    if (elect_one()) {
      auto load_own = [&](int t) {
        const KeyItem I = item(t);
        const uint32_t full = BAR(C::B_OWN + t % C::NB), own = base + t % C::NB * (2 * C::TB);
        mbar_arrive_expect_tx(full, 2 * C::TB);
        for (int h = 0; h < C::NH; ++h) {
          tma_load_3d(own + h * kBox, &tk, full, h * 64, I.kt * kTile, I.bh);
          tma_load_3d(own + C::TB + h * kBox, &tv, full, h * 64, I.kt * kTile, I.bh);
        }
      };
      auto finish = [&](int t) {  // item t's gradients: stored from K's and V's place, which is then free
        if (!bwait(BAR(C::B_OW + t % C::NB), (t / C::NB) & 1, abort_flag, budget)) return false;
        const KeyItem I = item(t);
        if (a.grad_fp32 || I.part(a)) return true;
        const uint32_t own = base + t % C::NB * (2 * C::TB);
        for (int h = 0; h < C::NH; ++h) {
          tma_store_3d(&tdk, own + h * kBox, h * 64, I.kt * kTile, I.bh);
          tma_store_3d(&tdv, own + C::TB + h * kBox, h * 64, I.kt * kTile, I.bh);
        }
        bulk_commit();
        bulk_wait_read_all();
        return true;
      };
      int issued = 0, owned = 0, done = 0;  // stages, items, items finished
      bool ok = true;
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tdo);
      for (; owned < min(C::NB, nt); ++owned) load_own(owned);
      // Launched programmatically: D and lse come from the kernel before.  The dQ kernel, which reads them too, may then take
      // SMs as this grid's last round leaves them idle.
      grid_dep_wait();
      grid_dep_launch();
      for (int t = 0; ok && t < nt; ++t) {
        const KeyItem I = item(t);
        int at = 0, head = 0, in_head = 0;  // the next stage: of the item, its query head and place there
        if (I.n_i > 0) {
          head = I.bh * a.group + I.s0 / I.ns;
          in_head = I.s0 % I.ns;
        }
        auto take = [&](int end) {  // the item's stages before `end`
          for (; ok && at < end; ++at, ++issued) {
            const int s = issued % C::ST, row = I.first + in_head * kTile;
            if (issued >= C::ST) ok = bwait(BAR(C::B_EMPTY + s), ((issued / C::ST) - 1) & 1, abort_flag, budget);
            if (!ok) return;
            const uint32_t st = sRing + s * C::STAGE, full = BAR(C::B_FULL + s);
            mbar_arrive_expect_tx(full, 2 * C::TB + C::VEC);
            for (int h = 0; h < C::NH; ++h) {
              tma_load_3d(st + h * kBox, &tq, full, h * 64, row, head);
              tma_load_3d(st + C::TB + h * kBox, &tdo, full, h * 64, row, head);
            }
            bulk_load(base + C::OFF_VEC + s * C::VEC, a.rows + (static_cast<size_t>(head) * a.row_stride + row) * 2, C::VEC, full);
            if (++in_head == I.ns) in_head = 0, ++head;
          }
        };
        take(min(C::ST, I.n_i));
        if (C::NB > 1 && t > 0 && ok) {
          ok = finish(done++);
          if (ok && owned < nt) load_own(owned++);
        }
        take(I.n_i);
        if (C::NB == 1 && ok && owned < nt) {
          ok = bwait(BAR(kOwnRead), t & 1, abort_flag, budget);
          if (ok) load_own(owned++);
        }
      }
      // every copy lands before the shared memory is released
      for (int t = max(0, owned - C::NB); t < owned; ++t) bdrain(BAR(C::B_OWN + t % C::NB), (t / C::NB) & 1, budget);
      for (int i = max(0, issued - C::ST); i < issued; ++i) bdrain(BAR(C::B_FULL + i % C::ST), (i / C::ST) & 1, budget);
      while (C::NB > 1 && ok && done < nt) ok = finish(done++);
      bulk_wait_all();  // the stores complete before the CTA exits
    }
  } else if (warp >= C::MMA) {
    // ------------------------------------------------------------ MMA issuers: the products, dV, dK
    if (elect_one()) {
      const int role = warp - C::MMA;
      bool ok = true;
      int H = 0;  // halves so far
      if (role == 0) {
        const uint64_t dO = sdesc_sw128(base, 16, 1024), dR = sdesc_sw128(sRing, 16, 1024);
        for (int t = 0; ok && t < nt; ++t) {
          const int n_h = 2 * item(t).n_i;
          const uint64_t dK = sdesc_add(dO, t % C::NB * (2 * C::TB)), dV = sdesc_add(dK, C::TB);
          ok = bwait(BAR(C::B_OWN + t % C::NB), (t / C::NB) & 1, abort_flag, budget);
          for (int hh = 0; ok && hh < n_h; ++hh, ++H) {
            const int i = H >> 1, g = H % C::FLIGHT;
            // the stage loaded, and the pair's last gradients done with its columns
            ok = bwait(BAR(C::B_FULL + i % C::ST), (i / C::ST) & 1, abort_flag, budget) &&
                 (H < C::FLIGHT || bwait(BAR(C::B_GD + g), ((H / C::FLIGHT) - 1) & 1, abort_flag, budget));
            if (!ok) break;
            tc_fence_after();
            const uint32_t st = (i % C::ST) * C::STAGE, d = tmem + kPair * g;
            issue_half_product<D>(d, dK, sdesc_add(dR, st), hh & 1);               // S^T = K Q^T
            issue_half_product<D>(d + 64, dV, sdesc_add(dR, st + C::TB), hh & 1);  // dP^T = V dO^T
            tc_commit(BAR(C::B_SF + g));
          }
          if (C::NB == 1 && ok) tc_commit(BAR(kOwnRead));
        }
      } else {
        // dV += P^T dO (role 1), dK += dS^T Q (role 2)
        const uint64_t dY = sdesc_add(sdesc_sw128(sRing, kBox, 1024), role == 1 ? C::TB : 0u);
        const uint32_t acc = tmem + (role == 1 ? kV : kK), x0 = tmem + (role == 1 ? 0u : 64u);
        for (int t = 0; ok && t < nt; ++t) {
          const int n_h = 2 * item(t).n_i;
          if (t > 0) {  // the accumulators' last item is out
            ok = bwait(BAR(C::B_OW + (t - 1) % C::NB), ((t - 1) / C::NB) & 1, abort_flag, budget);
            if (!ok) break;
          }
          for (int hh = 0; ok && hh < n_h; ++hh, ++H) {
            const int g = H % C::FLIGHT, s = (H >> 1) % C::ST;
            const uint64_t dy = sdesc_add(dY, s * C::STAGE);
            for (int c = 0; ok && c < 2; ++c) {
              ok = bwait(BAR(C::B_PF + 2 * g + c), (H / C::FLIGHT) & 1, abort_flag, budget);
              if (!ok) break;
              tc_fence_after();
              issue_half_chunk<D>(acc, x0 + kPair * g, dy, hh & 1, c, hh > 0 || c > 0);
            }
            if (!ok) break;
            tc_commit(BAR(C::B_GD + g));
            if (hh & 1) tc_commit(BAR(C::B_EMPTY + s));
          }
          if (ok) tc_commit(BAR(C::B_GF));
        }
      }
      tc_commit(BAR(C::B_DRAIN + role));
      bdrain(BAR(C::B_DRAIN + role), 0, budget);
    }
  } else {
    // ------------------------------------------------------------ elementwise warps: thread = key row
    const int g = warp >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t tS = lanes + kPair * g, tP = tS + 64;
    const uint64_t c2 = f2_pack(a.sl2, a.sl2);
    bool ok = true;
    int out = 0;  // items whose gradients are out: dV by the first four warps, dK by the next
    auto put_out = [&](int t) {
      const KeyItem I = item(t);
      ok = bwait_all(BAR(C::B_GF), t & 1, abort_flag, budget);
      if (!ok) return;
      tc_fence_after();
      // an item without queries: its copies have landed (nothing else here has waited for them) before zeros take their place
      if (C::NB > 1 && I.n_i == 0) ok = bwait_all(BAR(C::B_OWN + t % C::NB), (t / C::NB) & 1, abort_flag, budget);
      if (!ok) return;
      const uint32_t acc = lanes + (g == 0 ? kV : kK);
      const float scale = g == 0 ? 1.f : a.scale;
      const uint32_t place = base + t % C::NB * (2 * C::TB) + (g == 0 ? C::TB : 0u);
      const bool part = I.part(a), in = r < I.rows(a);
      const size_t row0 = static_cast<size_t>(I.bh) * a.Nk + I.kt * kTile;
      void* const grad = g == 0 ? a.dv : a.dk;
      auto no_query = [&](void* row, int bytes) {  // no query sees the tile
        if (in)
          for (int i = 0; i < bytes / 16; ++i) static_cast<uint4*>(row)[i] = make_uint4(0, 0, 0, 0);
      };
      if (part || a.grad_fp32) {
        float* const dst = part ? I.part_at(a, g == 0 ? 1 : 0, D) : static_cast<float*>(grad) + row0 * D;
        if (I.n_i > 0) store_grad_row<D>(dst, r, in, acc, scale);
        else no_query(dst + static_cast<size_t>(r) * D, D * 4);
      } else if constexpr (C::NB == 1) {
        __nv_bfloat16* const dst = static_cast<__nv_bfloat16*>(grad) + row0 * D;
        if (I.n_i > 0) store_row_bf16<D>(dst, r, in, acc, scale);
        else no_query(dst + static_cast<size_t>(r) * D, D * 2);
      } else if (I.n_i > 0) {  // through shared memory: the V and K tiles have their shape and are no longer read
        stage_row_bf16<D>(place, place + kBox, r, acc, scale);
      } else {
        for (int h = 0; h < C::NH; ++h)
          for (int i = 0; i < 8; ++i) sts128(place + h * kBox + static_cast<uint32_t>(r) * 128u + i * 16u, 0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      __syncwarp();
      tc_fence_before();
      mbar_arrive(BAR(C::B_OW + t % C::NB));
    };
    KeyItem I = item(0);
    int hh = g, H = g, before = 0;  // half of the item, halves, stages of the items before
    int in_head = I.n_i > 0 ? I.s0 % I.ns : 0, at = 0;  // the item's stage `at`: its place among its query head's
    for (int t = 0; ok; hh += C::FLIGHT, H += C::FLIGHT) {
      while (t < nt && hh >= 2 * I.n_i) {
        hh -= 2 * I.n_i;
        before += I.n_i;
        at = 0;
        if (++t < nt) {
          I = item(t);
          in_head = I.n_i > 0 ? I.s0 % I.ns : 0;
        }
      }
      if (g < 2)
        while (ok && out < t) put_out(out++);
      if (!ok || t >= nt) break;
      const int i = hh >> 1, stage = before + i, s = stage % C::ST;
      for (; at < i; ++at)
        if (++in_head == I.ns) in_head = 0;
      // of the half's first query
      const int pos = a.Nk - N + I.first + in_head * kTile + kHalf * (hh & 1), key = I.kt * kTile + r;
      ok = bwait_all(BAR(C::B_FULL + s), (stage / C::ST) & 1, abort_flag, budget) &&
           bwait_all(BAR(C::B_SF + g), (H / C::FLIGHT) & 1, abort_flag, budget);
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

// One CTA per a.own_tiles query tiles, scanned one after another, the next one's Q, dO and first keys
// on their way meanwhile: into places of their own (d = 64), or into the last one's once its last products with them are
// complete (d = 128; dQ then goes straight to memory, not through Q's place; with the dK/dV kernel's items likewise, the
// backward of 2 x 16/4 x 8192, window 1024: 462 -> 453 us, of 2 x 16/2 x 4096, window 256: 138 -> 132).  Halves and
// stages are counted over all its tiles, so that their phases go on.  dS is packed into its dP.
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
  constexpr int kQRead = C::B_OW + 1;  // (free with one place)
  const int per_head = (N + kTile - 1) / kTile;
  const BlockItems mine(a.flat, a.kv_heads * a.group, per_head, a.own_tiles, a.ng_q, true);  // the rows with whole windows first
  const int nt = mine.n;
  const bool producer = threadIdx.x == C::TMA * 32;
  struct Place {
    int bh, row;
  };
  auto place_of = [&](int t) {  // tile t's query head and first row
    int bh, tile;
    mine.place(t, bh, tile);
    return Place{bh, tile * kTile};
  };
  auto keys_of = [&](int t) { return DqTile(a, place_of(t).row); };
  if (producer) {
    for (int b = 0; b < C::NB; ++b) {
      mbar_init(BAR(C::B_OWN + b), 1);
      mbar_init(BAR(C::B_GF + b), 1);    // the tile's dQ is complete
      mbar_init(BAR(C::B_OW + b), 128);  // and out of TMEM (two places, bf16: in Q's)
    }
    if (C::NB == 1) mbar_init(BAR(kQRead), 2);  // the tile's products with Q and dO are complete
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
  auto load = [&](int jj, const DqTile& k, int kh, int j) {  // stage j of a tile, of key head kh, as the block's stage jj
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
    const Place p = place_of(t);
    mbar_arrive_expect_tx(full, 2 * C::TB);
    for (int h = 0; h < C::NH; ++h) {
      tma_load_3d(own + h * kBox, &tq, full, h * 64, p.row, p.bh);
      tma_load_3d(own + C::OFF_B + h * kBox, &tdo, full, h * 64, p.row, p.bh);
    }
  };
  const int first = min(C::ST, keys_of(0).n_j);  // stages asked for at once
  if (producer) {
    const DqTile k = keys_of(0);
    load_own(0);
    for (int j = 0; j < first; ++j) load(j, k, place_of(0).bh / a.group, j);
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
        const Place p = place_of(t);
        for (int h = 0; h < C::NH; ++h)
          tma_store_3d(&tdq, sOwn + t % C::NB * (2 * C::TB) + h * kBox, h * 64, p.row, p.bh);
        bulk_commit();
        bulk_wait_read_all();
      };
      int done = 0;  // tiles finished
      for (int t = 0; ok && t < nt; ++t) {
        const DqTile k = keys_of(t);
        const int kh = place_of(t).bh / a.group;
        auto take = [&](int end) {  // the tile's stages before `end`
          for (; ok && issued < before + end; ++issued) {
            const int s = issued % C::ST;
            if (issued >= C::ST) ok = bwait(BAR(C::B_EMPTY + s), ((issued / C::ST) - 1) & 1, abort_flag, budget);
            if (!ok) return;
            load(issued, k, kh, issued - before);
          }
        };
        take(min(C::ST, k.n_j));
        if (C::NB > 1 && ok && t > 0) {
          finish(done++);
          if (ok && owned < nt) load_own(owned++);
        }
        take(k.n_j);
        if (C::NB == 1 && ok && owned < nt) {
          ok = bwait(BAR(kQRead), t & 1, abort_flag, budget);
          if (ok) load_own(owned++);
        }
        before += k.n_j;
      }
      // every copy lands before the shared memory is released
      for (int t = max(0, owned - C::NB); t < owned; ++t) bdrain(BAR(C::B_OWN + t % C::NB), (t / C::NB) & 1, budget);
      for (int j = max(0, issued - C::ST); j < issued; ++j) bdrain(BAR(C::B_FULL + j % C::ST), (j / C::ST) & 1, budget);
      while (C::NB > 1 && ok && done < nt) finish(done++);
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
          if (C::NB == 1 && ok) tc_commit(BAR(kQRead));
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
      const Place p = place_of(t);
      const int b = t % C::NB, row = p.row + r;
      ok = bwait_all(BAR(C::B_GF + b), (t / C::NB) & 1, abort_flag, budget);
      if (!ok) return;
      tc_fence_after();
      const uint32_t acc = lanes + C::COL_ACC + b * D, place = sOwn + b * (2 * C::TB);
      if (a.grad_fp32) store_grad_row<D>(a.dq, static_cast<size_t>(p.bh) * N + row, row < N, acc, a.scale);
      else if (C::NB > 1) stage_row_bf16<D>(place, place + kBox, r, acc, a.scale);  // (its Q is no longer read)
      else store_row_bf16<D>(static_cast<__nv_bfloat16*>(a.dq), static_cast<size_t>(p.bh) * N + row, row < N, acc, a.scale);
      tc_fence_before();
      mbar_arrive(BAR(C::B_OW + b));
    };
    auto row_of = [&](int t) {  // {-lse2, -D}
      const Place p = place_of(t);
      const int row = p.row + r;  // (within the array: row < N + 127)
      const float* v = a.rows + (static_cast<size_t>(p.bh) * a.row_stride + (row & ~1)) * 2 + (row & 1);
      return make_float2(v[0], v[2]);
    };
    DqTile k = keys_of(0);
    float2 next = row_of(0);  // of tile t + 1, read a tile ahead
    int t = -1, hh = g, i = 0, pos = 0;  // pos: the row's position
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
        const float2 x = tile == t + 1 ? next : row_of(tile);
        t = tile;
        pos = a.Nk - N + place_of(t).row + r;
        nl2 = f2_pack(x.x, x.x);
        nd2 = f2_pack(x.y, x.y);
        if (t + 1 < nt) next = row_of(t + 1);
      }
      ok = bwait_all(BAR(C::B_SF + g), i & 1, abort_flag, budget);
      if (!ok) break;
      tc_fence_after();
      // the half's keys and what the row sees of them; the sinks' halves show their n_sink keys to every row
      const bool sink = hh < k.hs;
      const int key0 = sink ? hh * kHalf : k.lo + (hh - k.hs) * kHalf;
      const int upto = sink ? k.n_sink - 1 : pos, sinks = sink ? kTile : a.sinks;
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

// dK (blockIdx.y = 0) and dV (1) from the partial sums, in their order; 4 elements a thread, the first `rows` rows of each
// key head.
template <int D>
__global__ void __launch_bounds__(256) window_sum_kernel(const WindowBwdArgs a, int rows) {
  const long long e = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * 4;
  const int per_head = rows * D, which = static_cast<int>(blockIdx.y);
  grid_dep_wait();  // launched programmatically after the kernels that leave the partial sums
  const int bh = static_cast<int>(e / per_head);
  if (bh >= a.kv_heads) return;
  const int in_head = static_cast<int>(e - static_cast<long long>(bh) * per_head), row = in_head / D, col = in_head % D;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float* p, size_t stride, int count) {
    for (int s = 0; s < count; ++s) {
      const float4 y = *reinterpret_cast<const float4*>(p + s * stride);
      acc.x += y.x;
      acc.y += y.y;
      acc.z += y.z;
      acc.w += y.w;
    }
  };
  if (a.splits > 1) {
    const size_t stride = static_cast<size_t>(a.kv_heads) * a.Nk * D;
    add(a.part + which * a.splits * stride + (static_cast<size_t>(bh) * a.Nk + row) * D + col, stride, a.splits);
  } else {
    add(a.part0 + (static_cast<size_t>(which) * a.kv_heads + bh) * kTile * D + in_head, 0, 1);
  }
  if (row < a.sink_rows) {
    const size_t stride = static_cast<size_t>(a.kv_heads) * a.sink_rows * D;
    add(a.sink_part + which * a.sink_items * stride + (static_cast<size_t>(bh) * a.sink_rows + row) * D + col, stride,
        a.sink_items);
  }
  const size_t out = (static_cast<size_t>(bh) * a.Nk + row) * D + col;
  void* const dst = which ? a.dv : a.dk;
  if (a.grad_fp32)
    *reinterpret_cast<float4*>(static_cast<float*>(dst) + out) = acc;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(dst) + out) =
        make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
}

template <int D>
cudaError_t launch_t(const WindowBwdLaunch& l, cudaStream_t stream) {
  using KV = DkdvCfg<D>;
  using Q = CrossCfg<D, D>;
  WindowBwdArgs a = l.args;
  a.rows = l.rows;
  a.row_stride = row_stride(a.N);
  // Key heads in groups whose windows' Q and dO lie in half of L2 together.
  const long long span = (static_cast<long long>(a.window) + 2 * kTile) * D * 4 * a.group;
  const long long in_l2 = std::max<long long>(1, (64ll << 20) / span);
  a.ng = static_cast<int>((a.kv_heads + in_l2 - 1) / in_l2);
  const int q_heads = a.kv_heads * a.group, q_blocks = ((a.N + kTile - 1) / kTile + a.own_tiles - 1) / a.own_tiles;
  a.ng_q = head_groups(q_heads, q_blocks, false, l.sms);
  auto k1 = window_dkdv_kernel<D>;
  auto k2 = window_dq_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, KV::SMEM);
  if (e != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(k2, cudaFuncAttributeMaxDynamicSharedMemorySize, Q::SMEM)) != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto grid = [&](long long n, int each, int threads, size_t smem) {
    cfg.gridDim = dim3(static_cast<unsigned>((n + each - 1) / each));  // (y = 1)
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
  };
  using Rows = const __nv_bfloat16*;
  const int groups = (a.row_stride + 15) / 16, few = few_groups(a);
  auto delta = [&](auto kern, int from, int to, bool first) {
    grid(static_cast<long long>(q_heads) * (to - from), kDeltaThreads / 32, kDeltaThreads, 0);
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Rows>(l.q), static_cast<Rows>(l.k), static_cast<Rows>(l.v),
                              static_cast<Rows>(l.o), static_cast<Rows>(l.dout), l.lse, l.rows, a, from, to - from, first);
  };
  // (the rows that pad the array go with either)
  const bool all_few = few == (a.N + 15) / 16;
  if (few > 0 && (e = delta(window_delta_kernel<D, true>, 0, all_few ? groups : few, true)) != cudaSuccess) return e;
  if (!all_few && (e = delta(window_delta_kernel<D, false>, few, groups, few == 0)) != cudaSuccess) return e;
  auto items = [&](int heads, int per_head, int own, int threads, size_t smem) {
    grid(a.flat ? static_cast<long long>(heads) * per_head : own * static_cast<long long>(heads), own, threads, smem);
    if (!a.flat) cfg.gridDim.y = static_cast<unsigned>((per_head + own - 1) / own);
  };
  items(a.kv_heads, a.per_head, a.own_items, KV::THREADS, KV::SMEM);
  if ((e = cudaLaunchKernelEx(&cfg, k1, l.tq, l.tk, l.tv, l.tdo, l.tdk, l.tdv, a)) != cudaSuccess) return e;
  items(q_heads, (a.N + kTile - 1) / kTile, a.own_tiles, Q::THREADS, Q::SMEM);
  if ((e = cudaLaunchKernelEx(&cfg, k2, l.tq, l.tk, l.tv, l.tks, l.tvs, l.tdo, l.tdq, a)) != cudaSuccess) return e;
  if (a.splits < 2 && a.sink_items == 0) return cudaSuccess;
  const int rows = a.splits > 1 || a.Nk < kTile ? a.Nk : kTile;
  grid(static_cast<long long>(a.kv_heads) * rows * D / 4, 256, 256, 0);
  cfg.gridDim.y = 2;
  return cudaLaunchKernelEx(&cfg, window_sum_kernel<D>, a, rows);
}

}  // namespace

cudaError_t launch_window_bwd(const WindowBwdLaunch& l, cudaStream_t stream) {
  return l.d == 64 ? launch_t<64>(l, stream) : launch_t<128>(l, stream);
}

size_t window_bwd_rows_bytes(int heads, int N) { return static_cast<size_t>(heads) * row_stride(N) * 2 * sizeof(float); }

cudaError_t window_bwd_status_word(unsigned int** p) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_bwd_status);
}

}  // namespace fattn
