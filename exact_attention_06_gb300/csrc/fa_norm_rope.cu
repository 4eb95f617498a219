// RMS norm of each head's queries and keys and their rotation (fa_rope.cu) in one pass, and its gradient:
//     r = (mean(x^2) + eps)^(-1/2),   n = x r,   y = R (w n)
//     g = R^T dy,   h = w g,   dx = r (h - n mean(h n)),   dw = sum over rows of g n
// with R the rotation of the row's position and w the weights of q or of k.  One rounding to bf16, of y (dx).
//
// Bound by memory: 4 bytes an element forward, 6 backward.  A thread holds the 16 elements of 8 pairs of a row (2
// 16-byte vectors), the d / 16 threads of a row add their squares up by shuffles, and the row's angles serve several
// heads, as in fa_rope.cu.
//
// dw adds up every row of every head.  A block of the backward kernel takes a few heads of many rows, adds in registers,
// joins its threads through shared memory and leaves one partial sum; a second kernel adds those in a fixed
// order.  No atomics: the gradients are bitwise repeatable.
#include "rope_common.cuh"

namespace fattn {
namespace {

constexpr int kElems = 2 * kPairs;  // elements per thread and row
// Measured (GB300, us): heads whose loads are in flight together, blocks an SM (by registers), heads a thread:
//   forward, 1 x (32 + 8) x 16381, d = 128    4, 5, 4: 74.4   2, 5, 4: 68.1   2, 8, 4: 64.0   2, 8, 16: 57.9   2, 7, 16: 56.7
//   forward and backward, 2 x (16 + 4) x 8192  backward 2, 4, 4: 97.1   4, 3, 4: 91.1   4, 3, 8: 86.7   4, 3, 16: 83.5
// (6.0 TB/s forward; the second with two products an instruction, as here: 82.5, and with the next heads' loads before this
// one's work: 82.7).  Into pages, 4 x (16 + 2 x 16) x 517, d = 64: 4, 5, 4: 8.2   2, 8, 4: 10.3   2, 5, 4: 7.2.
constexpr int kFwdHeads = 2, kFwdBlocks = 7, kPagedBlocks = 1;
constexpr int kBwdHeads = 4, kBwdBlocks = 3, kBwdPerSm = 2 * kBwdBlocks;
constexpr int kMostHeads = 16, kMostPagedHeads = 4;

// Heads a thread takes: as many, and alike.
int heads_per_thread(int heads, int most) {
  const int groups = (heads + most - 1) / most;
  return (heads + groups - 1) / groups;
}

template <int D>
__device__ __forceinline__ void load_weights(const NormRopeLaunch& a, float (*w)[D]) {
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    const void* src = i < D ? a.q_weight : a.k_weight;
    float v = 1.f;
    if (src)
      v = a.weight_fp32 ? static_cast<const float*>(src)[i % D]
                        : __bfloat162float(static_cast<const __nv_bfloat16*>(src)[i % D]);
    w[i / D][i % D] = v;
  }
}

// The sum of x over the threads of the row (TPR of them, side by side).
template <int TPR>
__device__ __forceinline__ float row_sum(float x, unsigned int mask) {
#pragma unroll
  for (int o = TPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
  return x;
}
// The lanes of this thread's row.
template <int TPR>
__device__ __forceinline__ unsigned int row_mask() {
  return ((1u << TPR) - 1u) << (threadIdx.x & 31 & ~(TPR - 1));
}

// A thread's part of a row as 8 pairs (a, b) to turn, two pairs to a 64-bit register each: the products are for two at once.
struct Pairs {
  uint64_t a[kPairs / 2], b[kPairs / 2];
};

// From two 16-byte vectors: the pairs side by side (INTER), or the a's in the first and the b's in the second.
template <bool INTER>
__device__ __forceinline__ Pairs unpack(const uint4& v0, const uint4& v1) {
  const uint32_t x[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  Pairs p;
#pragma unroll
  for (int i = 0; i < kPairs / 2; ++i) {
    const uint32_t u = INTER ? x[2 * i] : x[i], w = INTER ? x[2 * i + 1] : x[i + 4];
    p.a[i] = INTER ? f2_pack(bf16lo(u), bf16lo(w)) : f2_pack(bf16lo(u), bf16hi(u));
    p.b[i] = INTER ? f2_pack(bf16hi(u), bf16hi(w)) : f2_pack(bf16lo(w), bf16hi(w));
  }
  return p;
}
template <bool INTER>
__device__ __forceinline__ void pack(const Pairs& p, uint4& v0, uint4& v1) {
  uint32_t x[8];
#pragma unroll
  for (int i = 0; i < kPairs / 2; ++i) {
    float a0, a1, b0, b1;
    f2_unpack(p.a[i], a0, a1);
    f2_unpack(p.b[i], b0, b1);
    x[INTER ? 2 * i : i] = INTER ? pack_bf16(a0, b0) : pack_bf16(a0, a1);
    x[INTER ? 2 * i + 1 : i + 4] = INTER ? pack_bf16(a1, b1) : pack_bf16(b0, b1);
  }
  v0 = make_uint4(x[0], x[1], x[2], x[3]);
  v1 = make_uint4(x[4], x[5], x[6], x[7]);
}

// The cos, sin and -sin of the thread's pairs.
struct Turn {
  uint64_t c[kPairs / 2], s[kPairs / 2], ns[kPairs / 2];
  __device__ __forceinline__ Turn(const unsigned long long* turns, const unsigned char* axis, int t,
                                  const int (&p)[FA_ROPE_MAX_AXES], float sign) {
    float cf[kPairs], sf[kPairs];
    angles(turns, axis, t, p, sign, cf, sf);
#pragma unroll
    for (int i = 0; i < kPairs / 2; ++i) {
      c[i] = f2_pack(cf[2 * i], cf[2 * i + 1]);
      s[i] = f2_pack(sf[2 * i], sf[2 * i + 1]);
      ns[i] = f2_pack(-sf[2 * i], -sf[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void operator()(Pairs& p) const {
#pragma unroll
    for (int i = 0; i < kPairs / 2; ++i) {
      const uint64_t a = p.a[i], b = p.b[i];
      p.a[i] = f2_fma(a, c[i], f2_mul(b, ns[i]));
      p.b[i] = f2_fma(a, s[i], f2_mul(b, c[i]));
    }
  }
};

__device__ __forceinline__ float sum_of(uint64_t x) {
  float lo, hi;
  f2_unpack(x, lo, hi);
  return lo + hi;
}

// The thread's 16 weights (w: a row of D in shared memory).
template <bool INTER>
__device__ __forceinline__ Pairs weights_of(const float* w, int e0, int e1) {
  Pairs p;
#pragma unroll
  for (int i = 0; i < kPairs / 2; ++i) {
    const float* const u = w + (INTER ? (i < 2 ? e0 + 4 * i : e1 + 4 * (i - 2)) : e0 + 2 * i);
    p.a[i] = INTER ? f2_pack(u[0], u[2]) : f2_pack(u[0], u[1]);
    p.b[i] = INTER ? f2_pack(u[1], u[3]) : f2_pack(u[e1 - e0], u[e1 - e0 + 1]);
  }
  return p;
}

__device__ __forceinline__ void positions(const RopeLaunch& a, long long rows, long long r, int (&p)[FA_ROPE_MAX_AXES]) {
#pragma unroll
  for (int k = 0; k < FA_ROPE_MAX_AXES; ++k) p[k] = k < a.plan.n_axes ? a.pos[k * rows + r] : 0;
}

// Heads 0 .. Hq - 1 are q's, the next Hk k's; PAGED: k's go to the pools, as do v's, the last Hk, as they are.
template <int D, bool INTER, bool PAGED>
__global__ void __launch_bounds__(kThreads, PAGED ? kPagedBlocks : kFwdBlocks) norm_rope_kernel(const NormRopeLaunch n) {
  using C = RopeCfg<D>;
  const RopeLaunch& a = n.r;
  __shared__ unsigned long long turns[D / 2];
  __shared__ unsigned char axis[D / 2];
  __shared__ __align__(16) float w[2][D];
  grid_dep_launch();
  grid_dep_wait();
  load_weights<D>(n, w);
  load_tables(a.plan, D, turns, axis);
  const int t = threadIdx.x % C::TPR;
  const long long rows = static_cast<long long>(a.B) * a.N;
  const long long r = static_cast<long long>(blockIdx.x) * C::ROWS + threadIdx.x / C::TPR;
  if (r >= rows) return;
  const long long b = r / a.N, tok = r - b * a.N;
  if (PAGED && a.new_lens && tok >= a.new_lens[b]) return;  // a padded token: nothing of it is written
  const unsigned int mask = row_mask<C::TPR>();
  // The token's row in the pools (of head 0), or none.
  bool has_page = false;
  long long page_row = 0;
  if constexpr (PAGED) {
    const long long slot = n.slots[r], page = slot >= 0 ? slot / a.page_size : a.num_pages;
    has_page = page < a.num_pages;
    page_row = page * a.Hk * a.page_size + (slot - page * a.page_size);
  }
  int p[FA_ROPE_MAX_AXES];
  positions(a, rows, r, p);
  const Turn turn(turns, axis, t, p, 1.f);
  const int heads = a.Hq + a.Hk * (PAGED ? 2 : 1);
  const int h0 = static_cast<int>(blockIdx.y) * a.heads, h1 = min(h0 + a.heads, heads);
  const int e0 = first_vec<D, INTER>(t), e1 = e0 + second_vec<D, INTER>();
  for (int h = h0; h < h1; h += kFwdHeads) {
    uint4 x0[kFwdHeads], x1[kFwdHeads];
    __nv_bfloat16* dst[kFwdHeads];
#pragma unroll
    for (int i = 0; i < kFwdHeads; ++i) {
      const int hh = min(h + i, h1 - 1);
      const __nv_bfloat16* src;
      if (hh < a.Hq) {
        const long long off = ((b * a.Hq + hh) * a.N + tok) * D;
        src = a.q + off;
        dst[i] = a.q_out + off;
      } else {
        const bool is_v = PAGED && hh >= a.Hq + a.Hk;
        const int hk = hh - a.Hq - (is_v ? a.Hk : 0);
        const long long off = ((b * a.Hk + hk) * a.N + tok) * D;
        src = (is_v ? a.v : a.k) + off;
        if constexpr (PAGED)
          dst[i] = has_page ? (is_v ? a.v_out : a.k_out) + (page_row + static_cast<long long>(hk) * a.page_size) * D
                            : nullptr;
        else
          dst[i] = a.k_out + off;
      }
      if (h + i >= h1) dst[i] = nullptr;
      if (dst[i]) {
        x0[i] = *reinterpret_cast<const uint4*>(src + e0);
        x1[i] = *reinterpret_cast<const uint4*>(src + e1);
      }
    }
#pragma unroll
    for (int i = 0; i < kFwdHeads; ++i)
      if (dst[i]) {  // (the same for all threads of the row)
        if (!PAGED || h + i < a.Hq + a.Hk) {
          Pairs f = unpack<INTER>(x0[i], x1[i]);
          uint64_t sa = 0, sb = 0;
#pragma unroll
          for (int e = 0; e < kPairs / 2; ++e) {
            sa = f2_fma(f.a[e], f.a[e], sa);
            sb = f2_fma(f.b[e], f.b[e], sb);
          }
          const float rs = rsqrtf(fmaf(row_sum<C::TPR>(sum_of(sa) + sum_of(sb), mask), 1.f / D, n.eps));
          const uint64_t r2 = f2_pack(rs, rs);
          const Pairs wf = weights_of<INTER>(w[h + i < a.Hq ? 0 : 1], e0, e1);
#pragma unroll
          for (int e = 0; e < kPairs / 2; ++e) {
            f.a[e] = f2_mul(f2_mul(f.a[e], r2), wf.a[e]);
            f.b[e] = f2_mul(f2_mul(f.b[e], r2), wf.b[e]);
          }
          turn(f);
          pack<INTER>(f, x0[i], x1[i]);
        }
        *reinterpret_cast<uint4*>(dst[i] + e0) = x0[i];
        *reinterpret_cast<uint4*>(dst[i] + e1) = x1[i];
      }
  }
}

// How the backward kernel's blocks share the work: `gx` blocks along the rows for each group of `heads` heads, of
// which the first yq are q's and the next yk k's.
struct BwdGrid {
  int heads, yq, yk, gx;
};

BwdGrid bwd_grid(int B, int Hq, int Hk, int N, int d, int sms) {
  BwdGrid g;
  const long long groups = (static_cast<long long>(B) * N + kThreads / (d / kElems) - 1) / (kThreads / (d / kElems));
  g.heads = heads_per_thread(Hq > Hk ? Hq : Hk, kMostHeads);
  auto ys = [&] {
    g.yq = (Hq + g.heads - 1) / g.heads;
    g.yk = (Hk + g.heads - 1) / g.heads;
    return g.yq + g.yk;
  };
  while (ys() && g.heads > 1 && groups * ys() < 4LL * sms) g.heads = (g.heads + 1) / 2;
  long long gx = static_cast<long long>(kBwdPerSm) * sms / ys();
  if (gx < 1) gx = 1;
  g.gx = static_cast<int>(gx < groups ? gx : groups);
  return g;
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) norm_rope_bwd_kernel(const NormRopeLaunch n, const BwdGrid g) {
  using C = RopeCfg<D>;
  const RopeLaunch& a = n.r;
  __shared__ unsigned long long turns[D / 2];
  __shared__ unsigned char axis[D / 2];
  __shared__ __align__(16) float w[2][D];
  __shared__ __align__(16) float sum[C::ROWS][D + 4];
  grid_dep_wait();
  load_weights<D>(n, w);
  load_tables(a.plan, D, turns, axis);
  grid_dep_launch();
  const int t = threadIdx.x % C::TPR, y = static_cast<int>(blockIdx.y);
  const bool is_q = y < g.yq;
  const int H = is_q ? a.Hq : a.Hk, h0 = (is_q ? y : y - g.yq) * g.heads, h1 = min(h0 + g.heads, H);
  const __nv_bfloat16* const x = is_q ? a.q : a.k;
  const __nv_bfloat16* const dy = is_q ? n.dq_out : n.dk_out;
  __nv_bfloat16* const dx = is_q ? n.dq : n.dk;
  const unsigned int mask = row_mask<C::TPR>();
  const int e0 = first_vec<D, INTER>(t), e1 = e0 + second_vec<D, INTER>();
  const Pairs wf = weights_of<INTER>(w[is_q ? 0 : 1], e0, e1);
  Pairs acc = {};
  const long long rows = static_cast<long long>(a.B) * a.N;
  for (long long r = static_cast<long long>(blockIdx.x) * C::ROWS + threadIdx.x / C::TPR; r < rows;
       r += static_cast<long long>(g.gx) * C::ROWS) {
    const long long b = r / a.N, tok = r - b * a.N;
    const long long off = (b * H * a.N + tok) * D;
    int p[FA_ROPE_MAX_AXES];
    positions(a, rows, r, p);
    const Turn turn(turns, axis, t, p, -1.f);
    for (int h = h0; h < h1; h += kBwdHeads) {
      uint4 x0[kBwdHeads], x1[kBwdHeads], y0[kBwdHeads], y1[kBwdHeads];
#pragma unroll
      for (int i = 0; i < kBwdHeads; ++i) {
        const long long at = off + static_cast<long long>(min(h + i, h1 - 1)) * a.N * D;
        x0[i] = *reinterpret_cast<const uint4*>(x + at + e0);
        x1[i] = *reinterpret_cast<const uint4*>(x + at + e1);
        y0[i] = *reinterpret_cast<const uint4*>(dy + at + e0);
        y1[i] = *reinterpret_cast<const uint4*>(dy + at + e1);
      }
#pragma unroll
      for (int i = 0; i < kBwdHeads; ++i)
        if (h + i < h1) {
          Pairs f = unpack<INTER>(x0[i], x1[i]), g = unpack<INTER>(y0[i], y1[i]);
          turn(g);
          uint64_t sa = 0, sb = 0, ha = 0, hb = 0;
#pragma unroll
          for (int e = 0; e < kPairs / 2; ++e) {
            sa = f2_fma(f.a[e], f.a[e], sa);
            sb = f2_fma(f.b[e], f.b[e], sb);
            ha = f2_fma(f2_mul(g.a[e], wf.a[e]), f.a[e], ha);
            hb = f2_fma(f2_mul(g.b[e], wf.b[e]), f.b[e], hb);
          }
          const float ss = row_sum<C::TPR>(sum_of(sa) + sum_of(sb), mask);
          const float hx = row_sum<C::TPR>(sum_of(ha) + sum_of(hb), mask);
          const float rs = rsqrtf(fmaf(ss, 1.f / D, n.eps));
          const float m = -hx * rs * (1.f / D);  // -mean(h n)
          const uint64_t r2 = f2_pack(rs, rs), m2 = f2_pack(m, m);
#pragma unroll
          for (int e = 0; e < kPairs / 2; ++e) {
            const uint64_t na = f2_mul(f.a[e], r2), nb = f2_mul(f.b[e], r2);
            acc.a[e] = f2_fma(g.a[e], na, acc.a[e]);
            acc.b[e] = f2_fma(g.b[e], nb, acc.b[e]);
            f.a[e] = f2_mul(r2, f2_fma(g.a[e], wf.a[e], f2_mul(na, m2)));
            f.b[e] = f2_mul(r2, f2_fma(g.b[e], wf.b[e], f2_mul(nb, m2)));
          }
          pack<INTER>(f, x0[i], x1[i]);
          __nv_bfloat16* const to = dx + off + static_cast<long long>(h + i) * a.N * D;
          *reinterpret_cast<uint4*>(to + e0) = x0[i];
          *reinterpret_cast<uint4*>(to + e1) = x1[i];
        }
    }
  }
  if (!n.part) return;
  float* const mine = sum[threadIdx.x / C::TPR];
#pragma unroll
  for (int i = 0; i < kPairs / 2; ++i) {
    float* const u = mine + (INTER ? (i < 2 ? e0 + 4 * i : e1 + 4 * (i - 2)) : e0 + 2 * i);
    f2_unpack(acc.a[i], u[0], u[INTER ? 2 : 1]);
    f2_unpack(acc.b[i], u[INTER ? 1 : e1 - e0], u[INTER ? 3 : e1 - e0 + 1]);
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < C::ROWS; ++i) v += sum[i][threadIdx.x];
    n.part[(static_cast<size_t>(y) * g.gx + blockIdx.x) * D + threadIdx.x] = v;
  }
}

// dw of q (blockIdx.y = 0) and k (1): 8 columns a block, 128 threads a column, which add every 128th partial sum each and
// are joined in their order.
constexpr int kSumThreads = 1024, kSumLanes = kSumThreads / 8;

template <int D>
__global__ void __launch_bounds__(kSumThreads) norm_rope_weights_kernel(const NormRopeLaunch n, const BwdGrid g) {
  __shared__ float sum[kSumLanes][9];
  grid_dep_wait();  // launched programmatically after the kernel that leaves the partial sums
  float* const out = blockIdx.y ? n.dk_weight : n.dq_weight;
  const int first = blockIdx.y ? g.yq * g.gx : 0, count = (blockIdx.y ? g.yk : g.yq) * g.gx;
  const int col = threadIdx.x % 8, lane = threadIdx.x / 8;
  const float* p = n.part + static_cast<size_t>(first) * D + blockIdx.x * 8 + col;
  float v = 0.f;
#pragma unroll 8
  for (int i = lane; i < count; i += kSumLanes) v += p[static_cast<size_t>(i) * D];
  sum[lane][col] = v;
  __syncthreads();
  const int c = threadIdx.x / 32, l = threadIdx.x % 32;  // a warp a column
  if (c >= 8) return;
  double total = 0.0;
#pragma unroll
  for (int i = 0; i < kSumLanes / 32; ++i) total += sum[l + 32 * i][c];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (l == 0 && out) out[blockIdx.x * 8 + c] = static_cast<float>(total);
}

template <typename Kern, typename... Args>
cudaError_t launch_kernel(Kern kern, dim3 grid, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, bool INTER>
cudaError_t launch_t(NormRopeLaunch n, cudaStream_t stream) {
  RopeLaunch& a = n.r;
  const long long bx = (static_cast<long long>(a.B) * a.N + RopeCfg<D>::ROWS - 1) / RopeCfg<D>::ROWS;
  const int heads = a.Hq + a.Hk * (n.slots ? 2 : 1);
  a.heads = heads_per_thread(heads, n.slots ? kMostPagedHeads : kMostHeads);
  while (a.heads > 1 && bx * ((heads + a.heads - 1) / a.heads) < 4LL * a.sms) a.heads = (a.heads + 1) / 2;
  const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>((heads + a.heads - 1) / a.heads));
  return n.slots ? launch_kernel(norm_rope_kernel<D, INTER, true>, grid, kThreads, stream, n)
                 : launch_kernel(norm_rope_kernel<D, INTER, false>, grid, kThreads, stream, n);
}

template <int D, bool INTER>
cudaError_t launch_bwd_t(const NormRopeLaunch& n, cudaStream_t stream) {
  const RopeLaunch& a = n.r;
  const BwdGrid g = bwd_grid(a.B, a.Hq, a.Hk, a.N, D, a.sms);
  cudaError_t e = launch_kernel(norm_rope_bwd_kernel<D, INTER>,
                                dim3(static_cast<unsigned>(g.gx), static_cast<unsigned>(g.yq + g.yk)), kThreads, stream, n, g);
  if (e != cudaSuccess || !n.part) return e;
  return launch_kernel(norm_rope_weights_kernel<D>, dim3(D / 8, a.Hk > 0 ? 2 : 1), kSumThreads, stream, n, g);
}

}  // namespace

int norm_rope_partials(int B, int Hq, int Hk, int N, int d, int sms) {
  const BwdGrid g = bwd_grid(B, Hq, Hk, N, d, sms);
  return g.gx * (g.yq + g.yk);
}

cudaError_t launch_norm_rope(const NormRopeLaunch& a, cudaStream_t stream) {
  const fa_rope_axes_plan_t& plan = a.r.plan;
  if (plan.d == 64) return plan.interleaved ? launch_t<64, true>(a, stream) : launch_t<64, false>(a, stream);
  return plan.interleaved ? launch_t<128, true>(a, stream) : launch_t<128, false>(a, stream);
}

cudaError_t launch_norm_rope_bwd(const NormRopeLaunch& a, cudaStream_t stream) {
  const fa_rope_axes_plan_t& plan = a.r.plan;
  if (plan.d == 64) return plan.interleaved ? launch_bwd_t<64, true>(a, stream) : launch_bwd_t<64, false>(a, stream);
  return plan.interleaved ? launch_bwd_t<128, true>(a, stream) : launch_bwd_t<128, false>(a, stream);
}

}  // namespace fattn
