// Rotary positions with several axes (time, height, width, ...): pair i of a row's dimensions is
// turned by the angle pos[axis_i] * rate_i,
//     (a, b) -> (a cos - b sin, a sin + b cos),
// its inverse (which is its transpose, so it is the gradient) by the negative angle.  rope_kernel
// turns whole [B, H, N, d] tensors; rope_paged_kernel turns the new tokens of a decode or chunked
// prefill step and writes their k and v straight into the paged cache that fa_decode_paged reads.
//
// Angles.  The plan holds rate_i / (2 pi) as a 64-bit binary fraction of a turn, so
// pos * turns_i mod 2^64 is the exact fractional turn of that stored rate for every 32-bit
// position, negative ones included: one integer product replaces the range reduction, and a far
// position loses nothing (a 32-bit float product would be off by 2^-24 of the whole angle, a
// quarter of a radian at position 4 million).  Its top 32 bits, in half turns, go through
// sincospif.
//
// The work is bound by memory (4 bytes moved per element, 3 flops), so what counts is that the
// angles cost little beside it: a thread computes the 8 angles of its 8 pairs once and turns those
// pairs of `heads` heads of the row with them, 16-byte loads and stores, four heads in flight.
#include "rope_common.cuh"

namespace fattn {
namespace {

// Turn 8 pairs: x0, x1 are the two vectors (see first_vec), rounded to bf16 (nearest even) once.
template <bool INTER>
__device__ __forceinline__ void turn(uint4& x0, uint4& x1, const float (&c)[kPairs], const float (&s)[kPairs]) {
  uint32_t* u = reinterpret_cast<uint32_t*>(&x0);
  uint32_t* w = reinterpret_cast<uint32_t*>(&x1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTER) {  // each word holds one pair
      const float a0 = bf16lo(u[i]), b0 = bf16hi(u[i]), a1 = bf16lo(w[i]), b1 = bf16hi(w[i]);
      u[i] = pack_bf16(fmaf(a0, c[i], -b0 * s[i]), fmaf(a0, s[i], b0 * c[i]));
      w[i] = pack_bf16(fmaf(a1, c[4 + i], -b1 * s[4 + i]), fmaf(a1, s[4 + i], b1 * c[4 + i]));
    } else {
      const float a0 = bf16lo(u[i]), a1 = bf16hi(u[i]), b0 = bf16lo(w[i]), b1 = bf16hi(w[i]);
      const float c0 = c[2 * i], c1 = c[2 * i + 1], s0 = s[2 * i], s1 = s[2 * i + 1];
      u[i] = pack_bf16(fmaf(a0, c0, -b0 * s0), fmaf(a1, c1, -b1 * s1));
      w[i] = pack_bf16(fmaf(a0, s0, b0 * c0), fmaf(a1, s1, b1 * c1));
    }
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeLaunch a) {
  using C = RopeCfg<D>;
  __shared__ unsigned long long turns[D / 2];
  __shared__ unsigned char axis[D / 2];
  load_tables(a.plan, D, turns, axis);
  const int t = threadIdx.x % C::TPR;
  const long long rows = static_cast<long long>(a.B) * a.N;
  const long long r = static_cast<long long>(blockIdx.x) * C::ROWS + threadIdx.x / C::TPR;
  if (r >= rows) return;
  const long long b = r / a.N, n = r - b * a.N;
  int p[FA_ROPE_MAX_AXES];
#pragma unroll
  for (int k = 0; k < FA_ROPE_MAX_AXES; ++k) p[k] = k < a.plan.n_axes ? a.pos[k * rows + r] : 0;
  float c[kPairs], s[kPairs];
  angles(turns, axis, t, p, a.sign, c, s);
  const int h0 = static_cast<int>(blockIdx.y) * a.heads, h1 = min(h0 + a.heads, a.Hq + a.Hk);
  const int e0 = first_vec<D, INTER>(t), e1 = e0 + second_vec<D, INTER>();
  for (int h = h0; h < h1; h += kUnroll) {  // heads 0 .. Hq - 1 of q, then those of k
    const __nv_bfloat16* src[kUnroll];
    __nv_bfloat16* dst[kUnroll];
    uint4 x0[kUnroll], x1[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int hh = min(h + i, h1 - 1);
      const bool is_q = hh < a.Hq;
      const long long row = is_q ? b * a.Hq + hh : b * a.Hk + (hh - a.Hq);
      const long long off = (row * a.N + n) * D;
      src[i] = (is_q ? a.q : a.k) + off;
      dst[i] = (is_q ? a.q_out : a.k_out) + off;
      if (h + i < h1) {
        x0[i] = *reinterpret_cast<const uint4*>(src[i] + e0);
        x1[i] = *reinterpret_cast<const uint4*>(src[i] + e1);
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      if (h + i < h1) {
        turn<INTER>(x0[i], x1[i], c, s);
        *reinterpret_cast<uint4*>(dst[i] + e0) = x0[i];
        *reinterpret_cast<uint4*>(dst[i] + e1) = x1[i];
      }
  }
}

// Token t of sequence b is key seq_lens[b] + t.  Heads 0 .. Hq - 1 are q's (to q_out), the next Hk
// k's (turned, to the cache), the last Hk v's (copied to the cache).
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_paged_kernel(const RopeLaunch a) {
  using C = RopeCfg<D>;
  __shared__ unsigned long long turns[D / 2];
  __shared__ unsigned char axis[D / 2];
  load_tables(a.plan, D, turns, axis);
  const int t = threadIdx.x % C::TPR;
  const long long rows = static_cast<long long>(a.B) * a.N;
  const long long r = static_cast<long long>(blockIdx.x) * C::ROWS + threadIdx.x / C::TPR;
  if (r >= rows) return;
  const long long b = r / a.N, n = r - b * a.N;
  if (a.new_lens && n >= a.new_lens[b]) return;  // a padded token: nothing of it is written
  int p[FA_ROPE_MAX_AXES];
#pragma unroll
  for (int k = 0; k < FA_ROPE_MAX_AXES; ++k) p[k] = k < a.plan.n_axes ? a.pos[k * rows + r] : 0;
  // The token's row in the pools (of head 0), or none where the table has no page for it.
  const long long key = static_cast<long long>(a.seq_lens[b]) + n;
  const long long lp = key >= 0 ? key / a.page_size : a.max_pages;
  const int id = lp < a.max_pages ? a.block_table[b * a.max_pages + lp] : -1;
  const bool has_page = id >= 0 && id < a.num_pages;
  const long long page_row = (static_cast<long long>(id) * a.Hk) * a.page_size + (key - lp * a.page_size);
  float c[kPairs], s[kPairs];
  angles(turns, axis, t, p, a.sign, c, s);
  const int h0 = static_cast<int>(blockIdx.y) * a.heads, h1 = min(h0 + a.heads, a.Hq + 2 * a.Hk);
  const int e0 = first_vec<D, INTER>(t), e1 = e0 + second_vec<D, INTER>();
  for (int h = h0; h < h1; h += kUnroll) {
    uint4 x0[kUnroll], x1[kUnroll];
    __nv_bfloat16* dst[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int hh = min(h + i, h1 - 1);
      const __nv_bfloat16* src;
      if (hh < a.Hq) {
        const long long off = ((b * a.Hq + hh) * a.N + n) * D;
        src = a.q + off;
        dst[i] = a.q_out + off;
      } else {
        const bool is_v = hh >= a.Hq + a.Hk;
        const int hk = hh - a.Hq - (is_v ? a.Hk : 0);
        src = (is_v ? a.v : a.k) + ((b * a.Hk + hk) * a.N + n) * D;
        dst[i] = has_page ? (is_v ? a.v_out : a.k_out) + (page_row + static_cast<long long>(hk) * a.page_size) * D
                          : nullptr;
      }
      if (h + i >= h1) dst[i] = nullptr;
      if (dst[i]) {
        x0[i] = *reinterpret_cast<const uint4*>(src + e0);
        x1[i] = *reinterpret_cast<const uint4*>(src + e1);
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      if (dst[i]) {
        if (h + i < a.Hq + a.Hk) turn<INTER>(x0[i], x1[i], c, s);
        *reinterpret_cast<uint4*>(dst[i] + e0) = x0[i];
        *reinterpret_cast<uint4*>(dst[i] + e1) = x1[i];
      }
  }
}

template <int D, bool INTER>
cudaError_t launch_t(RopeLaunch a, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.B) * a.N;
  const long long bx = (rows + RopeCfg<D>::ROWS - 1) / RopeCfg<D>::ROWS;
  const int heads = a.Hq + a.Hk * (a.block_table ? 2 : 1);
  // Heads per thread: the angles cost about as much as turning three heads, so few heads make the kernel bound by
  // them, many leave the SMs without blocks.  Measured (GB300), 1 / 2 / 4 / 8 / 16 heads: B2 H16+16 N8192 d128 92 / 57 /
  // 42.3 / 42.5 / 43.6 us (6.4 TB/s), B4 H16+16 N2048 d64 23.6 / 15.6 / 13.2 / 14.3 / 13.5, a paged chunk of 4 x 517
  // tokens of 16 + 32 heads 11.7 / 7.7 / 6.2 / 6.0 / 7.6, one token of 8 sequences 3.3 / 3.3 / 3.4 / 4.3 / 6.2.  (256
  // threads a block: 42.5 at best, 13.4 and 6.2.)
  a.heads = 4;
  while (a.heads > 1 && bx * ((heads + a.heads - 1) / a.heads) < 4LL * a.sms) a.heads /= 2;
  const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>((heads + a.heads - 1) / a.heads));
  if (a.block_table)
    rope_paged_kernel<D, INTER><<<grid, kThreads, 0, stream>>>(a);
  else
    rope_kernel<D, INTER><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& a, cudaStream_t stream) {
  if (a.plan.d == 64) return a.plan.interleaved ? launch_t<64, true>(a, stream) : launch_t<64, false>(a, stream);
  return a.plan.interleaved ? launch_t<128, true>(a, stream) : launch_t<128, false>(a, stream);
}

}  // namespace fattn
