// Pieces shared by the backward kernels that take the scanned side in halves of 64 rows (fa_cross_bwd.cu,
// fa_window_bwd.cu): layouts, products and gradients of a half, rows that no pair reaches.
#pragma once
#include "bwd_common.cuh"

namespace fattn {
namespace {

constexpr int kHalf = kTile / 2;
constexpr int kIssuers = 3;
constexpr uint32_t kPair = 128;  // TMEM: pair g has S at 128 g, dP at 128 g + 64; the accumulators are last

// ACC: accumulator columns (2 d for dV and dK, d for dQ).
template <int D, int ACC>
struct CrossCfg {
  static constexpr int NH = D / 64;             // 128-byte boxes per row
  static constexpr uint32_t TB = NH * kBox;     // bytes of a 128 x d bf16 tile
  static constexpr int FLIGHT = (512 - ACC) / 128 < 3 ? (512 - ACC) / 128 : 3;  // half hh uses pair hh % FLIGHT
  // dQ: places for a query tile's Q and dO, and for its accumulator (two at d = 64)
  static constexpr int NB = ACC == 64 ? 2 : 1;
  static constexpr uint32_t COL_ACC = 512 - NB * ACC;
  static constexpr int EW = 4 * FLIGHT;         // elementwise warps
  static constexpr int MMA = EW, TMA = EW + kIssuers, THREADS = (TMA + 1) * 32;
  static constexpr int ST = D == 64 ? 4 : 2;    // ring stages
  static constexpr uint32_t OFF_A = 0, OFF_B = TB;  // the block's own tiles: K, V or Q, dO
  static constexpr uint32_t OFF_RING = NB * 2 * TB;  // stage: Q_i, dO_i or K_j, V_j
  static constexpr uint32_t STAGE = 2 * TB;
  // dK/dV: per stage a float4 for each pair of its query rows, {-lse2, -lse2, -D, -D} (lse2 = lse * log2(e))
  static constexpr uint32_t OFF_VEC = OFF_RING + ST * STAGE;
  static constexpr uint32_t VEC = 2 * kTile * 4;
  static constexpr uint32_t OFF_BAR = OFF_VEC + ST * VEC;
  static constexpr int B_OWN = 0, B_FULL = 2, B_EMPTY = B_FULL + ST, B_SF = B_EMPTY + ST, B_PF = B_SF + FLIGHT,
                       B_GD = B_PF + 2 * FLIGHT, B_GF = B_GD + FLIGHT, B_DRAIN = B_GF + 2, B_OW = B_DRAIN + kIssuers,
                       B_KC = B_OW + 2, NBAR = B_KC + ST;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 8u * NBAR;
  static constexpr uint32_t SMEM = OFF_MISC + 16u + 1024u;
  static_assert(SMEM <= 232448, "shared memory");
};

// Rows row0 .. row0 + rows - 1 of a gradient [.., D] that no pair reaches: zeros.
template <int D>
__device__ __forceinline__ void zero_rows(void* out, size_t row0, int rows, bool fp32) {
  const int row_bytes = D * (fp32 ? 4 : 2);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + row0 * row_bytes);
  for (int i = threadIdx.x; i < rows * row_bytes / 16; i += blockDim.x) dst[i] = make_uint4(0, 0, 0, 0);
}

// A key row behind its sequence (whatever its K and V hold): no gradient.
__device__ __forceinline__ void clear_pairs(uint32_t (&pp)[16], uint32_t (&dp)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) pp[i] = dp[i] = 0;
}

// The dQ kernel needs nothing of the dK/dV kernel that it is launched programmatically after (and overlaps), and a block
// of padding needs nothing at all, but what follows in the stream may: a grid's last block ends only when the
// grid before is complete.
__device__ __forceinline__ void wait_as_last_block() {
  if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && blockIdx.z == gridDim.z - 1) grid_dep_wait();
}

// Products of a 128-row tile A with rows 64 q .. of a streamed tile: 128 x 64, K = d.
template <int D>
__device__ __forceinline__ void issue_half_product(uint32_t d_tmem, uint64_t da, uint64_t db, int q) {
  constexpr uint32_t idesc = idesc_bf16_f32(kTile, kHalf, 0);
  issue_product<D>(d_tmem, da, sdesc_add(db, static_cast<uint32_t>(q) * kHalf * 128u), idesc);
}
// G (+)= X Y for chunk c (32 of the half's 64 rows): X packed at columns 16 c .., Y rows 64 q + 32 c .. of an
// MN-major 128 x d tile
template <int D>
__device__ __forceinline__ void issue_half_chunk(uint32_t g_tmem, uint32_t x_tmem, uint64_t dy, int q, int c,
                                                 bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(kTile, D, 1);
#pragma unroll
  for (int m = 0; m < 2; ++m) {  // 16 rows each
    const uint32_t a = x_tmem + 16u * c + 8u * m;
    const uint64_t b = sdesc_add(dy, static_cast<uint32_t>(kHalf * q + 32 * c + 16 * m) * 128u);
    if (m == 0 && !accumulate) mma_ts_c<0>(g_tmem, a, b, idesc);
    else mma_ts_c<1>(g_tmem, a, b, idesc);
  }
}

}  // namespace
}  // namespace fattn
