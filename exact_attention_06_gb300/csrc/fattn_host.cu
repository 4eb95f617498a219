// Host side of the libfattn C ABI: argument validation, TMA tensor-map
// encoding, kernel launches and the status word.  Declared in fattn.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "fattn.h"
#include "internal.h"

namespace {

thread_local char g_last_error[512] = "";

fa_status_t fail(fa_status_t st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return st;
}

fa_status_t cuda_fail(cudaError_t e, const char* what) {
  return fail(FA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ---------------------------------------------------------------- device info
struct DevInfo {
  bool known = false;
  int major = 0, minor = 0, sms = 0;
};
constexpr int kMaxDevices = 64;
DevInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

fa_status_t check_device(int* sms) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0) return fail(FA_ERR_ARCH, "no CUDA device: %s", cudaGetErrorString(e));
  if (dev >= kMaxDevices) return fail(FA_ERR_ARCH, "device ordinal %d out of range", dev);
  DevInfo info;
  {
    std::lock_guard<std::mutex> lock(g_dev_mu);
    if (!g_dev[dev].known) {
      DevInfo d;
      if (cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
          cudaDeviceGetAttribute(&d.minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
          cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return fail(FA_ERR_ARCH, "cannot query device %d", dev);
      d.known = true;
      g_dev[dev] = d;
    }
    info = g_dev[dev];
  }
  if (info.major != 10 || info.minor != 3)
    return fail(FA_ERR_ARCH, "device %d has compute capability %d.%d; libfattn is built for sm_103a (10.3)", dev,
                info.major, info.minor);
  if (sms) *sms = info.sms;
  return FA_OK;
}

// ---------------------------------------------------------------- status words
// Each kernel file has a status word of its own.  One kernel takes (reads and clears) them all: a copy from and one to each
// of the seven words took fa_get_status 94 us; this takes 22.
constexpr int kStatusWords = 7;
struct StatusWords {
  unsigned int* p[kStatusWords];
};
__device__ unsigned int g_taken_status = 0;

__global__ void take_status_kernel(const StatusWords w) {
  unsigned int v = 0;
  for (int i = 0; i < kStatusWords; ++i) v |= atomicExch(w.p[i], 0u);
  g_taken_status = v;
}

// The bits raised since the last call on the current device.  One caller at a time, since they share g_taken_status.
cudaError_t take_status(cudaStream_t stream, unsigned int* bits) {
  using Word = cudaError_t (*)(unsigned int**);
  constexpr Word kWord[kStatusWords] = {
      fattn::fwd_status_word,        fattn::decode_status_word,      fattn::bwd_status_word,
      fattn::cross_bwd_status_word,  fattn::cross_rows_status_word,  fattn::cross_short_status_word,
      fattn::cross_bwd_short_status_word};
  static std::mutex mu;
  static StatusWords words[kMaxDevices];
  static bool known[kMaxDevices] = {};
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!known[dev]) {
    for (int i = 0; i < kStatusWords; ++i)
      if ((e = kWord[i](&words[dev].p[i])) != cudaSuccess) return e;
    known[dev] = true;
  }
  cudaGetLastError();
  take_status_kernel<<<1, 1, 0, stream>>>(words[dev]);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = cudaMemcpyFromSymbolAsync(bits, g_taken_status, sizeof(*bits), 0, cudaMemcpyDeviceToHost, stream);
  return e == cudaSuccess ? cudaStreamSynchronize(stream) : e;
}

// ---------------------------------------------------------------- tensor maps
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// A tensor [batches, rows, d] (d innermost) of bf16 (esz = 2) or bytes (esz = 1, E4M3
// codes) seen as 3-D {d, rows, batches}, loaded in boxes of 128 bytes (64 bf16 or 128
// E4M3 columns) x box_rows rows with 128-byte swizzle.  Rows past `rows` read as zeros.
fa_status_t make_map(CUtensorMap* map, const void* base, int d, long long rows, long long batches, int box_rows,
                     int esz = 2) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(batches)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * esz, static_cast<cuuint64_t>(rows) * d * esz};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / esz), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType dt = esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUresult r = enc(map, dt, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled failed with CUresult %d", static_cast<int>(r));
  return FA_OK;
}

using fattn::kDefaultBudget;

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct DecodePlan {
  int splits = 0;
  int keys_per_split = 0;
  size_t u_bytes = 0, m_bytes = 0, l_bytes = 0;
  size_t total() const { return u_bytes + m_bytes + l_bytes; }
};

// Splits per (b, h) when the caller passes 0: the fewest that fill the GPU's
// resident split-CTA slots to within 3% in the last wave (or, when even one
// partial per chunk cannot fill one wave, one partial per chunk).
int auto_splits(long long bh, int n_chunks, int sms) {
  const double slots = static_cast<double>(sms) * fattn::kDecodeCtasPerSm;
  int best = 1;
  double best_eff = -1.0;
  for (int s = 1; s <= n_chunks; ++s) {
    const int cps = (n_chunks + s - 1) / s;
    if ((n_chunks + cps - 1) / cps != s) continue;  // would leave a split empty
    const double waves = static_cast<double>(bh) * s / slots;
    const double eff = waves < 1.0 ? waves : waves / std::ceil(waves);
    if (eff >= 0.97) return s;
    if (eff > best_eff + 1e-12) {
      best_eff = eff;
      best = s;
    }
  }
  return best;
}

fa_status_t plan_decode(int B, int H, int L, int d, int chunk, int splits, int sms, DecodePlan* plan) {
  if (B < 1 || H < 1 || L < 1) return fail(FA_ERR_INVALID_ARG, "B, H and L must be >= 1 (got %d, %d, %d)", B, H, L);
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dimension d=%d is not supported (64 or 128)", d);
  if (chunk != 128) return fail(FA_ERR_UNSUPPORTED, "chunk=%d is not supported (128)", chunk);
  const long long bh = static_cast<long long>(B) * H;
  const int n_chunks = (L + chunk - 1) / chunk;
  if (splits < 0 || splits > n_chunks)
    return fail(FA_ERR_INVALID_ARG, "splits=%d must be in [0, %d] for L=%d", splits, n_chunks, L);
  const int s = splits == 0 ? auto_splits(bh, n_chunks, sms) : splits;
  if (bh * s > INT_MAX) return fail(FA_ERR_UNSUPPORTED, "B*H*splits=%lld exceeds the grid limit", bh * s);
  plan->splits = s;
  plan->keys_per_split = ((n_chunks + s - 1) / s) * chunk;
  plan->u_bytes = round256(static_cast<size_t>(bh) * s * d * sizeof(float));
  plan->m_bytes = round256(static_cast<size_t>(bh) * s * sizeof(float));
  plan->l_bytes = round256(static_cast<size_t>(bh) * s * sizeof(float));
  return FA_OK;
}


// Splits for the paged decode: as for the contiguous cache, then raised if a split would
// touch more than kMaxSplitPages pages (only for very long sequences with small pages).
fa_status_t plan_paged(int B, int H, int L, int d, int page_size, int splits, int sms, DecodePlan* plan) {
  fa_status_t st = plan_decode(B, H, L, d, 128, splits, sms, plan);
  if (st != FA_OK) return st;
  auto pages_of = [&](const DecodePlan& p) { return p.keys_per_split / page_size + 1; };
  if (pages_of(*plan) <= fattn::kMaxSplitPages) return FA_OK;
  if (splits != 0)
    return fail(FA_ERR_UNSUPPORTED, "splits=%d gives %d keys per split, more than %d pages of %d keys", splits,
                plan->keys_per_split, fattn::kMaxSplitPages - 1, page_size);
  const int n_chunks = (L + 127) / 128;
  const int chunks_per_split = ((fattn::kMaxSplitPages - 1) * page_size) / 128;
  return plan_decode(B, H, L, d, 128, (n_chunks + chunks_per_split - 1) / chunks_per_split, 0, plan);
}

// The last round of the non-causal d = 64 forward.  With one resident CTA per SM, U blocks of 256
// query rows run in ceil(U / sms) rounds, the last holding rem blocks.  Two ways to spread that
// round over more SMs:
//   key split: each of the rem blocks becomes k key pieces (>= 2 key tiles each) that leave
//     partial (U, m, l) rows, merged by the combine kernel (needs a workspace);
//   query split: each becomes two single-tile items (when 2 * rem <= sms; no workspace).
// Costs are counted in key-tile steps of a whole block: a block costs its n key tiles plus ~2
// of set-up and epilogue, a piece its share plus 2, the combine (with its launch) ~3; a
// single-tile item runs alone on its SM at ~0.72 of a whole block (both measured on GB300).
// The cheapest wins if it saves at least 5 % of the launch; ties go to the query split.
struct TailPlan {
  int ksplit = 1;  // > 1: key split into ksplit pieces
  int qsplit = 0;  // 1: query split (used when there is no key split, with or without a workspace)
  int n_full = 0, kchunk = 0;
  long long prow0 = 0, rows = 0;
  size_t u_bytes = 0, m_bytes = 0, l_bytes = 0;
  size_t total() const { return u_bytes + m_bytes + l_bytes; }
};

TailPlan plan_tail(long long bh, int N, int d, int causal, int sms) {
  TailPlan p;
  if (causal || d != 64 || sms < 1) return p;  // the persistent d = 64 kernel runs the split rounds
  const long long n_pairs = (N + 255) / 256;
  const long long U = bh * n_pairs;
  const int n_tiles = (N + 127) / 128;
  const long long waves = (U + sms - 1) / sms;
  const long long rem = U - (waves - 1) * sms;
  constexpr double kFixed = 2.0, kCombine = 3.0, kSingleTile = 0.72;
  const double t_whole = n_tiles + kFixed;
  const double t_q = 2 * rem <= sms ? kSingleTile * t_whole : t_whole;
  double best_t = t_whole;
  int best_k = 1, best_tpp = n_tiles;
  for (int k = 2; k <= 8 && 2 * k <= n_tiles; ++k) {
    const int tpp = (n_tiles + k - 1) / k;  // key tiles per piece
    if ((n_tiles + tpp - 1) / tpp != k) continue;
    const double t = std::ceil(static_cast<double>(k * rem) / sms) * (tpp + kFixed) + kCombine;
    if (t < best_t - 1e-9) {
      best_t = t;
      best_k = k;
      best_tpp = tpp;
    }
  }
  const double margin = 0.05 * waves * t_whole;
  if (U - rem + 2 * rem > INT_MAX || U - rem + rem * best_k > INT_MAX) return p;
  p.n_full = static_cast<int>(U - rem);
  if (t_q < t_whole - margin) p.qsplit = 1;  // the fallback whenever there is no key split
  if (best_k == 1 || best_t >= t_q || t_whole - best_t < margin) return p;
  p.ksplit = best_k;
  p.kchunk = best_tpp * 128;
  p.prow0 = (p.n_full / n_pairs) * N + (p.n_full % n_pairs) * 256;
  p.rows = bh * N - p.prow0;
  p.u_bytes = round256(static_cast<size_t>(p.rows) * best_k * d * sizeof(float));
  p.m_bytes = round256(static_cast<size_t>(p.rows) * best_k * sizeof(float));
  p.l_bytes = p.m_bytes;
  return p;
}

fa_status_t check_paged_args(int B, int H, int d, int page_size, int max_pages, int num_pages, int max_seq_len) {
  if (B < 1 || H < 1) return fail(FA_ERR_INVALID_ARG, "B and H must be >= 1 (got %d, %d)", B, H);
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dimension d=%d is not supported (64 or 128)", d);
  if (page_size < 64 || page_size % 64 != 0)
    return fail(FA_ERR_UNSUPPORTED, "page_size=%d must be a positive multiple of 64", page_size);
  if (max_pages < 1 || num_pages < 1)
    return fail(FA_ERR_INVALID_ARG, "max_pages and num_pages must be >= 1 (got %d, %d)", max_pages, num_pages);
  if (max_seq_len < 1 || static_cast<long long>(max_seq_len) > static_cast<long long>(max_pages) * page_size)
    return fail(FA_ERR_INVALID_ARG, "max_seq_len=%d must be in [1, max_pages * page_size]", max_seq_len);
  if (static_cast<long long>(num_pages) * H > INT_MAX)
    return fail(FA_ERR_UNSUPPORTED, "num_pages*H=%lld exceeds the page index range",
                static_cast<long long>(num_pages) * H);
  return FA_OK;
}

// Cross attention.  The G = Hq / Hkv query heads of a key head are adjacent in q, so their rows are
// G * Nq rows of one [B * Hkv, G * Nq, d] tensor against the key head's [Nk, d]: shared heads need
// nothing more, and dK, dV sum over the group by themselves.
struct CrossShape {
  long long bh = 0;  // B * Hkv
  int rows = 0;      // G * Nq
};

fa_status_t check_cross_args(int B, int Hq, int Hkv, int Nq, int Nk, int d, CrossShape* c) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1 || Nk < 1)
    return fail(FA_ERR_INVALID_ARG, "B, Hq, Hkv, Nq and Nk must be >= 1 (got %d, %d, %d, %d, %d)", B, Hq, Hkv, Nq, Nk);
  if (Hq % Hkv != 0) return fail(FA_ERR_INVALID_ARG, "Hq=%d must be a multiple of Hkv=%d", Hq, Hkv);
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dimension d=%d is not supported (64 or 128)", d);
  c->bh = static_cast<long long>(B) * Hkv;
  const long long rows = static_cast<long long>(Hq / Hkv) * Nq;
  if (c->bh > INT_MAX) return fail(FA_ERR_UNSUPPORTED, "B*Hkv=%lld exceeds the grid limit", c->bh);
  if ((rows + 127) / 128 > 65535)
    return fail(FA_ERR_UNSUPPORTED, "Hq/Hkv*Nq=%lld exceeds the 65535 query-tile grid limit", rows);
  if ((static_cast<long long>(Nk) + 127) / 128 > 65535)
    return fail(FA_ERR_UNSUPPORTED, "Nk=%d exceeds the 65535 key-tile grid limit", Nk);
  c->rows = static_cast<int>(rows);
  return FA_OK;
}

// How often to cut a scan of `tiles` tiles when `units` blocks (one per SM at a time) each make it:
// more, shorter blocks fill the SMs, at the price of fp32 partial results and a kernel that joins
// them.  Costs in tile steps (about 1 us): a block costs its tiles plus ~3 of set-up and epilogue,
// joining ~3 and its traffic, 8 MB a step.  A cut has to save 5 %.  `filler`: steps of work (over all
// SMs) of a kernel that runs on the SMs which this one's last round leaves idle; with it only the longest
// SM and the sum of the work count.
int cut_scan(long long units, int tiles, int sms, double part_bytes, double filler = 0.0) {
  constexpr double kFixed = 3.0, kJoin = 3.0, kStepBytes = 8e6;
  auto time = [&](int s, int each) {
    const double rounds = static_cast<double>((units * s + sms - 1) / sms);
    return std::fmax(rounds * (each + kFixed),
                     (static_cast<double>(units) * s * (each + kFixed) + filler) / sms);
  };
  const double whole = time(1, tiles);
  double best_t = 0.95 * whole;
  int best = 1;
  for (int s = 2; s <= tiles && s <= 256; ++s) {
    const int each = (tiles + s - 1) / s;
    if ((tiles + each - 1) / each != s) continue;  // would leave a block without tiles
    const double t = time(s, each) + kJoin + 2.0 * s * part_bytes / kStepBytes;
    if (t < best_t) {
      best_t = t;
      best = s;
    }
  }
  return best;
}

struct CrossPlan {
  int few = 0;    // 1: the few-row kernel; its splits are a cluster unless `parts`
  int tiles = 0;  // > 0: the short-key kernel, this many query tiles a block
  int parts = 0;
  int splits = 1, kchunk = 0;
  size_t u_bytes = 0, m_bytes = 0;
  size_t total() const { return parts ? u_bytes + 2 * m_bytes : 0; }
};

// The few-row kernel's blocks per key head.  Costs in the time a 64-key stage takes an SM at its share of
// HBM: the whole call cannot be faster than all stages shared out; a block takes at least 0.73 a stage
// (its chain of copies and products); set-up and join cost 3 a round of resident blocks and 0.12 a block of
// the cluster, partials and the combine kernel 3 more.  Clusters (up to 8 blocks) need neither partials
// nor a second kernel; of theirs the largest within 4 % of the best is taken, since shorter blocks even out
// sequences of different lengths.
// Measured (GB300, d = 128): 64 key heads x 577 keys, S = 1 / 2 / 4 / 5: 8.2 / 6.2 / 6.2 / 10.0 us;
// 64 x 18k-32k keys, S = 2 / 4 / 8 / 19: 143 / 124 / 120 / 128 us; 8 x 16384, S = 8 / 16 / 32: 20.3 / 15.6 /
// 17.7 us.
void plan_few(CrossPlan* p, const CrossShape& c, int Nk, int d, int sms, bool allow_parts) {
  constexpr double kBlock = 0.73, kFixed = 3.0, kMember = 0.12, kJoin = 3.0, kNear = 1.04;
  const int stages = (Nk + fattn::kRowsStageKeys - 1) / fattn::kRowsStageKeys;
  const long long slots = static_cast<long long>(sms) * fattn::cross_rows_per_sm(d, c.rows);
  const double all = static_cast<double>(c.bh) * stages / sms;
  auto cost = [&](int s) {
    const double rounds = static_cast<double>((c.bh * s + slots - 1) / slots);
    return std::fmax(all, kBlock * rounds * ((stages + s - 1) / s)) + kFixed * rounds + (s > 8 ? kJoin : kMember * s);
  };
  const int most = std::min(stages, 8);
  double best = cost(1);
  for (int s = 2; s <= most; ++s) best = std::fmin(best, cost(s));
  p->splits = 1;
  for (int s = 2; s <= most; ++s)
    if (cost(s) <= kNear * best && c.bh * s <= INT_MAX) p->splits = s;
  for (int s = 9; allow_parts && s <= 256 && s <= stages && c.bh * s <= INT_MAX; ++s)
    if (cost(s) < best) {
      best = cost(s);
      p->splits = s;
    }
  p->few = 1;
  p->parts = p->splits > 8;
}

// The short-key kernel's query tiles per block: about 1 us a tile, 4 a block's set-up and end.
// At most 128 keys take that kernel.  Measured (GB300) against the kernels for any number of keys, us:
//   heads, rows x keys        d = 64         d = 128
//   2 x 16, 8192 x 64     29.8 -> 15.7    53.1 -> 27.0
//   2 x 16, 8192 x 77     29.6 -> 19.1    53.1 -> 30.0
//   2 x 16, 8192 x 128    26.4 -> 23.7    51.0 -> 31.4
//   4 x 16, 2048 x 77     18.0 -> 12.6    31.2 -> 18.0
//   1 x 8, 1000 x 77       5.9 ->  4.3     6.7 ->  5.2
//   8 x 16/2, 5880 x 4    73.8 -> 35.8   137.7 -> 63.8
//   8 x 64/16, 4595 x 49   216 ->  101     414 ->  198   (6.1 TB/s)
// A tile has 64, 96 or 128 keys: at d = 64, 77 keys take 24.1 us where the tile has 128 (8192 rows).
int plan_short(const CrossShape& c, int sms) {
  const int n = (c.rows + 127) / 128;
  int best = 1;
  double best_t = 0;
  for (int tiles = 1; tiles <= n; tiles = tiles < 8 ? tiles + 1 : tiles + tiles / 8) {
    const long long blocks = c.bh * ((n + tiles - 1) / tiles);
    const double t = static_cast<double>((blocks + sms - 1) / sms) * (tiles + 4.0);
    if (tiles == 1 || t < best_t) {
      best_t = t;
      best = tiles;
    }
  }
  return best;
}

CrossPlan plan_cross(const CrossShape& c, int Nk, int d, int sms, bool workspace) {
  CrossPlan p;
  const int tiles = (Nk + 127) / 128;
  const long long rows = c.bh * c.rows;
  const bool can_join = workspace && rows <= INT_MAX;  // (the combine kernel's row count)
  // At most 32 rows a key head take the few-row kernel.  Measured against the 128-row tiles (d = 128, 1 / 16 / 17 / 32
  // rows): 64 key heads x 8192 keys 41 / 43 / 46 / 48 us against 51 / 53 / 53 / 54; 512 x 1500 keys 60 / 64 / 82 / 88
  // against 83 / 87 / 87 / 88; 64 x 577 keys 5.9 / 7.5 / 8.2 / 9.6 against 10.8.
  // Against the short-key kernel (d = 128, 77 keys, 1 / 8 / 17 / 32 rows): 16 key heads 4.6 / 4.8 / 6.1 / 7.3 against
  // 4.5 / 4.8 / 4.8 / 4.7; 512 key heads 9.6 / 11.4 / 22.6 / 28.7 against 15.7 / 15.9 / 16.2 / 16.8.  At d = 64, 512
  // key heads: 6.1 / 6.5 / 11.3 / 13.5 against 13.7 / 13.5 / 13.4 / 13.6.  So at most 128 keys: 16 rows, one row block.
  const bool short_keys = Nk <= fattn::kCrossShortKeys;
  if (c.rows <= (short_keys ? fattn::kCrossRowsMax / 2 : fattn::kCrossRowsMax))
    plan_few(&p, c, Nk, d, sms, can_join);
  else if (short_keys)
    p.tiles = plan_short(c, sms);
  else if (can_join)
    p.splits = cut_scan(c.bh * ((c.rows + 255) / 256), tiles, sms, static_cast<double>(rows) * (d + 2) * 4);
  if (!p.few) p.parts = p.splits > 1;
  p.kchunk = (tiles + p.splits - 1) / p.splits * 128;
  p.u_bytes = round256(static_cast<size_t>(rows) * p.splits * d * sizeof(float));
  p.m_bytes = round256(static_cast<size_t>(rows) * p.splits * sizeof(float));
  return p;
}

struct CrossBwdPlan {
  int kv_splits = 1, q_tiles = 0;  // dK, dV: ranges of query tiles
  int q_splits = 1, k_tiles = 0;   // dQ: ranges of key tiles
  size_t delta_bytes = 0, kv_bytes = 0, q_bytes = 0;
  size_t total() const { return std::max<size_t>(delta_bytes + kv_bytes + q_bytes, 256); }  // never none
};

// Query tiles that a block of the dQ kernel takes: each saves most of a block's set-up and end, but longer blocks end
// less evenly.  The dQ blocks take the SMs that the dK/dV kernel's last round leaves idle, then all; the choice is the
// number with which the last of them ends first, by these times in us of: a query tile of dK/dV, its blocks' fixed part,
// a key tile of dQ, a query tile's part of its own, its blocks' fixed part.  Measured (GB300, the whole backward, us):
//                                 tiles  1     2     3     4     6     8   (a kernel of one tile)
//   d = 64, 2 x 16 heads, 8192 x 256   121   101    96    94    91    93   (116)
//                         8192 x 512   176   153   147   144   141   153   (167)
//           4 x 16/4, 2048 x 1500      199   196   191   195   220   236   (195)
//   d = 128, 2 x 16, 8192 x 154        166   159   155   158   153   158   (164)
//                    4096 x 2048       403   397   414   439   479   438   (396)
// Where kv_lens is given (ragged), blocks end less evenly still, and a block takes at most 24 key tiles.  The lengths are
// device data, so the rule cannot see that they are all alike.  Measured (the whole backward, us, with the rule / without):
//                                      lengths from 1 to Nk   from Nk/2 to Nk   all Nk
//   d = 64,  4 x 32/8, 1024 x 640           70 / 82               90 / 90        95 / 91
//            8 x 16/4, 1000 x 577           67 / 81               87 / 89        94 / 92
//            8 x 8/2,  4096 x 1024         192 / 196             214 / 220      250 / 253
//            4 x 16/4, 2048 x 1500          97 / 95              167 / 171      199 / 191
//            2 x 16,   4096 x 2048          95 / 87              231 / 229      263 / 249
//   d = 128, 4 x 32/8, 1024 x 640          118 / 154             149 / 153      159 / 157
//            8 x 16/4, 1000 x 577          112 / 141             145 / 153      159 / 158
//            8 x 8/2,  4096 x 1024         317 / 334             348 / 373      416 / 413
//            4 x 16/4, 2048 x 1500         158 / 159             269 / 275      312 / 305
//            2 x 16,   4096 x 2048         142 / 141             357 / 363      407 / 402
int dq_own_tiles(const CrossBwdPlan& p, long long bh, int qt, int kt, int d, int sms, bool ragged) {
  const double kv_step = d == 64 ? 1.16 : 1.8, kv_fixed = 3.5;
  const double q_step = d == 64 ? 0.87 : 1.34, q_tile = d == 64 ? 0.9 : 2.5, q_fixed = 3.0;
  const long long kv_blocks = bh * kt * p.kv_splits, busy = kv_blocks % sms;  // SMs with a block in dK/dV's last round
  const double early = static_cast<double>(kv_blocks / sms) * (p.q_tiles * kv_step + kv_fixed);
  const double late = early + (busy ? p.q_tiles * kv_step + kv_fixed : 0.0);
  int best = 1;
  double best_t = 0;
  for (int own = 1; own <= qt && own <= 8; ++own) {
    if (ragged && own > 1 && own * p.k_tiles > 24) break;
    const long long blocks = bh * ((qt + own - 1) / own) * p.q_splits;
    const double each = own * (p.k_tiles * q_step + q_tile) + q_fixed;
    auto done_by = [&](double t) {  // blocks
      auto on = [&](double from) { return t > from ? static_cast<long long>((t - from) / each + 1e-9) : 0LL; };
      return (sms - busy) * on(early) + busy * on(late);
    };
    double even = early + blocks * each / (sms - busy);  // no earlier: work that can be shared evenly
    if (busy && even > late) even = (blocks * each + (sms - busy) * early + busy * late) / sms;
    auto last_end = [&](double from) {  // the first end of a block, on SMs that begin at `from`, by which all are done
      double n = std::fmax(1.0, std::ceil((even - from) / each - 1e-6));
      while (done_by(from + n * each) < blocks) n += 1.0;
      return from + n * each;
    };
    const double t = std::fmax(busy ? std::fmin(last_end(early), last_end(late)) : last_end(early), late);
    if (own == 1 || t < best_t) {
      best_t = t;
      best = own;
    }
  }
  return best;
}

CrossBwdPlan plan_cross_bwd(const CrossShape& c, int Nk, int d, int sms) {
  CrossBwdPlan p;
  const int qt = (c.rows + 127) / 128, kt = (Nk + 127) / 128;
  const double kv = 2.0 * c.bh * Nk * d * sizeof(float), q = 1.0 * c.bh * c.rows * d * sizeof(float);
  // At most 128 keys take the one-pass kernel, whose step is a query tile.  Measured (GB300) against the dQ and dK/dV
  // kernels of more keys, us:
  //   heads, rows x keys        d = 64         d = 128
  //   2 x 16, 8192 x 64        89 -> 27      117 -> 46
  //   2 x 16, 8192 x 77       102 -> 37      133 -> 51
  //   2 x 16, 8192 x 128      101 -> 44      134 -> 56
  //   4 x 16, 2048 x 77        57 -> 23       73 -> 32
  //   1 x 8, 1000 x 77       13.4 -> 9.5    16.5 -> 11.7
  //   8 x 16/2, 5880 x 4      244 -> 61      313 -> 105
  //   8 x 64/16, 4595 x 49    740 -> 176     960 -> 321
  //   64 x 8, 40 x 100         40 -> 25       49 -> 34
  // Ranges of queries per key head, 2 x 16 heads, 8192 x 77, d = 128, 1 / 2 / 4 / 8: 154 / 83 / 51 / 60 us.
  if (Nk <= fattn::kCrossShortKeys) {
    p.kv_splits = cut_scan(c.bh, qt, sms, kv);
    p.q_tiles = (qt + p.kv_splits - 1) / p.kv_splits;
    if (p.kv_splits > 1) p.kv_bytes = round256(static_cast<size_t>(kv) * p.kv_splits);
    return p;
  }
  // The dQ kernel fills the dK/dV kernel's last round; a step of it costs about 0.75 of the latter's.  Measured
  // (GB300, ranges of queries per key tile 1 / 2 / 3 / 4, both kernels and the join): B4 H16/4 2048 x 1500 at
  // d = 64: 193 / 204 / 215 / 222 us; B2 H16/4 1000 x 577: 40 / 33 / 36 / 35 us; B1 H8/2 4096 x 300, 1 / 8 / 16 / 32:
  // 134 / 28 / 26 / 32 us.
  p.q_splits = cut_scan(c.bh * qt, kt, sms, q);
  p.kv_splits = cut_scan(c.bh * kt, qt, sms, kv, 0.75 * c.bh * qt * (kt + 3));
  p.q_tiles = (qt + p.kv_splits - 1) / p.kv_splits;
  p.k_tiles = (kt + p.q_splits - 1) / p.q_splits;
  p.delta_bytes = round256(static_cast<size_t>(c.bh) * c.rows * sizeof(float));
  if (p.kv_splits > 1) p.kv_bytes = round256(2ull * c.bh * Nk * d * sizeof(float) * p.kv_splits);
  if (p.q_splits > 1) p.q_bytes = round256(1ull * c.bh * c.rows * d * sizeof(float) * p.q_splits);
  return p;
}

fa_status_t check_rope_args(const fa_rope_axes_plan_t* plan, const int* pos, int B, int Hq, int Hk, int N, int inverse) {
  if (!plan || !pos) return fail(FA_ERR_INVALID_ARG, "null plan or pos");
  if ((plan->d != 64 && plan->d != 128) || plan->n_axes < 1 || plan->n_axes > FA_ROPE_MAX_AXES)
    return fail(FA_ERR_INVALID_ARG, "plan was not made by fa_rope_axes_plan");
  for (int i = 0; i < plan->d / 2; ++i)
    if (plan->axis[i] >= plan->n_axes) return fail(FA_ERR_INVALID_ARG, "plan was not made by fa_rope_axes_plan");
  if (B < 1 || Hq < 1 || Hk < 0 || N < 1)
    return fail(FA_ERR_INVALID_ARG, "B, Hq and N must be >= 1, Hk >= 0 (got %d, %d, %d, %d)", B, Hq, N, Hk);
  if (inverse != 0 && inverse != 1) return fail(FA_ERR_INVALID_ARG, "inverse must be 0 or 1");
  if (!aligned(pos, 4)) return fail(FA_ERR_INVALID_ARG, "pos must be 4-byte aligned");
  if (static_cast<long long>(Hq) + 2LL * Hk > 65535)
    return fail(FA_ERR_UNSUPPORTED, "Hq=%d and Hk=%d exceed the 65535 head grid limit", Hq, Hk);
  if (static_cast<long long>(B) * N > INT_MAX)
    return fail(FA_ERR_UNSUPPORTED, "B*N=%lld exceeds the row limit", static_cast<long long>(B) * N);
  return FA_OK;
}

}  // namespace

extern "C" {

const char* fa_status_string(fa_status_t status) {
  switch (status) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED";
    case FA_ERR_ARCH: return "FA_ERR_ARCH";
    case FA_ERR_CUDA: return "FA_ERR_CUDA";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT";
    case FA_ERR_WORKSPACE: return "FA_ERR_WORKSPACE";
  }
  return "FA_ERR_UNKNOWN";
}

const char* fa_last_error(void) { return g_last_error; }

fa_status_t fa_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, int d,
                      float scale, int causal, void* stream, const fa_fwd_opts* opts) {
  g_last_error[0] = '\0';
  if (!q || !k || !v || !o || !lse) return fail(FA_ERR_INVALID_ARG, "null tensor pointer");
  if (B < 1 || H < 1 || N < 1) return fail(FA_ERR_INVALID_ARG, "B, H and N must be >= 1 (got %d, %d, %d)", B, H, N);
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dimension d=%d is not supported (64 or 128)", d);
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (causal != 0 && causal != 1) return fail(FA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16))
    return fail(FA_ERR_INVALID_ARG, "q, k, v and o must be 16-byte aligned");
  if (!aligned(lse, 4)) return fail(FA_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  const int o_fp32 = opts ? opts->o_fp32 : 0;
  if (o_fp32 != 0 && o_fp32 != 1) return fail(FA_ERR_INVALID_ARG, "opts->o_fp32 must be 0 or 1");
  const long long bh = static_cast<long long>(B) * H;
  if (bh > INT_MAX) return fail(FA_ERR_UNSUPPORTED, "B*H=%lld exceeds the grid limit", bh);
  if ((N + 127) / 128 > 65535) return fail(FA_ERR_UNSUPPORTED, "N=%d exceeds the 65535 query-tile grid limit", N);
  int sms = 0;
  fa_status_t st = check_device(&sms);
  if (st != FA_OK) return st;
  void* ws = opts ? opts->workspace : nullptr;
  TailPlan tail = plan_tail(bh, N, d, causal, sms);
  if (!ws) tail.ksplit = 1;  // no workspace: no key split (the query split still applies)
  if (tail.ksplit > 1) {
    if (opts->workspace_bytes < tail.total())
      return fail(FA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes fa_fwd_workspace_bytes gives",
                  opts->workspace_bytes, tail.total());
    if (!aligned(ws, 256)) return fail(FA_ERR_INVALID_ARG, "opts->workspace must be 256-byte aligned");
  }

  fattn::FwdLaunch a{};
  if ((st = make_map(&a.tq, q, d, N, bh, 128)) != FA_OK) return st;
  if ((st = make_map(&a.tk, k, d, N, bh, 128)) != FA_OK) return st;
  if ((st = make_map(&a.tv, v, d, N, bh, 128)) != FA_OK) return st;
  if (!o_fp32 && (st = make_map(&a.to, o, d, N, bh, 128)) != FA_OK) return st;
  a.o = o;
  a.lse = lse;
  a.N = N;
  a.BH = static_cast<int>(bh);
  a.d = d;
  a.causal = causal;
  a.o_fp32 = o_fp32;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.budget = (opts && opts->wait_budget_cycles) ? opts->wait_budget_cycles : kDefaultBudget;
  a.aux.Nk = N;
  a.sms = sms;
  if (tail.ksplit == 1 && tail.qsplit) {  // the last round's blocks as single query tiles
    a.aux.qsplit = 1;
    a.aux.n_full = tail.n_full;
  }
  if (tail.ksplit > 1) {
    uint8_t* w = static_cast<uint8_t*>(ws);
    a.aux.lin = 1;
    a.aux.n_full = tail.n_full;
    a.aux.ksplit = tail.ksplit;
    a.aux.kchunk = tail.kchunk;
    a.aux.prow0 = tail.prow0;
    a.aux.u_part = reinterpret_cast<float*>(w);
    a.aux.m_part = reinterpret_cast<float*>(w + tail.u_bytes);
    a.aux.l_part = reinterpret_cast<float*>(w + tail.u_bytes + tail.m_bytes);
  }
  cudaGetLastError();  // clear a stale, non-sticky error so that it is not blamed on this launch
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fattn::launch_fwd(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "fa_fwd launch");
  if (tail.ksplit > 1) {
    uint8_t* o_tail = static_cast<uint8_t*>(o) + static_cast<size_t>(tail.prow0) * d * (o_fp32 ? 4 : 2);
    e = fattn::launch_combine(a.aux.u_part, a.aux.m_part, a.aux.l_part, o_tail, lse + tail.prow0,
                              static_cast<int>(tail.rows), tail.ksplit, d, o_fp32, s);
    if (e != cudaSuccess) return cuda_fail(e, "fa_fwd tail combine launch");
  }
  return FA_OK;
}

size_t fa_fwd_workspace_bytes(int B, int H, int N, int d, int causal) {
  if (B < 1 || H < 1 || N < 1 || (d != 64 && d != 128) || (causal != 0 && causal != 1)) return 0;
  int sms = 0;
  if (check_device(&sms) != FA_OK) return 0;
  return plan_tail(static_cast<long long>(B) * H, N, d, causal, sms).total();
}

fa_status_t fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, int d,
                   float scale, int causal, void* stream) {
  return fa_fwd_ex(q, k, v, o, lse, B, H, N, d, scale, causal, stream, nullptr);
}

fa_status_t fa_fwd_partial_ex(const void* q, const void* k, const void* v, float* u_part, float* m_part,
                              float* l_part, int B, int H, int N, int Nk, int key_offset, int kv_rows, int d,
                              float scale, int causal, int shard, int S, void* stream) {
  g_last_error[0] = '\0';
  if (!q || !k || !v || !u_part || !m_part || !l_part) return fail(FA_ERR_INVALID_ARG, "null tensor pointer");
  if (B < 1 || H < 1 || N < 1 || Nk < 1)
    return fail(FA_ERR_INVALID_ARG, "B, H, N and Nk must be >= 1 (got %d, %d, %d, %d)", B, H, N, Nk);
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dimension d=%d is not supported (64 or 128)", d);
  if (key_offset < 0) return fail(FA_ERR_INVALID_ARG, "key_offset=%d must be >= 0", key_offset);
  if (kv_rows < 0 || (kv_rows > 0 && static_cast<long long>(key_offset) + Nk > kv_rows))
    return fail(FA_ERR_INVALID_ARG, "kv_rows=%d must be 0 or >= key_offset + Nk = %lld", kv_rows,
                static_cast<long long>(key_offset) + Nk);
  if (S < 1 || shard < 0 || shard >= S) return fail(FA_ERR_INVALID_ARG, "shard=%d must be in [0, S=%d)", shard, S);
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (causal != 0 && causal != 1) return fail(FA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(u_part, 16))
    return fail(FA_ERR_INVALID_ARG, "q, k, v and u_part must be 16-byte aligned");
  if (!aligned(m_part, 4) || !aligned(l_part, 4)) return fail(FA_ERR_INVALID_ARG, "m_part, l_part must be 4-byte aligned");
  const long long bh = static_cast<long long>(B) * H;
  if (bh > INT_MAX) return fail(FA_ERR_UNSUPPORTED, "B*H=%lld exceeds the grid limit", bh);
  if ((N + 127) / 128 > 65535) return fail(FA_ERR_UNSUPPORTED, "N=%d exceeds the 65535 query-tile grid limit", N);
  int sms = 0;
  fa_status_t st = check_device(&sms);
  if (st != FA_OK) return st;
  fattn::FwdLaunch a{};
  a.sms = sms;
  if ((st = make_map(&a.tq, q, d, N, bh, 128)) != FA_OK) return st;
  // The shard's own buffers ([B, H, Nk, d]), or the whole key tensors ([B, H, kv_rows, d]) read
  // from row key_offset on.
  const int rows = kv_rows > 0 ? kv_rows : Nk;
  if ((st = make_map(&a.tk, k, d, rows, bh, 128)) != FA_OK) return st;
  if ((st = make_map(&a.tv, v, d, rows, bh, 128)) != FA_OK) return st;
  a.aux.kload0 = kv_rows > 0 ? key_offset : 0;
  a.N = N;
  a.BH = static_cast<int>(bh);
  a.d = d;
  a.causal = causal;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.budget = kDefaultBudget;
  a.aux.Nk = Nk;
  a.aux.koff = key_offset;
  a.aux.u_part = u_part;
  a.aux.m_part = m_part;
  a.aux.l_part = l_part;
  a.aux.shard = shard;
  a.aux.S = S;
  cudaGetLastError();
  cudaError_t e = fattn::launch_fwd(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_fwd_partial launch");
  return FA_OK;
}

fa_status_t fa_fwd_partial(const void* q, const void* k, const void* v, float* u_part, float* m_part,
                           float* l_part, int B, int H, int N, int Nk, int key_offset, int d, float scale, int causal,
                           int shard, int S, void* stream) {
  return fa_fwd_partial_ex(q, k, v, u_part, m_part, l_part, B, H, N, Nk, key_offset, 0, d, scale, causal, shard, S,
                           stream);
}

fa_status_t fa_quantize_e4m3(const void* x, void* codes, float* scales, int B, int H, int N, int d, void* stream) {
  g_last_error[0] = '\0';
  if (!x || !codes || !scales) return fail(FA_ERR_INVALID_ARG, "null tensor pointer");
  if (B < 1 || H < 1 || N < 1) return fail(FA_ERR_INVALID_ARG, "B, H and N must be >= 1 (got %d, %d, %d)", B, H, N);
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dimension d=%d is not supported (64 or 128)", d);
  if (!aligned(x, 16) || !aligned(codes, 16)) return fail(FA_ERR_INVALID_ARG, "x and codes must be 16-byte aligned");
  if (!aligned(scales, 4)) return fail(FA_ERR_INVALID_ARG, "scales must be 4-byte aligned");
  const long long grid = static_cast<long long>(B) * H * ((N + 127) / 128);
  if (grid > INT_MAX) return fail(FA_ERR_UNSUPPORTED, "B*H*ceil(N/128)=%lld exceeds the grid limit", grid);
  fa_status_t st = check_device(nullptr);
  if (st != FA_OK) return st;
  cudaGetLastError();
  cudaError_t e = fattn::launch_quant_e4m3(x, codes, scales, B * H, N, d, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_quantize_e4m3 launch");
  return FA_OK;
}

fa_status_t fa_fwd_fp8(const void* q8, const void* k8, const void* v8, const float* sq, const float* sk,
                       const float* sv, void* o, float* lse, int B, int H, int N, int d, float scale, int causal,
                       void* stream, const fa_fwd_opts* opts) {
  g_last_error[0] = '\0';
  if (!q8 || !k8 || !v8 || !sq || !sk || !sv || !o || !lse) return fail(FA_ERR_INVALID_ARG, "null tensor pointer");
  if (B < 1 || H < 1 || N < 1) return fail(FA_ERR_INVALID_ARG, "B, H and N must be >= 1 (got %d, %d, %d)", B, H, N);
  if (d != 128) return fail(FA_ERR_UNSUPPORTED, "the FP8 forward supports d=128 only (got d=%d)", d);
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (causal != 0 && causal != 1) return fail(FA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!aligned(q8, 16) || !aligned(k8, 16) || !aligned(v8, 16) || !aligned(o, 16))
    return fail(FA_ERR_INVALID_ARG, "q8, k8, v8 and o must be 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(sq, 4) || !aligned(sk, 4) || !aligned(sv, 4))
    return fail(FA_ERR_INVALID_ARG, "lse and the scale arrays must be 4-byte aligned");
  const int o_fp32 = opts ? opts->o_fp32 : 0;
  if (o_fp32 != 0 && o_fp32 != 1) return fail(FA_ERR_INVALID_ARG, "opts->o_fp32 must be 0 or 1");
  const long long bh = static_cast<long long>(B) * H;
  if (bh > INT_MAX) return fail(FA_ERR_UNSUPPORTED, "B*H=%lld exceeds the grid limit", bh);
  if ((N + 127) / 128 > 65535) return fail(FA_ERR_UNSUPPORTED, "N=%d exceeds the 65535 query-tile grid limit", N);
  int sms = 0;
  fa_status_t st = check_device(&sms);
  if (st != FA_OK) return st;

  fattn::FwdLaunch a{};
  a.sms = sms;
  if ((st = make_map(&a.tq, q8, d, N, bh, 128, 1)) != FA_OK) return st;
  if ((st = make_map(&a.tk, k8, d, N, bh, 128, 1)) != FA_OK) return st;
  if ((st = make_map(&a.tv, v8, d, N, bh, 128, 1)) != FA_OK) return st;
  if (!o_fp32 && (st = make_map(&a.to, o, d, N, bh, 128)) != FA_OK) return st;
  a.o = o;
  a.lse = lse;
  a.N = N;
  a.BH = static_cast<int>(bh);
  a.d = d;
  a.causal = causal;
  a.o_fp32 = o_fp32;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.budget = (opts && opts->wait_budget_cycles) ? opts->wait_budget_cycles : kDefaultBudget;
  a.fp8 = 1;
  a.aux.sq = sq;
  a.aux.sk = sk;
  a.aux.sv = sv;
  a.aux.Nk = N;
  cudaGetLastError();
  cudaError_t e = fattn::launch_fwd(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_fwd_fp8 launch");
  return FA_OK;
}

size_t fa_decode_workspace_bytes(int B, int H, int L, int d, int chunk, int splits) {
  int sms = 0;
  if (splits == 0) {
    if (check_device(&sms) != FA_OK) return 0;
  }
  DecodePlan plan;
  if (plan_decode(B, H, L, d, chunk, splits, sms, &plan) != FA_OK) return 0;
  return plan.total();
}

fa_status_t fa_decode_splitkv_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                                 int L, int d, float scale, int chunk, int splits, void* workspace, size_t ws_bytes,
                                 void* stream, const fa_decode_opts* opts) {
  g_last_error[0] = '\0';
  if (!q || !k || !v || !o || !lse) return fail(FA_ERR_INVALID_ARG, "null tensor pointer");
  const int o_fp32 = opts ? opts->o_fp32 : 0;
  if (o_fp32 != 0 && o_fp32 != 1) return fail(FA_ERR_INVALID_ARG, "opts->o_fp32 must be 0 or 1");
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16))
    return fail(FA_ERR_INVALID_ARG, "q, k, v and o must be 16-byte aligned");
  if (!aligned(lse, 4)) return fail(FA_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  if (workspace && !aligned(workspace, 256)) return fail(FA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  DecodePlan plan;
  fa_status_t st;
  if (splits != 0) {
    if ((st = plan_decode(B, H, L, d, chunk, splits, 0, &plan)) != FA_OK) return st;
    if (!workspace || ws_bytes < plan.total())
      return fail(FA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", ws_bytes,
                  plan.total());
    if ((st = check_device(nullptr)) != FA_OK) return st;
  } else {
    int sms = 0;
    if ((st = plan_decode(B, H, L, d, chunk, 1, 0, &plan)) != FA_OK) return st;  // argument checks first
    if ((st = check_device(&sms)) != FA_OK) return st;
    if ((st = plan_decode(B, H, L, d, chunk, 0, sms, &plan)) != FA_OK) return st;
  }
  if (!workspace || ws_bytes < plan.total())
    return fail(FA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", ws_bytes,
                plan.total());
  const long long bh = static_cast<long long>(B) * H;
  fattn::DecodeLaunch a{};
  if ((st = make_map(&a.tk, k, d, L, bh, fattn::kDecodeStageKeys)) != FA_OK) return st;
  if ((st = make_map(&a.tv, v, d, L, bh, fattn::kDecodeStageKeys)) != FA_OK) return st;
  char* ws = static_cast<char*>(workspace);
  a.q = q;
  a.u_part = reinterpret_cast<float*>(ws);
  a.m_part = reinterpret_cast<float*>(ws + plan.u_bytes);
  a.l_part = reinterpret_cast<float*>(ws + plan.u_bytes + plan.m_bytes);
  a.o = o;
  a.lse = lse;
  a.L = L;
  a.BH = static_cast<int>(bh);
  a.d = d;
  a.splits = plan.splits;
  a.keys_per_split = plan.keys_per_split;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.budget = (opts && opts->wait_budget_cycles) ? opts->wait_budget_cycles : kDefaultBudget;
  cudaGetLastError();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fattn::launch_decode_split(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "fa_decode_splitkv split launch");
  e = fattn::launch_combine(a.u_part, a.m_part, a.l_part, o, lse, a.BH, a.splits, d, o_fp32, s);
  if (e != cudaSuccess) return cuda_fail(e, "fa_decode_splitkv combine launch");
  return FA_OK;
}

fa_status_t fa_decode_splitkv(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int L,
                              int d, float scale, int chunk, int splits, void* workspace, size_t ws_bytes,
                              void* stream) {
  return fa_decode_splitkv_ex(q, k, v, o, lse, B, H, L, d, scale, chunk, splits, workspace, ws_bytes, stream,
                              nullptr);
}

fa_status_t fa_decode_splitkv_noalloc(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                                      int L, int d, float scale, int chunk, int splits, void* stream) {
  g_last_error[0] = '\0';
  // Size the partials exactly as fa_decode_splitkv would, and refuse what the
  // fixed scratch cannot hold (argument errors are reported as such first).
  DecodePlan plan;
  fa_status_t st;
  if (splits != 0) {
    if ((st = plan_decode(B, H, L, d, chunk, splits, 0, &plan)) != FA_OK) return st;
  } else {
    int sms = 0;
    if ((st = plan_decode(B, H, L, d, chunk, 1, 0, &plan)) != FA_OK) return st;
    if ((st = check_device(&sms)) != FA_OK) return st;
    if ((st = plan_decode(B, H, L, d, chunk, 0, sms, &plan)) != FA_OK) return st;
  }
  if (splits == 0 && plan.total() > fattn::kNoAllocScratchBytes) {
    // The automatic plan does not fit: take the largest smaller split count (that leaves no split
    // empty) whose partials fit.
    const int n_chunks = (L + chunk - 1) / chunk;
    for (int s = plan.splits - 1; s >= 1; --s) {
      const int cps = (n_chunks + s - 1) / s;
      if ((n_chunks + cps - 1) / cps != s) continue;
      DecodePlan p2;
      if ((st = plan_decode(B, H, L, d, chunk, s, 0, &p2)) != FA_OK) return st;
      if (p2.total() <= fattn::kNoAllocScratchBytes) {
        plan = p2;
        break;
      }
    }
  }
  if (plan.total() > fattn::kNoAllocScratchBytes)
    return fail(FA_ERR_WORKSPACE,
                "fa_decode_splitkv_noalloc: B=%d H=%d with %d splits needs %zu bytes of partials, more than its "
                "fixed scratch of %zu bytes; use fewer splits or fa_decode_splitkv with a workspace",
                B, H, plan.splits, plan.total(), fattn::kNoAllocScratchBytes);
  if ((st = check_device(nullptr)) != FA_OK) return st;
  void* scratch = nullptr;
  cudaError_t e = fattn::decode_noalloc_scratch(&scratch);
  if (e != cudaSuccess) return cuda_fail(e, "fa_decode_splitkv_noalloc scratch address");
  return fa_decode_splitkv(q, k, v, o, lse, B, H, L, d, scale, chunk, plan.splits, scratch,
                           fattn::kNoAllocScratchBytes, stream);
}


size_t fa_decode_paged_workspace_bytes(int B, int H, int max_seq_len, int d, int page_size, int max_pages,
                                       int splits) {
  const int saved = g_last_error[0];
  DecodePlan plan;
  fa_status_t st = check_paged_args(B, H, d, page_size, max_pages, 1, max_seq_len);
  int sms = 0;
  if (st == FA_OK && splits == 0) st = check_device(&sms);
  if (st == FA_OK) st = plan_paged(B, H, max_seq_len, d, page_size, splits, sms, &plan);
  if (!saved) g_last_error[0] = '\0';
  return st == FA_OK ? plan.total() : 0;
}

fa_status_t fa_decode_paged_ex(const void* q, const void* k_pages, const void* v_pages, const int* block_table,
                               const int* seq_lens, void* o, float* lse, int B, int H, int d, int page_size,
                               int max_pages, int num_pages, int max_seq_len, float scale, int splits,
                               void* workspace, size_t ws_bytes, void* stream, const fa_decode_opts* opts) {
  g_last_error[0] = '\0';
  if (!q || !k_pages || !v_pages || !block_table || !seq_lens || !o || !lse)
    return fail(FA_ERR_INVALID_ARG, "null tensor pointer");
  const int o_fp32 = opts ? opts->o_fp32 : 0;
  if (o_fp32 != 0 && o_fp32 != 1) return fail(FA_ERR_INVALID_ARG, "opts->o_fp32 must be 0 or 1");
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(o, 16))
    return fail(FA_ERR_INVALID_ARG, "q, k_pages, v_pages and o must be 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return fail(FA_ERR_INVALID_ARG, "lse, block_table and seq_lens must be 4-byte aligned");
  if (workspace && !aligned(workspace, 256)) return fail(FA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  fa_status_t st = check_paged_args(B, H, d, page_size, max_pages, num_pages, max_seq_len);
  if (st != FA_OK) return st;
  if (splits < 0) return fail(FA_ERR_INVALID_ARG, "splits=%d must be >= 0", splits);
  DecodePlan plan;
  int sms = 0;
  if (splits != 0) {
    if ((st = plan_paged(B, H, max_seq_len, d, page_size, splits, 0, &plan)) != FA_OK) return st;
    if (!workspace || ws_bytes < plan.total())
      return fail(FA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", ws_bytes,
                  plan.total());
    if ((st = check_device(nullptr)) != FA_OK) return st;
  } else {
    if ((st = check_device(&sms)) != FA_OK) return st;
    if ((st = plan_paged(B, H, max_seq_len, d, page_size, 0, sms, &plan)) != FA_OK) return st;
  }
  if (!workspace || ws_bytes < plan.total())
    return fail(FA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", ws_bytes,
                plan.total());
  const long long bh = static_cast<long long>(B) * H;
  fattn::DecodeLaunch a{};
  const long long planes = static_cast<long long>(num_pages) * H;
  if ((st = make_map(&a.tk, k_pages, d, page_size, planes, fattn::kDecodeStageKeys)) != FA_OK) return st;
  if ((st = make_map(&a.tv, v_pages, d, page_size, planes, fattn::kDecodeStageKeys)) != FA_OK) return st;
  char* ws = static_cast<char*>(workspace);
  a.q = q;
  a.u_part = reinterpret_cast<float*>(ws);
  a.m_part = reinterpret_cast<float*>(ws + plan.u_bytes);
  a.l_part = reinterpret_cast<float*>(ws + plan.u_bytes + plan.m_bytes);
  a.o = o;
  a.lse = lse;
  a.L = max_seq_len;
  a.BH = static_cast<int>(bh);
  a.d = d;
  a.splits = plan.splits;
  a.keys_per_split = plan.keys_per_split;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.budget = (opts && opts->wait_budget_cycles) ? opts->wait_budget_cycles : kDefaultBudget;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.H = H;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  cudaGetLastError();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fattn::launch_decode_split(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "fa_decode_paged split launch");
  e = fattn::launch_combine(a.u_part, a.m_part, a.l_part, o, lse, a.BH, a.splits, d, o_fp32, s);
  if (e != cudaSuccess) return cuda_fail(e, "fa_decode_paged combine launch");
  return FA_OK;
}

fa_status_t fa_decode_paged(const void* q, const void* k_pages, const void* v_pages, const int* block_table,
                            const int* seq_lens, void* o, float* lse, int B, int H, int d, int page_size,
                            int max_pages, int num_pages, int max_seq_len, float scale, int splits, void* workspace,
                            size_t ws_bytes, void* stream) {
  return fa_decode_paged_ex(q, k_pages, v_pages, block_table, seq_lens, o, lse, B, H, d, page_size, max_pages,
                            num_pages, max_seq_len, scale, splits, workspace, ws_bytes, stream, nullptr);
}

fa_status_t fa_combine_ex(const float* u_part, const float* m_part, const float* l_part, void* o, float* lse, int R,
                          int S, int d, int o_fp32, void* stream) {
  g_last_error[0] = '\0';
  if (!u_part || !m_part || !l_part || !o || !lse) return fail(FA_ERR_INVALID_ARG, "null tensor pointer");
  if (o_fp32 != 0 && o_fp32 != 1) return fail(FA_ERR_INVALID_ARG, "o_fp32 must be 0 or 1");
  if (R < 1 || S < 1) return fail(FA_ERR_INVALID_ARG, "R and S must be >= 1 (got %d, %d)", R, S);
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dimension d=%d is not supported (64 or 128)", d);
  if (!aligned(u_part, 16) || !aligned(o, 16)) return fail(FA_ERR_INVALID_ARG, "u_part and o must be 16-byte aligned");
  if (!aligned(m_part, 4) || !aligned(l_part, 4) || !aligned(lse, 4))
    return fail(FA_ERR_INVALID_ARG, "m_part, l_part and lse must be 4-byte aligned");
  fa_status_t st = check_device(nullptr);
  if (st != FA_OK) return st;
  cudaGetLastError();
  cudaError_t e =
      fattn::launch_combine(u_part, m_part, l_part, o, lse, R, S, d, o_fp32, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_combine launch");
  return FA_OK;
}

fa_status_t fa_combine(const float* u_part, const float* m_part, const float* l_part, void* o, float* lse, int R,
                       int S, int d, void* stream) {
  return fa_combine_ex(u_part, m_part, l_part, o, lse, R, S, d, 0, stream);
}

size_t fa_bwd_workspace_bytes(int B, int H, int N) {
  if (B < 1 || H < 1 || N < 1) return 0;
  return round256(static_cast<size_t>(B) * H * N * sizeof(float));
}

fa_status_t fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                   void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale, int causal, int grad_fp32,
                   void* workspace, size_t ws_bytes, void* stream) {
  return fa_bwd_ex(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, grad_fp32, workspace, ws_bytes,
                   stream, nullptr);
}

fa_status_t fa_bwd_ex(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                      void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale, int causal, int grad_fp32,
                      void* workspace, size_t ws_bytes, void* stream, const fa_bwd_opts* opts) {
  g_last_error[0] = '\0';
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv) return fail(FA_ERR_INVALID_ARG, "null tensor pointer");
  if (B < 1 || H < 1 || N < 1) return fail(FA_ERR_INVALID_ARG, "B, H and N must be >= 1 (got %d, %d, %d)", B, H, N);
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dimension d=%d is not supported (64 or 128)", d);
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (causal != 0 && causal != 1) return fail(FA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (grad_fp32 != 0 && grad_fp32 != 1) return fail(FA_ERR_INVALID_ARG, "grad_fp32 must be 0 or 1");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(dout, 16) ||
      !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16))
    return fail(FA_ERR_INVALID_ARG, "q, k, v, o, dout, dq, dk and dv must be 16-byte aligned");
  if (!aligned(lse, 4)) return fail(FA_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  const long long bh = static_cast<long long>(B) * H;
  if (bh > INT_MAX) return fail(FA_ERR_UNSUPPORTED, "B*H=%lld exceeds the grid limit", bh);
  if ((N + 127) / 128 > 65535) return fail(FA_ERR_UNSUPPORTED, "N=%d exceeds the 65535 tile grid limit", N);
  const size_t need = fa_bwd_workspace_bytes(B, H, N);
  if (!workspace || ws_bytes < need)
    return fail(FA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", ws_bytes, need);
  if (!aligned(workspace, 256)) return fail(FA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  int sms = 0;
  fa_status_t st = check_device(&sms);
  if (st != FA_OK) return st;
  fattn::BwdLaunch a{};
  a.sms = sms;
  if ((st = make_map(&a.tq, q, d, N, bh, 128)) != FA_OK) return st;
  if ((st = make_map(&a.tk, k, d, N, bh, 128)) != FA_OK) return st;
  if ((st = make_map(&a.tv, v, d, N, bh, 128)) != FA_OK) return st;
  if ((st = make_map(&a.tdo, dout, d, N, bh, 128)) != FA_OK) return st;
  if (!grad_fp32) {
    if ((st = make_map(&a.tdq, dq, d, N, bh, 128)) != FA_OK) return st;
    if ((st = make_map(&a.tdk, dk, d, N, bh, 128)) != FA_OK) return st;
    if ((st = make_map(&a.tdv, dv, d, N, bh, 128)) != FA_OK) return st;
  }
  a.o = o;
  a.dout = dout;
  a.lse = lse;
  a.delta = static_cast<float*>(workspace);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.N = N;
  a.BH = static_cast<int>(bh);
  a.d = d;
  a.causal = causal;
  a.grad_fp32 = grad_fp32;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.budget = (opts && opts->wait_budget_cycles) ? opts->wait_budget_cycles : kDefaultBudget;
  cudaGetLastError();
  cudaError_t e = fattn::launch_bwd(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_bwd launch");
  return FA_OK;
}

size_t fa_cross_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  const int saved = g_last_error[0];
  CrossShape c;
  int sms = 0;
  fa_status_t st = check_cross_args(B, Hq, Hkv, Nq, Nk, d, &c);
  if (st == FA_OK) st = check_device(&sms);
  if (!saved) g_last_error[0] = '\0';
  return st == FA_OK ? plan_cross(c, Nk, d, sms, true).total() : 0;
}

fa_status_t fa_cross_fwd(const void* q, const void* k, const void* v, const int* kv_lens, void* o, float* lse, int B,
                         int Hq, int Hkv, int Nq, int Nk, int d, float scale, void* workspace, size_t ws_bytes,
                         void* stream, const fa_cross_opts* opts) {
  g_last_error[0] = '\0';
  if (!q || !k || !v || !o || !lse) return fail(FA_ERR_INVALID_ARG, "null tensor pointer");
  const int o_fp32 = opts ? opts->o_fp32 : 0;
  if (o_fp32 != 0 && o_fp32 != 1) return fail(FA_ERR_INVALID_ARG, "opts->o_fp32 must be 0 or 1");
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16))
    return fail(FA_ERR_INVALID_ARG, "q, k, v and o must be 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(kv_lens, 4)) return fail(FA_ERR_INVALID_ARG, "lse and kv_lens must be 4-byte aligned");
  if (workspace && !aligned(workspace, 256)) return fail(FA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  CrossShape c;
  fa_status_t st = check_cross_args(B, Hq, Hkv, Nq, Nk, d, &c);
  if (st != FA_OK) return st;
  int sms = 0;
  if ((st = check_device(&sms)) != FA_OK) return st;
  const CrossPlan plan = plan_cross(c, Nk, d, sms, workspace != nullptr);
  if (workspace && ws_bytes < plan.total())
    return fail(FA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes fa_cross_workspace_bytes gives",
                ws_bytes, plan.total());
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  float* u_part = plan.parts ? reinterpret_cast<float*>(w) : nullptr;
  float* m_part = plan.parts ? reinterpret_cast<float*>(w + plan.u_bytes) : nullptr;
  float* l_part = plan.parts ? reinterpret_cast<float*>(w + plan.u_bytes + plan.m_bytes) : nullptr;
  const float scale_log2 = scale * 1.4426950408889634f;
  const unsigned long long budget = (opts && opts->wait_budget_cycles) ? opts->wait_budget_cycles : kDefaultBudget;
  auto join = [&]() -> fa_status_t {
    if (!plan.parts) return FA_OK;
    const cudaError_t e = fattn::launch_combine(u_part, m_part, l_part, o, lse, static_cast<int>(c.bh * c.rows),
                                                plan.splits, d, o_fp32, s);
    return e == cudaSuccess ? FA_OK : cuda_fail(e, "fa_cross_fwd combine launch");
  };
  if (plan.few) {
    fattn::CrossRowsLaunch f{};
    if ((st = make_map(&f.tk, k, d, Nk, c.bh, fattn::kRowsStageKeys)) != FA_OK) return st;
    if ((st = make_map(&f.tv, v, d, Nk, c.bh, fattn::kRowsStageKeys)) != FA_OK) return st;
    f.BH = static_cast<int>(c.bh);
    f.d = d;
    f.args = {q, o, lse, u_part, m_part, l_part, kv_lens, Hkv, c.rows, Nk, plan.splits, o_fp32, scale_log2, budget};
    cudaGetLastError();
    const cudaError_t e = fattn::launch_cross_rows(f, s);
    if (e != cudaSuccess) return cuda_fail(e, "fa_cross_fwd launch");
    return join();
  }
  if (plan.tiles > 0) {
    fattn::CrossShortLaunch f{};
    if ((st = make_map(&f.tq, q, d, c.rows, c.bh, 128)) != FA_OK) return st;
    if ((st = make_map(&f.tk, k, d, Nk, c.bh, 128)) != FA_OK) return st;
    if ((st = make_map(&f.tv, v, d, Nk, c.bh, 128)) != FA_OK) return st;
    if (!o_fp32 && (st = make_map(&f.to, o, d, c.rows, c.bh, 128)) != FA_OK) return st;
    f.BH = static_cast<int>(c.bh);
    f.d = d;
    f.args = {o, lse, kv_lens, Hkv, c.rows, Nk, plan.tiles, o_fp32, scale_log2, budget};
    cudaGetLastError();
    const cudaError_t e = fattn::launch_cross_short(f, s);
    if (e != cudaSuccess) return cuda_fail(e, "fa_cross_fwd launch");
    return FA_OK;
  }
  fattn::FwdLaunch a{};
  if ((st = make_map(&a.tq, q, d, c.rows, c.bh, 128)) != FA_OK) return st;
  if ((st = make_map(&a.tk, k, d, Nk, c.bh, 128)) != FA_OK) return st;
  if ((st = make_map(&a.tv, v, d, Nk, c.bh, 128)) != FA_OK) return st;
  if (!o_fp32 && (st = make_map(&a.to, o, d, c.rows, c.bh, 128)) != FA_OK) return st;
  a.o = o;
  a.lse = lse;
  a.N = c.rows;
  a.BH = static_cast<int>(c.bh);
  a.d = d;
  a.o_fp32 = o_fp32;
  a.scale_log2 = scale_log2;
  a.budget = budget;
  a.sms = sms;
  a.cross = 1;
  a.aux.Nk = Nk;
  a.aux.kv_lens = kv_lens;
  a.aux.kv_heads = Hkv;
  a.aux.kchunk = plan.kchunk;
  a.aux.S = plan.splits;
  if (d == 64 && plan.splits == 1) {
    // The persistent kernel's last round, when at most half full, as single query tiles (as fa_fwd_ex).
    const long long units = c.bh * ((c.rows + 255) / 256), rem = units % sms;
    if (rem > 0 && 2 * rem <= sms && units + rem <= INT_MAX) {
      a.aux.qsplit = 1;
      a.aux.n_full = static_cast<int>(units - rem);
    }
  }
  a.aux.u_part = u_part;
  a.aux.m_part = m_part;
  a.aux.l_part = l_part;
  cudaGetLastError();
  cudaError_t e = fattn::launch_fwd(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "fa_cross_fwd launch");
  return join();
}

size_t fa_cross_bwd_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  const int saved = g_last_error[0];
  CrossShape c;
  int sms = 0;
  fa_status_t st = check_cross_args(B, Hq, Hkv, Nq, Nk, d, &c);
  if (st == FA_OK) st = check_device(&sms);
  if (!saved) g_last_error[0] = '\0';
  return st == FA_OK ? plan_cross_bwd(c, Nk, d, sms).total() : 0;
}

fa_status_t fa_cross_bwd(const void* q, const void* k, const void* v, const int* kv_lens, const void* o,
                         const void* dout, const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv,
                         int Nq, int Nk, int d, float scale, int grad_fp32, void* workspace, size_t ws_bytes,
                         void* stream, const fa_bwd_opts* opts) {
  g_last_error[0] = '\0';
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv) return fail(FA_ERR_INVALID_ARG, "null tensor pointer");
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(FA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (grad_fp32 != 0 && grad_fp32 != 1) return fail(FA_ERR_INVALID_ARG, "grad_fp32 must be 0 or 1");
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(dout, 16) ||
      !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16))
    return fail(FA_ERR_INVALID_ARG, "q, k, v, o, dout, dq, dk and dv must be 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(kv_lens, 4)) return fail(FA_ERR_INVALID_ARG, "lse and kv_lens must be 4-byte aligned");
  CrossShape c;
  fa_status_t st = check_cross_args(B, Hq, Hkv, Nq, Nk, d, &c);
  if (st != FA_OK) return st;
  if (!workspace) return fail(FA_ERR_WORKSPACE, "fa_cross_bwd needs a workspace (fa_cross_bwd_workspace_bytes)");
  if (!aligned(workspace, 256)) return fail(FA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  int sms = 0;
  if ((st = check_device(&sms)) != FA_OK) return st;
  const CrossBwdPlan plan = plan_cross_bwd(c, Nk, d, sms);
  if (ws_bytes < plan.total())
    return fail(FA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", ws_bytes, plan.total());
  fattn::BwdLaunch a{};
  a.sms = sms;
  if ((st = make_map(&a.tq, q, d, c.rows, c.bh, 128)) != FA_OK) return st;
  const int key_box = Nk <= 64 ? 64 : 128;
  if ((st = make_map(&a.tk, k, d, Nk, c.bh, key_box)) != FA_OK) return st;
  if ((st = make_map(&a.tv, v, d, Nk, c.bh, key_box)) != FA_OK) return st;
  if ((st = make_map(&a.tdo, dout, d, c.rows, c.bh, 128)) != FA_OK) return st;
  if (!grad_fp32) {
    if ((st = make_map(&a.tdq, dq, d, c.rows, c.bh, 128)) != FA_OK) return st;
    if ((st = make_map(&a.tdk, dk, d, Nk, c.bh, 128)) != FA_OK) return st;
    if ((st = make_map(&a.tdv, dv, d, Nk, c.bh, 128)) != FA_OK) return st;
  }
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.o = o;
  a.dout = dout;
  a.lse = lse;
  a.delta = reinterpret_cast<float*>(w);
  a.kv_part = reinterpret_cast<float*>(w + plan.delta_bytes);
  a.q_part = reinterpret_cast<float*>(w + plan.delta_bytes + plan.kv_bytes);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.N = c.rows;
  a.BH = static_cast<int>(c.bh);
  a.d = d;
  a.grad_fp32 = grad_fp32;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.budget = (opts && opts->wait_budget_cycles) ? opts->wait_budget_cycles : kDefaultBudget;
  a.Nk = Nk;
  a.kv_lens = kv_lens;
  a.kv_heads = Hkv;
  a.q_tiles = plan.q_tiles;
  a.kv_splits = plan.kv_splits;
  a.k_tiles = plan.k_tiles;
  a.q_splits = plan.q_splits;
  const bool short_keys = Nk <= fattn::kCrossShortKeys;
  if (!short_keys)
    a.own_tiles = dq_own_tiles(plan, c.bh, (c.rows + 127) / 128, (Nk + 127) / 128, d, sms, kv_lens != nullptr);
  cudaGetLastError();
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = short_keys ? fattn::launch_cross_bwd_short(a, s) : fattn::launch_cross_bwd(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "fa_cross_bwd launch");
  return FA_OK;
}

fa_status_t fa_rope_axes_plan(fa_rope_axes_plan_t* plan, int d, int n_axes, const int* sections, double base,
                              int interleaved, int per_axis, int cyclic) {
  g_last_error[0] = '\0';
  if (!plan || !sections) return fail(FA_ERR_INVALID_ARG, "null plan or sections");
  if (d != 64 && d != 128) return fail(FA_ERR_UNSUPPORTED, "head dimension d=%d is not supported (64 or 128)", d);
  if (n_axes < 1 || n_axes > FA_ROPE_MAX_AXES)
    return fail(FA_ERR_INVALID_ARG, "n_axes=%d must be in [1, %d]", n_axes, FA_ROPE_MAX_AXES);
  if (!std::isfinite(base) || !(base >= 1.0)) return fail(FA_ERR_INVALID_ARG, "base must be finite and >= 1");
  if ((interleaved | per_axis | cyclic) & ~1)
    return fail(FA_ERR_INVALID_ARG, "interleaved, per_axis and cyclic must be 0 or 1");
  long long sum = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (sections[a] < 1) return fail(FA_ERR_INVALID_ARG, "sections[%d]=%d must be >= 1", a, sections[a]);
    sum += sections[a];
  }
  const int n = d / 2;
  if (sum != n) return fail(FA_ERR_INVALID_ARG, "sections sum to %lld pairs, expected d/2 = %d", sum, n);
  *plan = fa_rope_axes_plan_t{};
  plan->d = d;
  plan->n_axes = n_axes;
  plan->interleaved = interleaved;
  int used[FA_ROPE_MAX_AXES] = {};
  for (int i = 0, a = 0; i < n; ++i) {
    while (used[a] == sections[a]) a = (a + 1) % n_axes;  // (pairs are left, so some axis has one)
    plan->axis[i] = static_cast<unsigned char>(a);
    const double exponent = per_axis ? static_cast<double>(used[a]) / sections[a] : static_cast<double>(i) / n;
    ++used[a];
    // rate / (2 pi) <= 0.16 turns a position, to the nearest 2^-64 turn
    const double turns = std::pow(base, -exponent) * 0.15915494309189533577;
    plan->turns[i] = static_cast<unsigned long long>(std::rint(std::ldexp(turns, 64)));
    if (cyclic) a = (a + 1) % n_axes;
  }
  return FA_OK;
}

fa_status_t fa_rope_axes(const void* q, const void* k, const int* pos, void* q_out, void* k_out, int B, int Hq, int Hk,
                         int N, const fa_rope_axes_plan_t* plan, int inverse, void* stream) {
  g_last_error[0] = '\0';
  if (!q || !q_out) return fail(FA_ERR_INVALID_ARG, "null tensor pointer");
  fa_status_t st = check_rope_args(plan, pos, B, Hq, Hk, N, inverse);
  if (st != FA_OK) return st;
  if (Hk > 0 && (!k || !k_out)) return fail(FA_ERR_INVALID_ARG, "null tensor pointer");
  if (!aligned(q, 16) || !aligned(q_out, 16) || (Hk > 0 && (!aligned(k, 16) || !aligned(k_out, 16))))
    return fail(FA_ERR_INVALID_ARG, "q, k, q_out and k_out must be 16-byte aligned");
  fattn::RopeLaunch a{};
  if ((st = check_device(&a.sms)) != FA_OK) return st;
  a.plan = *plan;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.pos = pos;
  a.B = B;
  a.Hq = Hq;
  a.Hk = Hk;
  a.N = N;
  a.sign = inverse ? -1.f : 1.f;
  cudaGetLastError();
  cudaError_t e = fattn::launch_rope(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_rope_axes launch");
  return FA_OK;
}

fa_status_t fa_rope_axes_paged(const void* q, const void* k, const void* v, const int* pos, void* q_out, void* k_pages,
                               void* v_pages, const int* block_table, const int* seq_lens, const int* new_lens, int B,
                               int Hq, int Hk, int N, int page_size, int max_pages, int num_pages,
                               const fa_rope_axes_plan_t* plan, void* stream) {
  g_last_error[0] = '\0';
  if (!q || !k || !v || !q_out || !k_pages || !v_pages || !block_table || !seq_lens)
    return fail(FA_ERR_INVALID_ARG, "null tensor pointer");
  fa_status_t st = check_rope_args(plan, pos, B, Hq, Hk, N, 0);
  if (st != FA_OK) return st;
  if ((st = check_paged_args(B, Hk, plan->d, page_size, max_pages, num_pages, 1)) != FA_OK) return st;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_pages, 16) ||
      !aligned(v_pages, 16))
    return fail(FA_ERR_INVALID_ARG, "q, k, v, q_out, k_pages and v_pages must be 16-byte aligned");
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(new_lens, 4))
    return fail(FA_ERR_INVALID_ARG, "block_table, seq_lens and new_lens must be 4-byte aligned");
  fattn::RopeLaunch a{};
  if ((st = check_device(&a.sms)) != FA_OK) return st;
  a.plan = *plan;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_pages);
  a.v_out = static_cast<__nv_bfloat16*>(v_pages);
  a.pos = pos;
  a.B = B;
  a.Hq = Hq;
  a.Hk = Hk;
  a.N = N;
  a.sign = 1.f;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.page_size = page_size;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  cudaGetLastError();
  cudaError_t e = fattn::launch_rope(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_rope_axes_paged launch");
  return FA_OK;
}

fa_status_t fa_get_status(void* stream) {
  g_last_error[0] = '\0';
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fa_get_status synchronize");
  unsigned int bits = 0;
  e = take_status(static_cast<cudaStream_t>(stream), &bits);
  if (e != cudaSuccess) return cuda_fail(e, "fa_get_status");
  if (bits & fattn::kStatusTimeout) return fail(FA_ERR_TIMEOUT, "a kernel wait exceeded its budget");
  return FA_OK;
}

}  // extern "C"
