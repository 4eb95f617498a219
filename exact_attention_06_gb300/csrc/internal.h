// Internal interface between the C-ABI host code and the kernel translation
// units.  Not installed; callers use include/fattn.h.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "fattn.h"

namespace fattn {

// Bits of the status words (one per device and kernel file) that kernels raise.
constexpr unsigned int kStatusTimeout = 1u;
// Default per-wait budget in SM cycles (about 2 s), and the least any drain of in-flight copies
// and MMAs gets before a CTA releases its shared memory and TMEM.
constexpr unsigned long long kDefaultBudget = 4000000000ull;
constexpr unsigned long long kDrainBudget = kDefaultBudget;

// Forward (prefill) launch description.  The tensor maps describe q, k, v as
// 3-D tensors {d, N, B*H} (innermost first) with 64 x 128 boxes and 128-byte
// swizzle.
// Per-launch extras of the forward kernel, passed by value.
struct FwdAux {
  const float* sq;  // FP8: block scales [BH, ceil(N/128)] of q, k, v
  const float* sk;
  const float* sv;
  int Nk;           // keys of this launch (= N unless a key shard)
  int koff;         // global index of key 0 (causal masking of a key shard)
  int kload0;       // row of the k, v tensors (as mapped) that holds key 0 of this launch
  float* u_part;    // key shard: partials [BH*N, S, d], [BH*N, S], [BH*N, S]; null = write O, lse
  float* m_part;
  float* l_part;
  int shard, S;
  // Key split of the last round (lin = 1; work items over 256-row query blocks in (b*h, block)
  // order): items [0, n_full) are whole blocks writing O and lse; each later block is split
  // into ksplit key pieces of kchunk keys (items n_full + ksplit*(block - n_full) + piece),
  // and piece s of flat row r (= b*h*N + n) writes partial slot (r - prow0) * ksplit + s.
  int lin;
  int n_full;
  int ksplit;
  int kchunk;
  long long prow0;
  // Query split (persistent kernel, lin = 0): the blocks from n_full on run as two single-tile
  // items each (items n_full + 2*(block - n_full) + tile).
  int qsplit;
  // Persistent CTAs (non-causal bf16 d = 64): the number of work items; set by launch_fwd.
  int n_items;
  // Cross attention (fa_cross_fwd): rows of a key head are its query heads' rows, one after
  // another; Nk above is the tensors' key count, the sequence of key head bh has kv_lens[bh /
  // kv_heads] of them (null: all).  blockIdx.z takes the keys z * kchunk .. + kchunk - 1 and, with
  // u_part, partial slot z of S.
  const int* kv_lens;
  int kv_heads;
  // One-block-per-CTA kernel: the heads are dispatched in ng groups (each group's blocks
  // longest first) so that the blocks of a head run close together in time; set by launch_fwd.
  int ng;
};

// Number of head groups for a grid (B*H, P) whose CTAs are ordered by grouped_block.  Causal:
// every group needs enough heads that its work, spread over the SMs, outlasts its longest block
// (about 2P tile steps against P^2 + P per head), or that block runs alone at the end of the
// launch: at least 2 * sms / (P + 1) heads per group.  Non-causal blocks are all alike: about one
// wave of CTAs per group.  Groups of near-equal size, so that no small group is left over.
inline int head_groups(int bh, int n_ranks, bool causal, int sms) {
  if (sms < 1 || n_ranks < 1 || bh < 1) return 1;
  long long min_heads = causal ? (2LL * sms + n_ranks) / (n_ranks + 1) : (sms + n_ranks - 1) / n_ranks;
  if (min_heads < 1) min_heads = 1;
  const long long ng = bh / min_heads;
  return static_cast<int>(ng < 1 ? 1 : ng);
}

struct FwdLaunch {
  CUtensorMap tq, tk, tv;
  CUtensorMap to;  // bf16 O as {d, N, B*H} (persistent kernel's TMA store; unused for fp32 O and partials)
  void* o;
  float* lse;
  int N;
  int BH;
  int d;
  int causal;
  int o_fp32;
  float scale_log2;  // scale * log2(e)
  unsigned long long budget;
  int fp8;            // 1: q, k, v are E4M3 with per-128-row block scales in aux (d = 128)
  int sms;            // SMs of the device: the persistent grid size (0: one CTA per work item)
  int cross;          // 1: cross attention (aux.kv_lens, aux.kv_heads, aux.kchunk, aux.S splits)
  FwdAux aux;
};
cudaError_t launch_fwd(const FwdLaunch& a, cudaStream_t stream);
// The current device's address of the word in which the kernels of fa_fwd.cu raise status bits; likewise below.
cudaError_t fwd_status_word(unsigned int** p);

// Split-KV decode launch description.  The tensor maps describe k, v as 3-D
// tensors {d, L, B*H} with 64 x kDecodeStageKeys boxes and 128-byte swizzle.
struct DecodeLaunch {
  CUtensorMap tk, tv;
  const void* q;
  float* u_part;  // [BH, splits, d]
  float* m_part;  // [BH, splits]
  float* l_part;  // [BH, splits]
  void* o;        // [BH, d] bf16
  float* lse;     // [BH]
  int L;
  int BH;
  int d;
  int splits;
  int keys_per_split;  // multiple of 128
  float scale_log2;
  unsigned long long budget;
  // paged KV cache (block_table != nullptr): tk/tv map pools [P * H, page_size, d]
  const int* block_table;  // [B, max_pages]
  const int* seq_lens;     // [B]; L above is the longest length planned for
  int H, page_size, max_pages, num_pages;
};
constexpr int kDecodeStageKeys = 64;  // keys per pipeline stage of the split kernel
constexpr int kMaxSplitPages = 1024;  // page ids one split of the paged decode may touch
constexpr int kDecodeCtasPerSm = 2;   // resident split CTAs per SM (shared-memory bound)
cudaError_t launch_decode_split(const DecodeLaunch& a, cudaStream_t stream);
cudaError_t launch_combine(const float* u_part, const float* m_part, const float* l_part, void* o, float* lse,
                           int R, int S, int d, int o_fp32, cudaStream_t stream);
cudaError_t decode_status_word(unsigned int** p);

// Cross attention over at most kCrossShortKeys keys: R rows of each of BH key heads, `tiles` tiles of 128 a block.
constexpr int kCrossShortKeys = 128;
struct CrossShortArgs {
  void* o;
  float* lse;
  const int* kv_lens;
  int kv_heads, R, Nk, tiles, o_fp32;
  float sl2;  // scale * log2(e)
  unsigned long long budget;
};
struct CrossShortLaunch {
  CUtensorMap tq, tk, tv, to;  // 128-row boxes (to: bf16 O only)
  CrossShortArgs args;
  int BH, d;
};
cudaError_t launch_cross_short(const CrossShortLaunch& l, cudaStream_t stream);
cudaError_t cross_short_status_word(unsigned int** p);

// Cross attention of few rows: R <= kCrossRowsMax query rows of each of BH key heads against the first
// kv_lens[bh / kv_heads] (null: Nk) of its keys, shared out over S blocks.  u_part == null: the S <= 8
// blocks of a key head are a cluster and write o and lse; else partial slots [BH * R, S].
constexpr int kRowsStageKeys = 64;
constexpr int kCrossRowsMax = 32;
// Resident blocks per SM: at d = 128 two by shared memory, one of 32 rows by registers; at d = 64 four, or two.
constexpr int cross_rows_per_sm(int d, int rows) { return (d == 128 ? 2 : 4) / (rows > 16 ? 2 : 1); }
struct CrossRowsArgs {
  const void* q;
  void* o;
  float* lse;
  float* u_part;
  float* m_part;
  float* l_part;
  const int* kv_lens;
  int kv_heads, R, Nk, S, o_fp32;
  float sl2;  // scale * log2(e)
  unsigned long long budget;
  // Paged cache (block_table != nullptr): tk, tv map pools [num_pages * kv_heads, page_size, d], kv_lens (not null) has
  // at most Nk keys a sequence, of which the last `window` and the first `sinks` count.
  const int* block_table;  // [B, max_pages]
  int page_size, max_pages, num_pages, window, sinks;
};
struct CrossRowsLaunch {
  CUtensorMap tk, tv;  // 64-key boxes
  CrossRowsArgs args;
  int BH, d;
};
cudaError_t launch_cross_rows(const CrossRowsLaunch& a, cudaStream_t stream);
cudaError_t cross_rows_status_word(unsigned int** p);

// Backward launch description: q, k, v, dO as 3-D tensors {d, N, B*H} with
// 64 x 128 boxes and 128-byte swizzle; delta is the caller's [B*H, N] fp32 scratch.
struct BwdLaunch {
  CUtensorMap tq, tk, tv, tdo;
  CUtensorMap tdq, tdk, tdv;  // bf16 gradients as {d, N, B*H} for the TMA stores (unused for fp32)
  const void* o;
  const void* dout;
  const float* lse;
  float* delta;
  void* dq;
  void* dk;
  void* dv;
  int N;
  int BH;
  int d;
  int causal;
  int grad_fp32;
  float scale;
  float scale_log2;
  unsigned long long budget;
  int sms;  // SMs of the device (block order of the dK/dV and dQ kernels)
  // Cross attention (fa_cross_bwd): N query rows (of all the query heads of a key head) against
  // Nk keys, kv_lens[bh / kv_heads] of them real (null: all).  The dK/dV kernel's blocks take
  // q_tiles query tiles each (kv_splits blocks per key tile), the dQ kernel's k_tiles key tiles
  // (q_splits blocks per query tile); with more than one, they leave fp32 partial sums
  // [splits][rows, d] in kv_part (dK's, then dV's) and q_part, which a last kernel adds up.
  int Nk;
  const int* kv_lens;
  int kv_heads;
  int q_tiles, kv_splits;
  int k_tiles, q_splits;
  int own_tiles;  // query tiles that a block of the dQ kernel takes one after another
  float* kv_part;
  float* q_part;
};
cudaError_t launch_bwd(const BwdLaunch& a, cudaStream_t stream);
cudaError_t launch_cross_bwd(const BwdLaunch& a, cudaStream_t stream);
cudaError_t cross_bwd_status_word(unsigned int** p);
// out (and out2, from the S sums after those) = the sum of S partial sums of n elements each
cudaError_t launch_cross_sum(const float* part, void* out, void* out2, long long n, int S, int fp32, cudaStream_t stream);
// The backward over at most kCrossShortKeys keys (tk, tv: boxes of 64 rows for up to 64 keys), q_tiles and kv_splits as
// above.
cudaError_t launch_cross_bwd_short(const BwdLaunch& a, cudaStream_t stream);
cudaError_t cross_bwd_short_status_word(unsigned int** p);
// delta[r] = rowsum(o_r * dout_r) of `rows` bf16 rows of d
cudaError_t launch_delta(const void* o, const void* dout, float* delta, long long rows, int d, cudaStream_t stream);
cudaError_t bwd_status_word(unsigned int** p);

// E4M3 block quantization: x [BH, N, d] bf16 -> codes [BH, N, d] bytes, scales [BH, ceil(N/128)].
cudaError_t launch_quant_e4m3(const void* x, void* codes, float* scales, int BH, int N, int d, cudaStream_t stream);

// Rotary positions: q [B, Hq, N, d] and k [B, Hk, N, d] turned into q_out, k_out; with a block
// table k_out and v_out are the pools [num_pages, Hk, page_size, d] and token n of sequence b is key
// seq_lens[b] + n (tokens from new_lens[b] on are skipped).
struct RopeLaunch {
  fa_rope_axes_plan_t plan;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  const int* pos;  // [n_axes, B, N]
  int B, Hq, Hk, N;
  float sign;      // -1: the inverse rotation
  int heads;       // heads per block; set by launch_rope
  int sms;
  const int* block_table;  // [B, max_pages], or null
  const int* seq_lens;
  const int* new_lens;
  int page_size, max_pages, num_pages;
};
cudaError_t launch_rope(const RopeLaunch& a, cudaStream_t stream);

// Causal attention with a sliding window and sinks: N queries of each of the query heads, `group` of which share a key
// head, against its Nk >= N keys.  A tile's 128 rows are `tile` positions of `pack` query heads side by side (all that
// share the key head, or 1), a position's heads one after another; units = B * Hq / pack.
struct WindowFwdArgs {
  void* o;
  float* lse;
  int N, Nk, window, sinks, o_fp32;
  float sl2;  // scale * log2(e)
  unsigned long long budget;
  int units, share;  // units that share a key head: group / pack
  int pack, tile;
  int n_items, ng;   // items of two tiles, groups of units; set by launch_window_fwd
};
struct WindowFwdLaunch {
  CUtensorMap tq;        // {d, pack, N, units}, boxes of 64 x pack x tile
  CUtensorMap tk, tv;    // 128-row boxes
  CUtensorMap tks, tvs;  // k and v up to their first `sinks` rows
  CUtensorMap to;        // as tq, of a bf16 O (unset for fp32): at d = 64, and at d = 128 where pack > 1 for columns 0 .. 63
  WindowFwdArgs args;
  int d, sms;
};
cudaError_t launch_window_fwd(const WindowFwdLaunch& l, cudaStream_t stream);
cudaError_t window_fwd_status_word(unsigned int** p);

// Its backward.  The dK/dV kernel's items, per key head: every key tile's window of queries (a list of 128-row stages) in
// `splits` ranges of `stages`, then the queries behind tile 0's window, which see its sinks, in sink_items ranges of
// sink_stages.  fp32 partial sums [2 (dK, dV)][range][kv_heads][rows, d]: of the ranges (part, Nk rows) where there are more
// than one, of tile 0 (part0, 128 rows) where there are not but sinks, of the sinks' ranges (sink_part, sink_rows rows: the
// sinks).  A last kernel adds them up.
struct WindowBwdArgs {
  const float* rows;  // lse and rowsum(O dO) of the query rows, a head's row_stride apart; set by launch_window_bwd
  int row_stride;
  void* dq;
  void* dk;
  void* dv;
  float* part;
  float* part0;
  float* sink_part;
  int N, Nk, group, window, sinks, grad_fp32;
  int kv_heads;               // B * Hkv
  int splits, stages;
  int sink_items, sink_stages, sink_rows;
  int per_head;               // items of a key head
  int own_items, own_tiles;   // items, query tiles that a block takes one after another
  bool flat;                  // of the list of all heads', not of one head's
  int ng, ng_q;               // groups of key heads, of query heads; set by launch_window_bwd
  float sl2, scale;
  unsigned long long budget;
};
struct WindowBwdLaunch {
  CUtensorMap tq, tk, tv, tks, tvs, tdo;  // as WindowFwdLaunch
  CUtensorMap tdq, tdk, tdv;              // bf16 gradients only
  WindowBwdArgs args;
  const void* q;
  const void* k;
  const void* v;
  const void* o;
  const void* dout;
  const float* lse;
  float* rows;  // window_bwd_rows_bytes() of scratch, 256-byte aligned
  int d, sms;
};
size_t window_bwd_rows_bytes(int heads, int N);
cudaError_t launch_window_bwd(const WindowBwdLaunch& l, cudaStream_t stream);
cudaError_t window_bwd_status_word(unsigned int** p);

// RMS norm of each head's q and k, then the rotation: tensors and plan as RopeLaunch (block_table, seq_lens and
// max_pages unused), weights [d] bf16 or fp32 (null: ones).  slots [B, N] (not null): k and v go to the pools, token n
// of sequence b to row slots[b * N + n] of the pages' keys.
struct NormRopeLaunch {
  RopeLaunch r;
  const void* q_weight;
  const void* k_weight;
  int weight_fp32;
  float eps;
  const long long* slots;
  // backward: the gradients of q_out and k_out, those of q and k, and those of the weights (null: not wanted) by way
  // of `part`, fp32 partial sums [norm_rope_partials()][d]
  const __nv_bfloat16* dq_out;
  const __nv_bfloat16* dk_out;
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  float* dq_weight;
  float* dk_weight;
  float* part;
};
cudaError_t launch_norm_rope(const NormRopeLaunch& a, cudaStream_t stream);
cudaError_t launch_norm_rope_bwd(const NormRopeLaunch& a, cudaStream_t stream);
// Partial sums of the weights' gradients that launch_norm_rope_bwd leaves for these sizes.
int norm_rope_partials(int B, int Hq, int Hk, int N, int d, int sms);

// Pages for new_lens[b] more tokens of each sequence (fewer where negative): see fa_pages_extend.
struct PagesLaunch {
  int* block_table;  // [B, max_pages]
  int* seq_lens;
  const int* new_lens;
  int* free_pages;  // [num_pages]
  int* n_free;
  int* granted;
  long long* slots;  // [B, N], or null
  int B, N, page_size, max_pages, num_pages;
};
cudaError_t launch_pages(const PagesLaunch& a, cudaStream_t stream);

// Fixed device scratch used by fa_decode_splitkv_noalloc in place of a
// caller-provided workspace.  Size limit of that entry point.
constexpr size_t kNoAllocScratchBytes = size_t(8) << 20;
// Device address of that scratch on the current device (looked up once per device).
cudaError_t decode_noalloc_scratch(void** ptr);

}  // namespace fattn
