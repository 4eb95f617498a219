/*
 * libfattn -- exact fused attention for GB300 (sm_103a): the fused forward
 * (bf16, or E4M3 inputs with block scales), its backward, a split-KV decode
 * (contiguous or paged KV cache), the log-sum-exp combine of partials and a
 * forward over one key shard; cross attention, sliding windows with sinks,
 * rotary positions with or without the heads' norms, and the pages of a paged
 * cache.  C ABI: plain pointers, sizes and a stream handle.
 *
 * What is computed (per batch b and head h, scores scaled by `scale`):
 *     S = scale * Q K^T,   P = softmax(S) row-wise,   O = P V,
 *     lse_i = m_i + ln(l_i)   (natural log of the scaled scores),
 * in a single tiled pass with online softmax, so that the N x N score and
 * probability matrices never reach device memory (xuesongtap.github.io
 * "flash-attention" page, §1 equation for S, P, O, §2.1 tiling, §2.2 online
 * softmax, §3 saved log-sum-exp; triton-tutorial "8. FlashAttention 实战",
 * §8.3.3 incremental formula and §8.4 kernel walk-through).
 *
 * Conventions shared by every entry point
 *   - Device pointers only (memory the caller allocated with the CUDA runtime
 *     on the current device).  The library allocates nothing, frees nothing
 *     and keeps no state beyond cached per-device queries (arch, SM count,
 *     addresses), the per-device status words taken by fa_get_status() and the
 *     fixed scratch array of fa_decode_splitkv_noalloc.
 *   - All tensors are contiguous, row-major in the head dimension d.
 *   - `stream` is a cudaStream_t (CUstream) handle; NULL is the legacy
 *     default stream.  Every call is asynchronous on that stream.
 *   - Arguments are checked before anything is launched; a rejected call
 *     returns an error status, writes nothing and launches nothing.  No C++
 *     exception crosses this boundary.  There is no CPU fallback and no
 *     other backend: an unsupported request is an error.
 *   - Supported head dimensions: d = 64 and d = 128 (the FP8 forward: 128).
 *   - Scaled scores: below 2^29 in magnitude.  An exponent is the difference
 *     of a score and its row's maximum, both times log2(e), of which the
 *     maximum is rounded to fp32: by up to 2^-24 of it, in all the row's
 *     exponents alike, so it cancels in O and lse -- until, from 2^31 on, that
 *     alone takes 2^x out of fp32's range (O NaN or 0).  Gradients start from
 *     the fp32 lse, whose rounding does not cancel: P is off by 2^-23 |lse|.
 *   - Device: compute capability 10.3 (GB300).  Anything else gives
 *     FA_ERR_ARCH.
 */
#ifndef FATTN_H
#define FATTN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1, /* null pointer, bad size, misaligned pointer, non-finite or non-positive scale */
  FA_ERR_UNSUPPORTED = 2, /* valid request this library does not implement (e.g. d not in {64, 128}) */
  FA_ERR_ARCH = 3,        /* current device is not compute capability 10.3, or no device */
  FA_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed (launch, attribute, tensor map) */
  FA_ERR_TIMEOUT = 5,     /* a kernel's bounded wait expired; its outputs are undefined */
  FA_ERR_WORKSPACE = 6    /* workspace missing or smaller than fa_decode_workspace_bytes() */
} fa_status_t;

/* Options for fa_fwd_ex.  A zero-initialised struct gives fa_fwd's behaviour. */
typedef struct {
  int o_fp32;                            /* 0: O is bf16 (round to nearest even); 1: O is fp32 */
  unsigned long long wait_budget_cycles; /* per-wait spin budget in SM clock cycles; 0 = default (about 2 s) */
  void* workspace;                       /* optional device scratch, 256-byte aligned, for the key split
                                            (fa_fwd_workspace_bytes); NULL: one launch, no split */
  size_t workspace_bytes;                /* its size in bytes */
} fa_fwd_opts;

/*
 * fa_fwd -- fused attention forward (prefill).
 *
 * Follows the FA-2 scan order: a 128-row query tile Q_i stays on chip while
 * the 128-key tiles K_j, V_j stream past it; per tile the running row max m,
 * the denominator l and the unnormalised output U are updated with
 * alpha = exp(m_old - m_new), and O = U / l is formed once after the scan
 * (xuesongtap §2.1-§2.2; triton-tutorial §8.4.1-§8.4.5).
 *
 *   q, k, v  [B, H, N, d] bf16, 16-byte aligned.
 *   o        [B, H, N, d] bf16, 16-byte aligned (written).
 *   lse      [B, H, N] fp32, 4-byte aligned (written): m + ln(l) of the
 *            scaled scores, the statistic a backward pass recomputes P from.
 *   B, H, N  >= 1.   d in {64, 128}.
 *   scale    finite and > 0 (callers usually pass 1/sqrt(d)).
 *   causal   0: every key; 1: query i attends keys j <= i (top-left aligned,
 *            square), masked scores are -inf and tiles above the diagonal
 *            are skipped (triton-tutorial §8.7.1).
 * Returns FA_OK once the kernel is queued.  Kernel-side timeouts are reported
 * by fa_get_status().
 */
fa_status_t fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                   int B, int H, int N, int d, float scale, int causal, void* stream);

/* fa_fwd with options (opts may be NULL).  With opts->o_fp32 = 1, `o` is an
 * fp32 [B, H, N, d] tensor.
 *
 * The last round (non-causal, d = 64): the forward works on blocks of 256
 * query rows of a (b, h), one block per SM at a time, so when the last round
 * of blocks only partly fills the SMs most of them idle through it.  Such a
 * round is split, whichever of two ways the plan (by the device's SM count)
 * finds cheaper: its blocks run as their two 128-row query tiles, each on an
 * SM of its own (no workspace); or, given a workspace of
 * fa_fwd_workspace_bytes() bytes, they are cut along the keys into pieces that
 * each leave a partial (U, m, l) per row, which a second kernel merges by the
 * online-softmax rule, as the split-KV decode does (FlashDecoding split-K,
 * cnblogs jzssuanfa page, §三 场景 B).  O and lse are the same function of
 * q, k, v up to rounding order.  With a workspace too small for the plan:
 * FA_ERR_WORKSPACE. */
fa_status_t fa_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse,
                      int B, int H, int N, int d, float scale, int causal, void* stream,
                      const fa_fwd_opts* opts);

/* fa_fwd_workspace_bytes -- scratch bytes the key split of fa_fwd_ex's last
 * round needs on the current device for this problem, or 0 when it plans no
 * key split (causal launches, d = 128, last rounds that are nearly full or
 * that the query split serves as well, fewer than 4 key tiles, invalid sizes,
 * no sm_103a device).  The plan depends on the device's SM count. */
size_t fa_fwd_workspace_bytes(int B, int H, int N, int d, int causal);

/*
 * fa_fwd_partial -- the forward over one shard of the keys, leaving a partial
 * (U, m, l) per query row for fa_combine instead of O and lse.  This is the
 * sequence-sharded prefill of Ring Attention without the ring: each KV shard
 * is one pass of the forward kernel, and the partials merge by the
 * online-softmax rule (cnblogs jzssuanfa page, §三 场景 A; xuesongtap §5).
 *
 *   q        [B, H, N, d] bf16, 16-byte aligned: every query row.
 *   k, v     [B, H, Nk, d] bf16, 16-byte aligned: the shard's keys, whose
 *            global indices are key_offset .. key_offset + Nk - 1.
 *   u_part   [B*H*N, S, d] fp32, 16-byte aligned: slot `shard` of each row is
 *            written with U = sum_j exp(s_j - m) v_j over the row's admissible
 *            keys of the shard.
 *   m_part,  [B*H*N, S] fp32, 4-byte aligned: slot `shard` gets m (the row max
 *   l_part   of the scaled scores, natural-log units) and l = sum_j exp(s_j - m).
 *            A row with no admissible key in the shard gets m = -inf and
 *            l = 0; its U slot is left as it was (fa_combine does not use it).
 *   causal   1: query i attends global keys j <= i (top-left aligned).
 *   d in {64, 128}; 0 <= shard < S; key_offset >= 0; other arguments as fa_fwd.
 * After one call per shard (any order, any stream order that completes them
 * first), fa_combine(u_part, m_part, l_part, o, lse, B*H*N, S, d) gives the
 * forward over all the shards' keys.
 */
fa_status_t fa_fwd_partial(const void* q, const void* k, const void* v, float* u_part, float* m_part,
                           float* l_part, int B, int H, int N, int Nk, int key_offset, int d,
                           float scale, int causal, int shard, int S, void* stream);

/* fa_fwd_partial reading the shard straight from the whole key tensors, with no per-shard copy:
 *   k, v     [B, H, kv_rows, d] bf16, 16-byte aligned: the full key sequence of every head; the
 *            shard is rows key_offset .. key_offset + Nk - 1 of each head (its global key
 *            indices, as for fa_fwd_partial).  kv_rows >= key_offset + Nk.  Keys of the tensor
 *            outside the shard may be read (a tile that ends inside the shard) and are masked
 *            as inadmissible.
 *   kv_rows  0: k, v are the shard's own [B, H, Nk, d] buffers, exactly fa_fwd_partial.
 * Other arguments, results and errors as fa_fwd_partial (FA_ERR_INVALID_ARG for kv_rows < 0 or
 * kv_rows < key_offset + Nk). */
fa_status_t fa_fwd_partial_ex(const void* q, const void* k, const void* v, float* u_part, float* m_part,
                              float* l_part, int B, int H, int N, int Nk, int key_offset, int kv_rows,
                              int d, float scale, int causal, int shard, int S, void* stream);

/*
 * fa_quantize_e4m3 -- block quantization of Q, K or V for fa_fwd_fp8
 * (triton-tutorial "8. FlashAttention 实战", §8.9.4: one scale per block of
 * 128 rows x d; scale = max|x| / 448, 448 being E4M3's largest finite value).
 *
 *   x        [B, H, N, d] bf16, 16-byte aligned (read).
 *   codes    [B, H, N, d] bytes, 16-byte aligned (written): the E4M3 code
 *            (OCP FP8 E4M3, bias 7, no infinities) of x / scale, rounded to
 *            nearest, ties to even, saturating at +-448; the sign of x is kept.
 *   scales   [B, H, ceil(N/128)] fp32, 4-byte aligned (written): the block's
 *            scale, fp32(max|x| / 448), or 1 for an all-zero block.
 *   B, H, N  >= 1;  d in {64, 128}.
 * The scale and the division are IEEE fp32 operations, so the codes are a
 * deterministic function of x.  Returns FA_OK once the kernel is queued.
 */
fa_status_t fa_quantize_e4m3(const void* x, void* codes, float* scales,
                             int B, int H, int N, int d, void* stream);

/*
 * fa_fwd_fp8 -- fused attention forward on E4M3 inputs (triton-tutorial
 * §8.9.3: both GEMMs in FP8 with fp32 accumulation, the softmax in fp32,
 * P quantized to FP8 before the second GEMM).
 *
 *   q8, k8, v8  [B, H, N, d] E4M3 codes (fa_quantize_e4m3), 16-byte aligned.
 *   sq, sk, sv  [B, H, ceil(N/128)] fp32 block scales, 4-byte aligned:
 *               row r of a head dequantizes as code * s[r / 128].
 *   o           [B, H, N, d] bf16 (fp32 with opts->o_fp32), 16-byte aligned.
 *   lse         [B, H, N] fp32 (written), as for fa_fwd.
 *   d           must be 128 (FA_ERR_UNSUPPORTED otherwise).
 *   scale, causal, opts: as for fa_fwd_ex (opts may be NULL; no split last round:
 *               opts->workspace is not used).
 * Scores are S = (q8 k8^T) * sq_i * sk_j * scale in fp32; P~ of key tile j
 * is stored as E4M3 of p * 256 * sv_j / max_j(sv_j) (p <= 1 after the row
 * max is subtracted), so that P~ V8 accumulates in one unit for every key
 * tile and O = U * max(sv) / 256 / l.  l sums the fp32 p.
 */
fa_status_t fa_fwd_fp8(const void* q8, const void* k8, const void* v8,
                       const float* sq, const float* sk, const float* sv,
                       void* o, float* lse, int B, int H, int N, int d, float scale,
                       int causal, void* stream, const fa_fwd_opts* opts);

/* Options of fa_decode_splitkv_ex and fa_decode_paged_ex.  A zero-initialised
 * struct (or NULL) gives the behaviour of the entry points without _ex. */
typedef struct {
  int o_fp32;                            /* 0: O is bf16 (round to nearest even); 1: O is fp32 [B, H, d] */
  unsigned long long wait_budget_cycles; /* per-wait spin budget of the split kernel in SM clock
                                            cycles; 0 = default (about 2 s).  A wait that runs out
                                            ends the kernel and fa_get_status() reports
                                            FA_ERR_TIMEOUT; O and lse are then undefined. */
} fa_decode_opts;

/*
 * fa_decode_workspace_bytes -- bytes of scratch that fa_decode_splitkv needs.
 *
 * The workspace holds one partial (U [d] fp32, m fp32, l fp32) per (b, h, split).
 * `chunk` is the key granularity of a split (must be 128); `splits` is the
 * number of partials per (b, h), or 0 to let the library choose from L and the
 * current device's SM count.  Returns 0 for invalid arguments.
 */
size_t fa_decode_workspace_bytes(int B, int H, int L, int d, int chunk, int splits);

/*
 * fa_decode_splitkv -- single-token decode with the KV sequence split
 * (FlashDecoding split-K: the query row is broadcast, each split of the KV
 * cache yields a partial (O_partial, m, l), and the partials are merged by
 * the online-softmax rule; cnblogs jzssuanfa page, §三 场景 B; iceferryling
 * "FlashAttention 1 和 FlashAttention 2 的区别", §13 decode is KV-bandwidth
 * bound).
 *
 *   q        [B, H, d] bf16, 16-byte aligned.
 *   k, v     [B, H, L, d] bf16, 16-byte aligned (the KV cache, every key
 *            admissible: no mask).
 *   o        [B, H, d] bf16 (written).   lse [B, H] fp32 (written).
 *   L >= 1.  chunk = 128.  splits in [0, ceil(L/128)], 0 = automatic; each
 *   split covers a whole number of 128-key chunks.  splits = ceil(L/128)
 *   gives one partial per chunk.
 *   workspace, ws_bytes: caller-owned device scratch of at least
 *   fa_decode_workspace_bytes(B, H, L, d, chunk, splits) bytes, 256-byte
 *   aligned; FA_ERR_WORKSPACE if smaller or NULL.  Its contents on return
 *   are the partials in fa_combine's layout (u_part, then m_part, then
 *   l_part, each 256-byte aligned).
 * Two kernels run on `stream`: the split kernel, then the combine kernel.
 */
fa_status_t fa_decode_splitkv(const void* q, const void* k, const void* v, void* o, float* lse,
                              int B, int H, int L, int d, float scale, int chunk, int splits,
                              void* workspace, size_t ws_bytes, void* stream);

/* fa_decode_splitkv with options (opts may be NULL): opts->o_fp32 = 1 makes `o`
 * an fp32 [B, H, d] tensor (16-byte aligned); opts->wait_budget_cycles bounds
 * each wait of the split kernel. */
fa_status_t fa_decode_splitkv_ex(const void* q, const void* k, const void* v, void* o, float* lse,
                                 int B, int H, int L, int d, float scale, int chunk, int splits,
                                 void* workspace, size_t ws_bytes, void* stream, const fa_decode_opts* opts);

/*
 * fa_decode_splitkv_noalloc -- fa_decode_splitkv for callers that cannot
 * allocate device memory.  (The pages have no counterpart to this entry
 * point: it exists for embedding, not for the method.)
 *
 * Some callers are handed only their input and output buffers and may not
 * call cudaMalloc themselves: plugins inside inference runtimes that own all
 * device memory through their own allocator, and request paths that must not
 * pay for, or risk the device-wide synchronisation of, an allocation or a
 * free.  They have no workspace to pass, so this entry point keeps the
 * per-split partials in a fixed array of device memory compiled into the
 * library (FA_NOALLOC_SCRATCH_BYTES, 8 MiB) instead.  It calls no cudaMalloc,
 * cudaFree or other allocating routine.
 *
 *   Arguments as fa_decode_splitkv, without workspace and ws_bytes.
 *   The partials of B*H rows with S splits take
 *   fa_decode_workspace_bytes(B, H, L, d, chunk, S) bytes; B*H*S*(d+2)*4 bytes
 *   is about the need: e.g. B*H = 2048 rows at d = 128 fit up to 7 splits.
 *   With splits = 0 the split count is the automatic one of fa_decode_splitkv
 *   when its partials fit, else the largest smaller count whose partials fit
 *   (O and lse are the same function of q, k, v either way, up to rounding
 *   order).  An explicit split count whose partials do not fit, or B*H rows
 *   that do not fit even with one split (more than 16131 rows at d = 128),
 *   return FA_ERR_WORKSPACE (fa_last_error() says by how much) and launch
 *   nothing.
 *   Every GPU that loads the library's decode code holds the 8 MiB array until
 *   the process exits.  The first call on each device looks up the array's
 *   device address (cudaGetSymbolAddress) with that device current; make that
 *   first call before any stream capture.
 *   All calls share the one array and it keeps the last call's partials:
 *   nothing in it needs to start at zero (every partial is written before it
 *   is read), but calls whose kernels overlap on the GPU -- on different
 *   streams, or from different host threads -- race on it and give undefined
 *   results.  Serialise them (one stream, or events).
 */
#define FA_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
fa_status_t fa_decode_splitkv_noalloc(const void* q, const void* k, const void* v, void* o, float* lse,
                                      int B, int H, int L, int d, float scale, int chunk, int splits,
                                      void* stream);

/*
 * fa_decode_paged -- fa_decode_splitkv over a paged KV cache (iceferryling
 * "FlashAttention 1 和 FlashAttention 2 的区别", §13: decode kernels read the
 * cache through a paged block table).  Same split and combine; only the
 * address of each key changes.
 *
 *   q            [B, H, d] bf16, 16-byte aligned.
 *   k_pages,     [num_pages, H, page_size, d] bf16 pools, 16-byte aligned:
 *   v_pages      page p holds page_size consecutive keys of one sequence for
 *                every head.
 *   block_table  [B, max_pages] int32, 4-byte aligned: logical page i of
 *                sequence b (keys i*page_size .. +page_size-1) is pool page
 *                block_table[b*max_pages + i].  Only the entries covering
 *                seq_lens[b] keys are read.  An id outside [0, num_pages)
 *                reads as zero keys and values (no fault).
 *   seq_lens     [B] int32, 4-byte aligned: keys of sequence b.  Values are
 *                clamped to [0, max_seq_len]; a length of 0 gives O = 0 and
 *                lse = -inf for that sequence.
 *   o [B, H, d] bf16, lse [B, H] fp32 (written), as for fa_decode_splitkv.
 *   page_size    a positive multiple of 64.  max_pages, num_pages >= 1.
 *   max_seq_len  the longest seq_lens value, 1 .. max_pages*page_size: the
 *                host plans the splits for it (the lengths are device data).
 *   splits       partials per (b, h), 0 = chosen from max_seq_len and the SM
 *                count, as for fa_decode_splitkv; a split covers at most
 *                1023 pages (FA_ERR_UNSUPPORTED beyond).
 *   workspace    >= fa_decode_paged_workspace_bytes(...) bytes, 256-byte aligned.
 * Keys at or past seq_lens[b] are masked and their rows never read into O,
 * whatever the page holds there.  Returns FA_OK once both kernels are queued.
 */
size_t fa_decode_paged_workspace_bytes(int B, int H, int max_seq_len, int d, int page_size, int max_pages,
                                       int splits);
fa_status_t fa_decode_paged(const void* q, const void* k_pages, const void* v_pages,
                            const int* block_table, const int* seq_lens, void* o, float* lse,
                            int B, int H, int d, int page_size, int max_pages, int num_pages,
                            int max_seq_len, float scale, int splits, void* workspace,
                            size_t ws_bytes, void* stream);
/* fa_decode_paged with options (opts may be NULL), as for fa_decode_splitkv_ex. */
fa_status_t fa_decode_paged_ex(const void* q, const void* k_pages, const void* v_pages,
                               const int* block_table, const int* seq_lens, void* o, float* lse,
                               int B, int H, int d, int page_size, int max_pages, int num_pages,
                               int max_seq_len, float scale, int splits, void* workspace,
                               size_t ws_bytes, void* stream, const fa_decode_opts* opts);

/*
 * fa_combine -- merge S partial (U, m, l) triples per row into O and lse:
 *     m = max_s m_s,  w_s = exp(m_s - m),  l = sum_s w_s l_s,
 *     O = sum_s w_s U_s / l,  lse = m + ln(l)
 * (iceferryling page §6, cross-warp merge formula; the same rule is the
 * FlashDecoding tree reduction and the Ring Attention merge).
 *
 *   u_part [R, S, d] fp32, unnormalised numerators (relative to exp(s - m_s)).
 *   m_part [R, S] fp32, row maxima in natural-log units of scaled scores.
 *   l_part [R, S] fp32, denominators.
 *   An empty partial (m = -inf) has weight 0 and its U and l are not used;
 *   a row whose partials are all empty gets O = 0 and lse = -inf.
 *   o [R, d] bf16 (written), lse [R] fp32 (written).  R, S >= 1, d in {64, 128}.
 *   u_part 16-byte aligned; m_part, l_part, lse 4-byte aligned; o 16-byte aligned.
 */
fa_status_t fa_combine(const float* u_part, const float* m_part, const float* l_part,
                       void* o, float* lse, int R, int S, int d, void* stream);
/* fa_combine with the output type chosen: o_fp32 = 0 writes o [R, d] bf16
 * (round to nearest even), o_fp32 = 1 writes o [R, d] fp32 (16-byte aligned). */
fa_status_t fa_combine_ex(const float* u_part, const float* m_part, const float* l_part,
                          void* o, float* lse, int R, int S, int d, int o_fp32, void* stream);

/*
 * fa_bwd_workspace_bytes -- scratch bytes fa_bwd needs: the per-row
 * D_i = rowsum(O_i * dO_i), B*H*N fp32, rounded up to 256 bytes.  0 for
 * invalid sizes.
 */
size_t fa_bwd_workspace_bytes(int B, int H, int N);

/*
 * fa_bwd -- attention backward with recomputation: from Q, K, V, the
 * forward's O and lse, and dO, compute
 *     D  = rowsum(O * dO),   P = exp(scale Q K^T - lse)  (recomputed per tile),
 *     dV = P^T dO,   dS = P * (dO V^T - D),   dQ = scale dS K,   dK = scale dS^T Q
 * (triton-tutorial "8. FlashAttention 实战", §8.8.1-§8.8.4; operatorworld,
 * "反向传播：用重算换显存").  P is never stored: one kernel owns a key tile
 * and produces its dK, dV; another owns a query tile and produces its dQ
 * (no atomics: every output is written by one CTA in a fixed order, so the
 * gradients are bitwise repeatable).
 *
 *   q, k, v, o, dout  [B, H, N, d] bf16, 16-byte aligned; o and lse must be the
 *                     forward's outputs for the same q, k, v, scale, causal.
 *   lse               [B, H, N] fp32 (natural log of scaled scores).
 *   dq, dk, dv        [B, H, N, d], written: bf16, or fp32 when grad_fp32 = 1.
 *   d in {64, 128}; scale finite > 0; causal 0/1 as for fa_fwd.
 *   workspace         >= fa_bwd_workspace_bytes(B, H, N) bytes, 256-byte
 *                     aligned, caller-owned (holds D); FA_ERR_WORKSPACE if
 *                     smaller or NULL.
 * Three kernels run on `stream`: D, then dK/dV, then dQ.
 */
fa_status_t fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                   const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                   float scale, int causal, int grad_fp32, void* workspace, size_t ws_bytes,
                   void* stream);

/* Options of fa_bwd_ex.  wait_budget_cycles: per-wait budget in SM cycles of
 * the dK/dV and dQ kernels, as in fa_fwd_opts (0 = the default, about 2 s);
 * a wait that runs out ends the kernel, and fa_get_status then reports
 * FA_ERR_TIMEOUT (the gradients are undefined). */
typedef struct fa_bwd_opts {
  unsigned long long wait_budget_cycles;
} fa_bwd_opts;

/* fa_bwd with options; opts may be NULL (then it is fa_bwd).  Arguments,
 * results and errors otherwise as fa_bwd. */
fa_status_t fa_bwd_ex(const void* q, const void* k, const void* v, const void* o, const void* dout,
                      const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                      float scale, int causal, int grad_fp32, void* workspace, size_t ws_bytes,
                      void* stream, const fa_bwd_opts* opts);

/*
 * Cross attention: queries of a decoder against an encoder's states, whose count differs from the
 * queries' and from sequence to sequence (the scaled-dot-product interface takes k and v of another
 * length than q: xuesongtap §6).  Not causal.  Query heads may share key heads: query head h reads
 * key head h / (Hq / Hkv).  With Nq = 1 it is the single-token form, by the same call: where a key
 * head has few query rows, up to eight blocks (a thread-block cluster) share its keys and join their
 * partials themselves.
 *
 *   q         [B, Hq, Nq, d] bf16, 16-byte aligned.
 *   k, v      [B, Hkv, Nk, d] bf16, 16-byte aligned.  Hq a multiple of Hkv.
 *   kv_lens   [B] int32, 4-byte aligned, or NULL: sequence b attends its keys 0 .. kv_lens[b] - 1
 *             (values are clamped to [0, Nk]; NULL: all Nk).  What k and v hold behind them may be
 *             anything, infinities and NaN included, and has no influence.  A sequence of length 0
 *             gets O = 0 and lse = -inf, and gradients of 0.
 *   o         [B, Hq, Nq, d] bf16, or fp32 with opts->o_fp32 (written), 16-byte aligned.
 *   lse       [B, Hq, Nq] fp32 (written), natural log of the scaled scores, as for fa_fwd.
 *   d in {64, 128}; scale finite and > 0; every size >= 1.
 */
typedef struct {
  int o_fp32;                            /* 0: O is bf16 (round to nearest even); 1: O is fp32 */
  unsigned long long wait_budget_cycles; /* per-wait budget in SM cycles, as in fa_fwd_opts (0 = default) */
} fa_cross_opts;

/* Scratch bytes for the partials of fa_cross_fwd where it cuts the keys into ranges that a second
 * kernel joins, so that few query rows still fill the SMs: more than eight ranges of a few rows, or
 * ranges of many rows' long keys.  0 when the call leaves no partials (keys uncut, or shared within
 * a cluster), for invalid sizes, or without a device. */
size_t fa_cross_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d);

/* fa_cross_fwd -- workspace: caller-owned device scratch of fa_cross_workspace_bytes() bytes,
 * 256-byte aligned (FA_ERR_WORKSPACE if smaller), or NULL: one kernel without partials (the keys of a
 * few rows may still be shared within a cluster).  O and lse are the same function of the inputs either
 * way, up to rounding order.  A workspace serves one call at a time (calls that overlap on the GPU need
 * one each).  opts may be NULL. */
fa_status_t fa_cross_fwd(const void* q, const void* k, const void* v, const int* kv_lens, void* o, float* lse,
                         int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale, void* workspace,
                         size_t ws_bytes, void* stream, const fa_cross_opts* opts);

/* Scratch bytes of fa_cross_bwd on the current device: rowsum(O * dO) per query row (of more than
 * 128 keys), and fp32 partial gradients where it cuts a long scan into ranges (few key tiles under
 * many queries, or the reverse).  Never 0 for valid sizes; 0 for invalid ones or without a device. */
size_t fa_cross_bwd_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d);

/* fa_cross_bwd -- the gradients, by the formulas of fa_bwd: dq like q, dk and dv like k and v (bf16,
 * or fp32 when grad_fp32 = 1).  dk and dv sum over the query heads that share the key head; rows of
 * keys behind kv_lens[b] are written as 0.  o (bf16) and lse are fa_cross_fwd's for the same q, k, v,
 * kv_lens and scale.  No atomics: the gradients are bitwise repeatable.  opts may be NULL. */
fa_status_t fa_cross_bwd(const void* q, const void* k, const void* v, const int* kv_lens, const void* o,
                         const void* dout, const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv,
                         int Nq, int Nk, int d, float scale, int grad_fp32, void* workspace, size_t ws_bytes,
                         void* stream, const fa_bwd_opts* opts);

/*
 * Rotary positions with several axes, for q and k before attention: pair i of a row's d
 * dimensions belongs to one axis (time, height, width, ...) and is turned by the angle
 * pos[axis_i] * rate_i: (a, b) -> (a cos - b sin, a sin + b cos).
 */
#define FA_ROPE_MAX_AXES 4
typedef struct {  /* made by fa_rope_axes_plan; host memory, copied by each call */
  int d, n_axes, interleaved;
  unsigned char axis[64];       /* of each pair */
  unsigned long long turns[64]; /* rate / (2 pi) of each pair, in 2^-64 turns per position */
} fa_rope_axes_plan_t;

/*
 * fa_rope_axes_plan -- fill *plan (host only; no device is touched).
 *   d            64 or 128.
 *   sections     [n_axes] pairs of each axis, each >= 1, d/2 in all; 1 <= n_axes <= FA_ROPE_MAX_AXES
 *                (one axis is the ordinary rotary embedding).
 *   base         finite, >= 1.
 *   interleaved  0: pair i is dimensions i and i + d/2; 1: dimensions 2i and 2i + 1.
 *   per_axis     0: rate_i = base^(-i / (d/2)) over all pairs; 1: each axis starts anew,
 *                base^(-j / sections[a]) for its j-th pair.
 *   cyclic       0: the axes' pairs lie one section after another; 1: they are dealt out in turn
 *                (t h w t h w ..) to the axes that have pairs left.
 */
fa_status_t fa_rope_axes_plan(fa_rope_axes_plan_t* plan, int d, int n_axes, const int* sections, double base,
                              int interleaved, int per_axis, int cyclic);

/*
 * fa_rope_axes -- turn q [B, Hq, N, d] into q_out and k [B, Hk, N, d] into k_out (bf16, 16-byte
 * aligned), in one kernel.  An output may be its own input (in place); otherwise they do not overlap.
 *   pos      [n_axes, B, N] int32, 4-byte aligned: any values; angles are exact to 2^-24 of a half
 *            turn for every position up to 2^24 (2^-18 for any 32-bit one).
 *   Hk       0: q alone (k and k_out are not used).
 *   inverse  1: turn back.  The rotation's inverse is its transpose, so this is the backward pass:
 *            the gradients of q and k from those of q_out and k_out.
 * cos, sin and products in fp32, one rounding to bf16 (nearest even).
 */
fa_status_t fa_rope_axes(const void* q, const void* k, const int* pos, void* q_out, void* k_out, int B, int Hq,
                         int Hk, int N, const fa_rope_axes_plan_t* plan, int inverse, void* stream);

/*
 * fa_rope_axes_paged -- the serving form: N new tokens of each sequence (1 in a decode step, more in
 * a chunk of a prompt).  q [B, Hq, N, d] is turned into q_out; k [B, Hk, N, d] is turned and v (the
 * same shape) copied into the paged cache of fa_decode_paged: pools [num_pages, Hk, page_size, d] with
 * block_table [B, max_pages].
 *   seq_lens   [B] int32: keys that sequence b had before; its token t becomes key seq_lens[b] + t.
 *   new_lens   [B] int32 or NULL: tokens of sequence b in this call; those from new_lens[b] on are
 *              padding, for which nothing is written (not to q_out either).
 *   A token whose key has no page (seq_lens[b] + t negative, or at or past max_pages * page_size, or
 *   an id outside [0, num_pages)) is not written to the pools.  page_size as for fa_decode_paged; Hk >= 1.
 *   The pools are written only at the new tokens' rows; two tokens of one call must not share a row.
 */
fa_status_t fa_rope_axes_paged(const void* q, const void* k, const void* v, const int* pos, void* q_out,
                               void* k_pages, void* v_pages, const int* block_table, const int* seq_lens,
                               const int* new_lens, int B, int Hq, int Hk, int N, int page_size, int max_pages,
                               int num_pages, const fa_rope_axes_plan_t* plan, void* stream);

/*
 * Causal attention with a sliding window and sinks (the first tokens, which stay visible).  The N queries of a sequence
 * are its last ones: query i stands at position p = Nk - N + i and sees key j when
 *     j <= p   and   (j > p - window  or  j < sinks).
 * Query heads may share key heads: query head h reads key head h / (Hq / Hkv).  N = Nk is a whole prompt or a
 * training step, N < Nk a chunk of a prompt behind earlier keys.  (One token over a paged cache:
 * fa_window_decode_paged.)
 *
 *   q         [B, Hq, N, d] bf16, 16-byte aligned.
 *   k, v      [B, Hkv, Nk, d] bf16, 16-byte aligned.  Hq a multiple of Hkv, N <= Nk.  Keys that no query sees
 *             (before the first query's window, but for the sinks) may hold anything, infinities and NaN
 *             included, and have no influence; they get gradients of 0.
 *             (Of keys that some query sees, one that is not finite may make other queries near it NaN too, as a product with
 *             a probability of 0 does.)
 *   window    >= 1 (1: its own key alone; >= Nk: plain causal attention).
 *   sinks     0 .. 128 (FA_ERR_UNSUPPORTED beyond).
 *   o         [B, Hq, N, d] bf16, or fp32 with opts->o_fp32 (written), 16-byte aligned.
 *   lse       [B, Hq, N] fp32 (written), natural log of the scaled scores, as for fa_fwd.
 *   d in {64, 128}; scale finite and > 0; every size >= 1, Nk at most 2^30.  Outputs and gradients overlap no input
 *   and not one another.
 */
typedef struct {
  int o_fp32;                            /* 0: O is bf16 (round to nearest even); 1: O is fp32 */
  unsigned long long wait_budget_cycles; /* per-wait budget in SM cycles, as in fa_fwd_opts (0 = default) */
} fa_window_opts;

/* fa_window_fwd -- opts may be NULL.  One kernel, no workspace. */
fa_status_t fa_window_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int N,
                          int Nk, int d, float scale, int window, int sinks, void* stream, const fa_window_opts* opts);

/* Scratch bytes of fa_window_bwd on the current device: rowsum(O * dO) per query row, and fp32 partial gradients of
 * the key tile with the sinks, which every query reaches, and of all keys where there are few key tiles under many
 * queries.  0 for invalid sizes or without a device. */
size_t fa_window_bwd_workspace_bytes(int B, int Hq, int Hkv, int N, int Nk, int d, int window, int sinks);

/* fa_window_bwd -- the gradients, by the formulas of fa_bwd: dq like q, dk and dv like k and v (bf16, or fp32 when
 * grad_fp32 = 1).  dk and dv sum over the query heads that share the key head.  o (bf16) and lse are
 * fa_window_fwd's for the same q, k, v, scale, window and sinks.  No atomics: the gradients are bitwise
 * repeatable.  A workspace serves one call at a time.  opts may be NULL. */
fa_status_t fa_window_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                          void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N, int Nk, int d, float scale,
                          int window, int sinks, int grad_fp32, void* workspace, size_t ws_bytes, void* stream,
                          const fa_bwd_opts* opts);

/*
 * fa_window_decode_paged -- one token of each sequence, at its last position, over the paged cache of fa_decode_paged
 * with shared heads: it sees the last `window` keys of its sequence and the first `sinks`.
 *
 *   q            [B, Hq, d] bf16, 16-byte aligned.  Hq / Hkv at most 32 (FA_ERR_UNSUPPORTED beyond).
 *   k_pages,     [num_pages, Hkv, page_size, d] bf16 pools, block_table [B, max_pages] and seq_lens [B] int32,
 *   v_pages      page_size and max_seq_len as for fa_decode_paged.  Only pages that hold a visible key are read: pages
 *                between the sinks and the window may be given back.  Any entry of the table may be read and must be readable
 *                (up to 128 pages a sequence, its whole row is); what entries without a visible key hold has no influence.  A
 *                sequence of length 0 gets O = 0 and lse = -inf.
 *   window       >= 1 (>= max_seq_len: every key);   sinks 0 .. 128.
 *   o [B, Hq, d] bf16 (fp32 with opts->o_fp32), 16-byte aligned; lse [B, Hq] fp32 (written).
 *   workspace    caller-owned scratch of fa_window_decode_paged_workspace_bytes() bytes (0 where none is needed),
 *                256-byte aligned (FA_ERR_WORKSPACE if smaller), or NULL: one kernel without partials.  O and lse are
 *                the same function of the inputs either way, up to rounding order.
 * What a page holds in rows that are not visible has no influence.  opts may be NULL.
 */
size_t fa_window_decode_paged_workspace_bytes(int B, int Hq, int Hkv, int d, int page_size, int max_pages, int max_seq_len,
                                              int window, int sinks);
fa_status_t fa_window_decode_paged(const void* q, const void* k_pages, const void* v_pages, const int* block_table,
                                   const int* seq_lens, void* o, float* lse, int B, int Hq, int Hkv, int d, int page_size,
                                   int max_pages, int num_pages, int max_seq_len, float scale, int window, int sinks,
                                   void* workspace, size_t ws_bytes, void* stream, const fa_decode_opts* opts);

/*
 * RMS norm of each head's q and k, then the rotation of fa_rope_axes, in one pass:
 *     y = R (w * x / sqrt(mean(x^2) + eps))     over the d elements of a head's row.
 *
 *   q, k      as for fa_rope_axes (Hk = 0: q alone); pos, plan likewise.
 *   q_weight, [d] bf16, or fp32 with weight_fp32 = 1; NULL: all ones.
 *   k_weight
 *   eps       finite and > 0.
 * Norm, cos, sin and products in fp32, one rounding to bf16 (nearest even); elements below 2^60 in magnitude (the squares'
 * sum has to stay in fp32).
 */

/* fa_norm_rope_axes -- q into q_out and k into k_out, in one kernel.  An output may be its own input; otherwise
 * they do not overlap. */
fa_status_t fa_norm_rope_axes(const void* q, const void* k, const void* q_weight, const void* k_weight, int weight_fp32,
                              const int* pos, void* q_out, void* k_out, int B, int Hq, int Hk, int N, float eps,
                              const fa_rope_axes_plan_t* plan, void* stream);

/* Scratch bytes of fa_norm_rope_axes_bwd's partial sums on the current device; 0 for invalid sizes or without one. */
size_t fa_norm_rope_axes_bwd_workspace_bytes(int B, int Hq, int Hk, int N, int d);

/* fa_norm_rope_axes_bwd -- from q, k (the inputs of fa_norm_rope_axes) and the gradients dq_out, dk_out of its outputs:
 *   dq, dk      [B, H, N, d] bf16 (written): the gradients of q and k.  One may be its dq_out (dk_out), or its q (k),
 *               in place; otherwise they do not overlap.
 *   dq_weight,  [d] fp32 (written), or NULL: the gradients of the weights, summed over sequences, heads and tokens.
 *   dk_weight
 *   workspace   >= fa_norm_rope_axes_bwd_workspace_bytes() bytes, 256-byte aligned; needed where a weight's gradient is
 *               wanted (FA_ERR_WORKSPACE).
 * No atomics: the gradients are bitwise repeatable. */
fa_status_t fa_norm_rope_axes_bwd(const void* q, const void* k, const void* q_weight, const void* k_weight, int weight_fp32,
                                  const int* pos, const void* dq_out, const void* dk_out, void* dq, void* dk,
                                  float* dq_weight, float* dk_weight, int B, int Hq, int Hk, int N, float eps,
                                  const fa_rope_axes_plan_t* plan, void* workspace, size_t ws_bytes, void* stream);

/*
 * fa_norm_rope_axes_paged -- the serving form: the N new tokens of each sequence.  q is normed and turned into q_out, k
 * (the same) and v [B, Hk, N, d] (copied) go into the pools [num_pages, Hk, page_size, d] at the slots that
 * fa_pages_extend gives.  q_out may be q.
 *   slots      [B, N] int64, 8-byte aligned: token n of sequence b goes to row slot % page_size of page
 *              slot / page_size.  A slot outside [0, num_pages * page_size) is no place: that token's k and v are not
 *              written.  Two tokens of one call must not share a slot.
 *   new_lens   [B] int32 or NULL: tokens from new_lens[b] on are padding, for which nothing is written (not to
 *              q_out either), as for fa_rope_axes_paged.
 */
fa_status_t fa_norm_rope_axes_paged(const void* q, const void* k, const void* v, const void* q_weight, const void* k_weight,
                                    int weight_fp32, const int* pos, void* q_out, void* k_pages, void* v_pages,
                                    const long long* slots, const int* new_lens, int B, int Hq, int Hk, int N, int page_size,
                                    int num_pages, float eps, const fa_rope_axes_plan_t* plan, void* stream);

/*
 * fa_pages_extend -- the pages of a paged cache, on the GPU: sequence b grows by new_lens[b] tokens, or shrinks by
 * -new_lens[b] (a finished request by its whole length, rejected draft tokens by their number).
 *
 *   block_table  [B, max_pages] int32, read and written: entries of new pages get their ids, those of pages given back
 *                become -1; no other entry is touched.
 *   seq_lens     [B] int32, read and written: lengths (clamped to [0, max_pages * page_size]), which grow by what is
 *                granted.
 *   new_lens     [B] int32: the change of each sequence; no sequence shrinks below 0.
 *   free_pages   [num_pages] int32, read and written: a stack of free page ids, of which the first n_free[0] count.
 *   n_free       [1] int32, read and written.
 *   granted      [B] int32 (written): the change made: new_lens[b], or 0 where a sequence would outgrow its table or
 *                the stack runs out.  Pages are handed out in the order of the sequences, each sequence's from the top
 *                of the stack down, and from the first that the stack cannot serve on, none is; a sequence whose tokens
 *                fit its last page is always served.  Fit to be the new_lens of the calls that write the tokens.
 *   slots        [B, N] int64 (written), or NULL: token n of those granted to sequence b is row slot % page_size of page
 *                slot / page_size; -1 for n >= granted[b].  N: tokens a sequence that the caller has slots for.
 * Pages given back go onto the stack once the call's own pages are taken, so that they come off again in their old
 * order: giving back what the call before granted leaves the stack as it was.  Entries given back must be
 * pages that the stack handed out: they are put on it as they are.  seq_lens, new_lens and granted are arrays of their own.
 * page_size is a positive multiple of 64.  The result does not depend on timing.
 */
fa_status_t fa_pages_extend(int* block_table, int* seq_lens, const int* new_lens, int* free_pages, int* n_free, int* granted,
                            long long* slots, int B, int N, int page_size, int max_pages, int num_pages, void* stream);

/*
 * fa_get_status -- synchronise `stream`, then read and clear the current
 * device's kernel status words (by a small kernel and a copy on `stream`, and
 * a second synchronisation).  Returns FA_ERR_TIMEOUT if any kernel of this
 * library ran out of its wait budget since the last call, FA_ERR_CUDA if a
 * synchronisation, the kernel or the copy failed, else FA_OK.
 */
fa_status_t fa_get_status(void* stream);

/* Human-readable name of a status code (static storage, never NULL). */
const char* fa_status_string(fa_status_t status);

/* Detail of the most recent error on the calling thread (static thread-local
 * storage, "" if none). */
const char* fa_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* FATTN_H */
