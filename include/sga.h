/*
 * sga.h -- C ABI of libsga.so: vocab-sharded greedy token selection for
 * speculative decoding, hand-written CUDA kernels for GB300 (sm_103a).
 *
 * The method (web pages, cited by title and section):
 *   vLLM PR #34049 "[Spec Decode] Reduce TP communication for speculative
 *     decoding draft token generation", Solution: each tensor-parallel rank
 *     takes the argmax of its own vocab shard, only (max_value, global_index)
 *     pairs are gathered, and a reduction across ranks gives the global
 *     argmax.
 *   vLLM PR #39419 "[SpecDecode] Reduce TP communication for large-vocab
 *     draft models speculative decoding", review "Refactor local argmax code":
 *     the draft-to-target id map target_id = k + d2t[k] is applied after the
 *     local argmax.
 *   vLLM PR #62604 (sharded greedy verification), Purpose item 1: per-shard
 *     statistics, all-gathered on dim 0, then ONE kernel for the global
 *     argmax, the acceptance, the bonus token and the sampled/rejected
 *     counts; item 2: the padding mask, "lowest id on ties, NaN wins, as
 *     torch.argmax"; vocabulary < 2^24.
 *
 * Tensor-parallel ranks are emulated on one GPU: shard s writes its stats to
 * rows [s*R, (s+1)*R) of one buffer, which is byte-for-byte what
 * all_gather(dim=0) of the per-rank [R] stats would produce.
 *
 * Conventions for every entry point:
 *   - Every pointer is a DEVICE pointer unless stated otherwise; the caller
 *     owns every buffer.  The library allocates no memory and keeps no state
 *     besides per-device cached kernel attributes, a device error word, and
 *     the merge slots of the decode-size LM head (see sga_lmhead_argmax).
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and the call returns without synchronising.
 *   - Arguments are validated on the host BEFORE anything is launched; a
 *     negative SGA_ERR_* means nothing was enqueued.  SGA_ERR_CUDA means a
 *     launch failed (cudaGetLastError); the CUDA error is left for the caller
 *     to inspect through cudaGetLastError/cudaPeekAtLastError semantics.
 *   - Inputs are never written.  Outputs are fully written on success.
 *   - Comparison order ("argmax order"): NaN beats every number and the
 *     lowest-id NaN wins; among numbers the larger wins (+0 and -0 are equal);
 *     equal values resolve to the lower global id.  Ids at or past org_vocab
 *     are padding and count as -inf.  A row (or shard) with no value above
 *     -inf reports its first id with value -inf.  The reported value is the
 *     winning element widened exactly to fp32 (its own bits, NaN payload
 *     kept), or -inf for a padded winner.
 */
#ifndef SGA_H
#define SGA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SGA_VERSION 100 /* 1.0.0 */

/* One per-row statistic of one shard: 8 bytes, {fp32 value bits, int32 id}. */
typedef struct sga_stat {
  float v;
  int32_t id;
} sga_stat;

/* Logits element types. */
enum sga_dtype { SGA_F32 = 0, SGA_BF16 = 1 };

/* A cudaStream_t passed as an opaque pointer. */
typedef void *sga_stream;

/* Status codes (0 = success). */
enum sga_status {
  SGA_OK = 0,
  SGA_ERR_NULL = -1,        /* a required pointer is NULL */
  SGA_ERR_SIZE = -2,        /* a size or count is negative / out of range */
  SGA_ERR_SHARD = -3,       /* shard outside the vocab or wider than the row stride */
  SGA_ERR_VOCAB = -4,       /* org_vocab <= 0, or an id would reach 2^24 */
  SGA_ERR_DTYPE = -5,       /* unknown dtype */
  SGA_ERR_ALIGN = -6,       /* pointer not aligned as the entry point requires */
  SGA_ERR_WORKSPACE = -7,   /* workspace smaller than the *_workspace() size */
  SGA_ERR_MAXK = -8,        /* max_k outside [1, SGA_MAX_K] */
  SGA_ERR_CUDA = -9,        /* a CUDA runtime call or launch failed */
  SGA_ERR_DEVICE = -10,     /* the device has no sm_103 kernels (not a GB300) */
  SGA_ERR_UNSUPPORTED = -11 /* shape outside what the kernel supports */
};

/* Largest number of drafts per request the verify kernel handles. */
#define SGA_MAX_K 15

/* Largest id + 1 any entry point accepts (the pages' vocabulary bound). */
#define SGA_MAX_VOCAB (1 << 24)

/* Library version, SGA_VERSION of the build. */
int sga_version(void);

/* Static English text for a status code; never NULL. */
const char *sga_status_string(int status);

/*
 * sga_local_argmax -- per-shard argmax with the padding mask.
 * Page: vLLM PR #34049, Solution step 1 (local argmax on each TP rank's vocab
 * shard, index made global); vLLM PR #62604, Purpose item 2 (padding mask,
 * torch.argmax order) and item 1 (per-shard statistics).
 *
 *   logits       device, rows x (>= shard_width) elements of `dtype`, row
 *                stride `ld` ELEMENTS; points at the shard's first column,
 *                i.e. element (0, shard_start) of the full matrix, or at
 *                element 0 of a separate per-rank [rows, shard_width] buffer.
 *                Must be aligned to the element size.  Any row stride and
 *                any 16-byte misalignment of the rows is handled.
 *   dtype        SGA_F32 or SGA_BF16.
 *   rows         >= 0; 0 enqueues nothing and returns SGA_OK.
 *   ld           >= shard_width.
 *   shard_start  global id of column 0 of the shard (>= 0).
 *   shard_width  > 0; shard_start + shard_width <= SGA_MAX_VOCAB.
 *   org_vocab    1 .. SGA_MAX_VOCAB; global ids >= org_vocab are padding.
 *   out_stats    device, `rows` entries, 8-byte aligned: out_stats[r] =
 *                argmax (value, GLOBAL id) of row r over the shard.  To
 *                emulate the dim-0 all-gather pass stats + s*rows.
 * Reads each non-padding logit of the shard once; padding ids are not read.
 */
int sga_local_argmax(const void *logits, int dtype, int64_t rows, int64_t ld,
                     int64_t shard_start, int64_t shard_width, int64_t org_vocab,
                     sga_stat *out_stats, sga_stream stream);

/*
 * sga_local_argmax_shards -- sga_local_argmax for several shards of one
 * logits buffer in a single launch (one GPU holding the vocab slices of
 * several tensor-parallel ranks).  Same statistics, same layout: shard s of
 * row r goes to out_stats[s*rows + r], exactly the dim-0 all-gather order.
 * Page: as sga_local_argmax (vLLM PR #34049, Solution; vLLM PR #62604,
 * Purpose items 1-2 and Test Plan: TP ranks emulated in one process with the
 * per-shard statistics concatenated in rank order).
 *
 *   logits        device; element (r, 0) holds global id shard_starts[0] of
 *                 row r; global id g sits at column g - shard_starts[0].
 *   num_shards    1 .. 64.
 *   shard_starts, shard_widths   HOST arrays of num_shards entries; shards
 *                 ascending and non-overlapping (shard_starts[s] >=
 *                 shard_starts[s-1] + shard_widths[s-1]); every width > 0;
 *                 the last shard must end at or before column ld.
 *   rows          0 .. 2^28 / num_shards.
 *   out_stats     device, num_shards * rows entries, 8-byte aligned.
 * Other arguments and the errors as sga_local_argmax.
 */
int sga_local_argmax_shards(const void *logits, int dtype, int64_t rows, int64_t ld,
                            int num_shards, const int64_t *shard_starts,
                            const int64_t *shard_widths, int64_t org_vocab,
                            sga_stat *out_stats, sga_stream stream);

/*
 * sga_block_slots -- statistics per row that sga_local_argmax_blocks writes
 * for one shard: the larger of the numbers of fixed global blocks of
 * draft_block and of bonus_block ids that meet [shard_start, shard_start +
 * shard_width).  Returns that count (>= 1), or a negative SGA_ERR_* for an
 * invalid shard or block size.  Pure host arithmetic, no CUDA call.
 */
int64_t sga_block_slots(int64_t shard_start, int64_t shard_width, int64_t draft_block,
                        int64_t bonus_block);

/*
 * sga_local_argmax_blocks -- block-granular statistics of one shard: for
 * every row, the argmax (value, GLOBAL id) of each fixed global block of ids
 * [b*B, (b+1)*B) that meets the shard, clipped to the shard; a block that
 * straddles a shard edge gives one piece on each side.
 * Page: vLLM PR #62604, Purpose item 1 (each rank reduces its shard to
 * per-block (max, token id) statistics; the blocks keep the unsharded
 * kernels' global boundaries, 8192 ids for draft positions and 1024 for the
 * bonus position, also across shard edges, so ties resolve as on the full
 * logits).
 *
 *   logits, dtype, rows, ld, shard_start, shard_width, org_vocab
 *                 as sga_local_argmax (rows <= 2^28 / slots).
 *   draft_block   block size B of the draft rows, 1 .. SGA_MAX_VOCAB.
 *   bonus_block   block size of the bonus rows, 1 .. SGA_MAX_VOCAB.
 *   num_reqs, cu_num_draft   the request layout of sga_greedy_verify
 *                 (device int32 [num_reqs + 1]; rows == cu_num_draft[num_reqs]
 *                 + num_reqs is a precondition).  Row cu_num_draft[i+1] + i
 *                 is the bonus row of request i.  cu_num_draft may be NULL:
 *                 then every row is a draft row and num_reqs is ignored.
 *   out_stats     device, slots * rows entries, 8-byte aligned, with slots =
 *                 sga_block_slots(shard_start, shard_width, draft_block,
 *                 bonus_block).  Piece p of row r (ascending ids) goes to
 *                 out_stats[p*rows + r]; a row with fewer pieces than slots
 *                 (the rows whose block size gives the smaller count) gets
 *                 (-inf, shard_start + shard_width - 1) in its remaining
 *                 slots, which never wins a reduction.  An all-padding piece
 *                 reports (-inf, its first id).
 * The stats of all shards, concatenated in shard order, go to
 * sga_shard_reduce or sga_greedy_verify with num_shards = the sum of the
 * shards' slots (at most 4096) and give the same ids as per-shard stats.
 * Errors as sga_local_argmax, plus SGA_ERR_SIZE for a block size out of range.
 */
int sga_local_argmax_blocks(const void *logits, int dtype, int64_t rows, int64_t ld,
                            int64_t shard_start, int64_t shard_width, int64_t org_vocab,
                            int64_t draft_block, int64_t bonus_block, int num_reqs,
                            const int32_t *cu_num_draft, sga_stat *out_stats,
                            sga_stream stream);

/*
 * sga_local_argmax_blocks_shards -- sga_local_argmax_blocks for several
 * shards of one logits buffer in a single launch (one GPU holding the vocab
 * slices of several tensor-parallel ranks), as sga_local_argmax_shards is
 * for per-shard statistics.  Shard s's slots follow shard s-1's: with
 * slots_s = sga_block_slots(starts[s], widths[s], draft_block, bonus_block),
 * piece p of row r of shard s goes to out_stats[(slots_0 + ... + slots_{s-1}
 * + p) * rows + r], exactly what concatenating the per-shard calls' outputs
 * in shard order gives.
 * Page: as sga_local_argmax_blocks (vLLM PR #62604, Purpose item 1).
 *
 *   logits        device; element (r, 0) holds global id shard_starts[0] of
 *                 row r; global id g sits at column g - shard_starts[0].
 *   num_shards    1 .. 64.
 *   shard_starts, shard_widths   HOST arrays, shards ascending and
 *                 non-overlapping; the last shard ends at or before column ld.
 *   rows          0 .. 2^28 / (total slots).
 *   out_stats     device, (total slots) * rows entries, 8-byte aligned.
 * Other arguments and the errors as sga_local_argmax_blocks.
 */
int sga_local_argmax_blocks_shards(const void *logits, int dtype, int64_t rows, int64_t ld,
                                   int num_shards, const int64_t *shard_starts,
                                   const int64_t *shard_widths, int64_t org_vocab,
                                   int64_t draft_block, int64_t bonus_block, int num_reqs,
                                   const int32_t *cu_num_draft, sga_stat *out_stats,
                                   sga_stream stream);

/*
 * sga_shard_reduce -- global argmax from the gathered shard statistics,
 * optionally mapped from draft ids to target ids.
 * Page: vLLM PR #34049, Solution step 3 (reduce across ranks to the global
 * argmax); vLLM PR #62604, Purpose item 2 (dim-0 all-gather layout, same
 * result as torch.argmax); vLLM PR #39419, "Refactor local argmax code"
 * (target_id = k + draft_id_to_target_id[k], after the local argmax).
 *
 *   stats       device, num_shards * rows entries, shard-major
 *               (stats[s*rows + r]); shards in ascending id order.
 *   num_shards  1 .. 4096.
 *   rows        >= 0 (0: nothing enqueued).
 *   out_vals    device fp32 [rows] (nullable): value of the winner.
 *   out_ids     device int32 [rows]: global id of the winner, after d2t.
 *   d2t         device int64 [d2t_len] or NULL.  When given, out_ids[r] =
 *               k + d2t[k] for the winning id k; an id outside [0, d2t_len)
 *               is left unmapped and sets the device error word (see
 *               sga_device_error).
 */
int sga_shard_reduce(const sga_stat *stats, int num_shards, int64_t rows, float *out_vals,
                     int32_t *out_ids, const int64_t *d2t, int64_t d2t_len,
                     sga_stream stream);

/*
 * sga_greedy_verify -- one fused kernel: cross-shard reduce of every target
 * row, greedy acceptance, bonus token and sampled/rejected counts.
 * Page: vLLM PR #62604, Purpose item 1 (one kernel finishes the global
 * argmax, acceptance, bonus token and sampled/rejected counts) and Test Plan
 * (compared with rejection_sample + get_num_sampled_and_rejected on the full
 * logits; placeholder drafts).
 *
 *   stats          device, num_shards * R_tot entries, shard-major, where
 *                  R_tot = cu_num_draft[num_reqs] + num_reqs.
 *   num_shards     1 .. 4096.
 *   num_reqs       >= 0 (0: nothing enqueued).
 *   cu_num_draft   device int32 [num_reqs + 1], cu[0] = 0, non-decreasing:
 *                  request i has K_i = cu[i+1] - cu[i] drafts and owns target
 *                  rows b_i .. b_i + K_i with b_i = cu[i] + i (K_i draft
 *                  positions, then its bonus row).  K_i must lie in
 *                  [0, max_k]; a request that breaks this gets num_sampled =
 *                  num_rejected = 0, bonus = -1, sampled all -1, and the
 *                  device error word is set.
 *   draft_tokens   device int32 [cu[num_reqs]] (may be NULL when every K_i is
 *                  0).  A negative id is a placeholder and never matches.
 *   max_k          1 .. SGA_MAX_K: row length - 1 of out_sampled.
 *   out_sampled    device int32 [num_reqs, max_k + 1]: with a_i = number of
 *                  leading drafts equal to the target argmax of their row,
 *                  entries 0..a_i are the target argmaxes of rows
 *                  b_i .. b_i + a_i, the rest -1.
 *   out_num_sampled, out_num_rejected   device int32 [num_reqs]: a_i + 1 and
 *                  K_i - a_i.
 *   out_bonus      device int32 [num_reqs]: the last emitted token, the target
 *                  argmax of row b_i + a_i.
 *   out_target_ids device int32 [R_tot] or NULL: every row's global argmax.
 * All int32 pointers must be 4-byte aligned, stats 8-byte aligned.
 */
int sga_greedy_verify(const sga_stat *stats, int num_shards, int num_reqs,
                      const int32_t *cu_num_draft, const int32_t *draft_tokens, int max_k,
                      int32_t *out_sampled, int32_t *out_num_sampled,
                      int32_t *out_num_rejected, int32_t *out_bonus,
                      int32_t *out_target_ids, sga_stream stream);

/*
 * sga_greedy_verify_prefill -- sga_greedy_verify for a batch that mixes
 * decoding requests with requests still in prefill.
 * Page: vLLM PR #62604, Test Plan (the sharded verifier handles "prefilling
 * requests").  The pages do not say what such a request yields; this library
 * reads it as: a request still in prefill emits nothing this step.
 *
 *   in_prefill     device uint8 [num_reqs] or NULL (NULL = sga_greedy_verify):
 *                  nonzero marks request i as still in prefill.  Such a
 *                  request gets out_sampled row all -1, out_num_sampled =
 *                  out_num_rejected = 0 and out_bonus = -1; the target
 *                  argmaxes of its rows still go to out_target_ids.  Its
 *                  K_i must still lie in [0, max_k] (else the K_i error
 *                  result of sga_greedy_verify applies).
 * Other arguments, results and errors as sga_greedy_verify.
 */
int sga_greedy_verify_prefill(const sga_stat *stats, int num_shards, int num_reqs,
                              const int32_t *cu_num_draft, const int32_t *draft_tokens,
                              const uint8_t *in_prefill, int max_k, int32_t *out_sampled,
                              int32_t *out_num_sampled, int32_t *out_num_rejected,
                              int32_t *out_bonus, int32_t *out_target_ids, sga_stream stream);

/*
 * sga_lmhead_argmax -- fused LM-head GEMM + per-shard argmax: the shard's
 * logits hidden . weight_shard^T are computed on the tensor cores (tcgen05,
 * fp32 accumulation in tensor memory) and reduced to per-row statistics in
 * the epilogue; the logits are never written to global memory.
 * Page: vLLM PR #62604, Purpose (vocab-parallel LM head: each rank holds a
 * vocab slice of the weight) and item 2 (fused get_top_tokens); vLLM PR
 * #39419, Changes (get_top_tokens on the model: lm_head applied to the hidden
 * states, then the local argmax).
 *
 *   hidden        device bf16 [M, H] row-major (row stride H), 16-byte aligned.
 *   M             0 .. 1048576 (0: nothing enqueued).
 *   H             hidden size: a positive multiple of 64.
 *   weight_shard  device bf16 [shard_width, H] row-major, 16-byte aligned; row j
 *                 holds global id shard_start + j.
 *   shard_start, shard_width, org_vocab   as for sga_local_argmax.
 *   out_stats     device [M], 8-byte aligned: argmax (value, global id) of
 *                 each row's logits over the shard.  The value is the fp32
 *                 accumulator of the winning logit; accumulation order is
 *                 the kernel's, so values match an exact dot product only to
 *                 fp32 rounding and near-ties may resolve to either id.
 *   workspace     device, >= sga_lmhead_argmax_workspace(M, shard_width)
 *                 bytes, 8-byte aligned; holds partial statistics.
 *                 Contents on entry are ignored; the caller must not use it
 *                 concurrently from two calls.  Unused for M <= 128.
 * Decode sizes (M <= 128; one CTA per SM up to M = 64, CTA pairs above):
 * one kernel launch, whose CTAs merge their per-row
 * winners in library-owned device memory (32 merge slots per device, one
 * taken per call in turn; the last CTA writes out_stats and clears the
 * slot).  Calls whose kernels overlap on the GPU must not share a slot: at
 * most 32 decode-size LM-head calls (of any LM-head entry point) may be in
 * flight on one device at once, and a captured graph that holds such a call
 * must not be replayed concurrently with itself.
 * Requires a GPU of compute capability 10.3 (SGA_ERR_DEVICE otherwise).
 */
size_t sga_lmhead_argmax_workspace(int64_t M, int64_t shard_width);
int sga_lmhead_argmax(const void *hidden, int64_t M, int64_t H, const void *weight_shard,
                      int64_t shard_start, int64_t shard_width, int64_t org_vocab,
                      sga_stat *out_stats, void *workspace, size_t workspace_bytes,
                      sga_stream stream);

/*
 * sga_lmhead_argmax_fp8 -- sga_lmhead_argmax with FP8 (OCP E4M3, "e4m3fn")
 * operands: hidden states and the weight shard stored as E4M3 codes (one byte
 * each) with a positive scale per hidden row and one positive weight scale.
 * logit[r][j] = hidden_scale[r] * weight_scale * sum_k h[r][k] * w[j][k].
 * Positive scales cannot change which id is the argmax of a row, so the
 * tensor cores (tcgen05 kind::f8f6f4, fp32 accumulation) work on the raw
 * codes and only the reported value is scaled.
 * Page: as sga_lmhead_argmax (vLLM PR #62604, Purpose; PR #39419, Changes);
 * FP8 models are the pages' workloads (vLLM PR #34049, Test Plan:
 * Llama 4 Maverick FP8), an fp8 LM head is this library's extension.
 *
 *   hidden_q      device uint8 [M, H] E4M3 codes, 16-byte aligned.
 *   hidden_scale  device fp32 [M] (nullable: all 1), 4-byte aligned; each
 *                 scale must be positive and finite (not checked).
 *   H             a positive multiple of 128.
 *   weight_q      device uint8 [shard_width, H] E4M3 codes, 16-byte aligned.
 *   weight_scale  host value, positive and finite (SGA_ERR_SIZE otherwise).
 *   workspace     as sga_lmhead_argmax (same size function).
 * The reported value is fp32(acc) * (hidden_scale[r] * weight_scale).
 */
int sga_lmhead_argmax_fp8(const void *hidden_q, const float *hidden_scale, int64_t M, int64_t H,
                          const void *weight_q, float weight_scale, int64_t shard_start,
                          int64_t shard_width, int64_t org_vocab, sga_stat *out_stats,
                          void *workspace, size_t workspace_bytes, sga_stream stream);

/*
 * sga_lmhead_argmax_shards -- sga_lmhead_argmax for several vocab shards of
 * one weight buffer in a single call (one GPU holding the vocab slices of
 * several tensor-parallel ranks), as sga_local_argmax_shards is for the
 * per-shard argmax.  At decode sizes (M <= 128) every shard runs in one
 * launch of a decode-size kernel, whose CTAs merge in library-owned memory
 * as in sga_lmhead_argmax (same 32-call limit); from M = 129 every shard
 * runs in one GEMM launch followed by one finalize launch.  The statistics
 * are identical to num_shards sga_lmhead_argmax calls.
 * Page: as sga_lmhead_argmax (vLLM PR #62604, Purpose; PR #39419, Changes).
 *
 *   weight        device [rows, H] (bf16), 16-byte aligned; row g -
 *                 shard_starts[0] holds global id g (the buffer spans every
 *                 shard, and any gap between them).
 *   num_shards    1 .. 64.
 *   shard_starts, shard_widths   HOST arrays, shards ascending and
 *                 non-overlapping, each as sga_lmhead_argmax's.
 *   out_stats     device, num_shards * M entries, 8-byte aligned: shard s's
 *                 stats at out_stats[s * M + r] (the gathered layout).
 *   workspace     device, >= sga_lmhead_argmax_shards_workspace(M,
 *                 num_shards, shard_widths) bytes, 8-byte aligned, as
 *                 sga_lmhead_argmax's.
 * Other arguments and the errors as sga_lmhead_argmax.
 */
size_t sga_lmhead_argmax_shards_workspace(int64_t M, int num_shards, const int64_t *shard_widths);
int sga_lmhead_argmax_shards(const void *hidden, int64_t M, int64_t H, const void *weight,
                             int num_shards, const int64_t *shard_starts,
                             const int64_t *shard_widths, int64_t org_vocab,
                             sga_stat *out_stats, void *workspace, size_t workspace_bytes,
                             sga_stream stream);

/*
 * sga_lmhead_argmax_shards_fp8 -- sga_lmhead_argmax_shards with the E4M3
 * operands of sga_lmhead_argmax_fp8: one weight_scale for the whole weight
 * buffer; otherwise as sga_lmhead_argmax_fp8 and sga_lmhead_argmax_shards.
 */
int sga_lmhead_argmax_shards_fp8(const void *hidden_q, const float *hidden_scale, int64_t M,
                                 int64_t H, const void *weight_q, float weight_scale,
                                 int num_shards, const int64_t *shard_starts,
                                 const int64_t *shard_widths, int64_t org_vocab,
                                 sga_stat *out_stats, void *workspace, size_t workspace_bytes,
                                 sga_stream stream);

/*
 * sga_lmhead_argmax_noalloc -- sga_lmhead_argmax for callers that must not
 * allocate device memory.  The pages have no counterpart to this entry point.
 *
 * Some callers of this code cannot call cudaMalloc on their decode path: an
 * inference server or framework plugin that owns a device memory pool sized
 * at start-up and forbids allocations outside it, or a latency-critical loop
 * where cudaMalloc/cudaFree would synchronise the device.  Such a caller may
 * have no way to provide the workspace that sga_lmhead_argmax needs.  This
 * entry point takes the same inputs and outputs but keeps its per-tile
 * partial statistics in a fixed scratch array inside the library's device
 * image (SGA_LMHEAD_NOALLOC_SCRATCH_BYTES = 4 MiB, held on every GPU that
 * loads the library until the process exits).  It calls no allocating
 * routine.
 *
 *   Arguments and results: as sga_lmhead_argmax, without workspace.
 *   Limit: sga_lmhead_argmax_workspace(M, shard_width) must not exceed
 *          SGA_LMHEAD_NOALLOC_SCRATCH_BYTES (M * P * 8 bytes, P partials per
 *          row: for M >= 129 P = min(ceil(shard_width / 256), 128); for
 *          M <= 128, where the scratch is not used, P =
 *          max(ceil(shard_width / 256), min(ceil(shard_width / 128), 256)));
 *          larger calls return SGA_ERR_WORKSPACE and enqueue nothing.
 *   Set-up: the first call on a device looks up the device address of the
 *          scratch array for that device (with that device current), so make
 *          the first call on each device before any stream capture.  The
 *          address is looked up again when the device's current context has
 *          changed (after cudaDeviceReset, for instance); make the first call
 *          after such a change outside any stream capture as well.
 *   Sharing: every call on a device uses the same scratch array, which keeps
 *          the last call's contents; each call writes every scratch entry it
 *          reads, so nothing has to start at zero.  Calls whose kernels
 *          overlap on the GPU (different streams, no ordering between them)
 *          race on the scratch array and may return wrong results.
 */
#define SGA_LMHEAD_NOALLOC_SCRATCH_BYTES (4u << 20)
int sga_lmhead_argmax_noalloc(const void *hidden, int64_t M, int64_t H,
                              const void *weight_shard, int64_t shard_start,
                              int64_t shard_width, int64_t org_vocab, sga_stat *out_stats,
                              sga_stream stream);

/*
 * sga_linear -- matrix product with bias, activation and residual in its
 * epilogue, on the tensor cores (bf16 operands, fp32 accumulation):
 *   z = x . weight^T + bias,   out = act(z) + residual.
 * A draft head is out = x + act(weight x + bias) in front of the LM head;
 * the LM head's logits themselves are the product alone.  (The pages take
 * hidden states and logits as given; this is the library's extension.)
 *
 *   x            device bf16 [M, K], row stride ldx >= K elements.
 *   weight       device bf16 [N, K], row stride ldw >= K elements.
 *                x and weight 16-byte aligned, ldx, ldw and K multiples of 8.
 *   M            0 .. 1048576 (0: nothing enqueued).
 *   N            1 .. SGA_MAX_VOCAB.    K   8 .. 1048576.
 *   bias         device fp32 or bf16 [N] (bias_dtype), nullable.
 *   act          one of enum sga_act.
 *   residual     device bf16 [M, N], row stride ldr >= N, nullable.
 *   out_preact   device bf16 [M, N], row stride ldp >= N, nullable: z, which
 *                sga_linear_grad needs when there is an activation.
 *   out          device bf16 [M, N], row stride ldo >= N.  May be the residual
 *                buffer itself (ldo == ldr); any other overlap is not allowed.
 * residual, out_preact, out: 2-byte aligned, any stride.  z is rounded to bf16
 * for out_preact only; out is rounded once.  Errors: SGA_ERR_SIZE (sizes and
 * strides), SGA_ERR_UNSUPPORTED (act), SGA_ERR_DTYPE (bias_dtype),
 * SGA_ERR_NULL, SGA_ERR_ALIGN.  One kernel launch, no workspace.
 */
enum sga_act {
  SGA_ACT_NONE = 0,
  SGA_ACT_RELU = 1,
  SGA_ACT_SILU = 2,     /* z / (1 + e^-z) */
  SGA_ACT_GELU = 3,     /* z (1 + erf(z / sqrt 2)) / 2 */
  SGA_ACT_GELU_TANH = 4 /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
};
int sga_linear(const void *x, int64_t M, int64_t K, int64_t ldx, const void *weight, int64_t N,
               int64_t ldw, const void *bias, int bias_dtype, int act, const void *residual,
               int64_t ldr, void *out_preact, int64_t ldp, void *out, int64_t ldo,
               sga_stream stream);

/*
 * sga_linear_grad -- gradient of sga_linear: with g the gradient of out,
 *   dz = g act'(z),  grad_x = dz . weight,  grad_weight = dz^T . x,
 *   grad_bias = sum over rows of dz          (the residual's gradient is g).
 * relu's dz is g where z > 0, 0 where z <= 0 (whatever g is there).
 *
 *   grad_out     device bf16 [M, N], row stride ldg >= N, 2-byte aligned.
 *   preact       device bf16 [M, N], row stride ldp >= N, 2-byte aligned: z
 *                from the forward pass; may be NULL iff act is SGA_ACT_NONE.
 *   x, weight    as sga_linear (both are always given).
 *   grad_x       device bf16 [M, K], row stride ldgx >= K, nullable.
 *   grad_weight  device bf16 [N, K], row stride ldgw >= K, nullable.
 *   grad_bias    device fp32 or bf16 [N] (bias_dtype), nullable; summed in
 *                fp32 from unrounded dz, in a fixed order.
 *   workspace    device, >= sga_linear_grad_workspace(M, N, K) bytes, 16-byte
 *                aligned; contents on entry are ignored; not to be used by two
 *                calls at once.
 * dz is rounded to bf16 as the products' operand.  M = 0 writes zeros to
 * grad_weight and grad_bias.  No output may overlap an input.  Errors as
 * sga_linear, and SGA_ERR_WORKSPACE.
 */
size_t sga_linear_grad_workspace(int64_t M, int64_t N, int64_t K);
int sga_linear_grad(const void *grad_out, int64_t M, int64_t N, int64_t ldg, const void *preact,
                    int64_t ldp, int act, const void *x, int64_t K, int64_t ldx,
                    const void *weight, int64_t ldw, void *grad_x, int64_t ldgx,
                    void *grad_weight, int64_t ldgw, void *grad_bias, int bias_dtype,
                    void *workspace, size_t workspace_bytes, sga_stream stream);

/*
 * sga_token_logprobs -- log probabilities of given tokens over a whole
 * vocabulary, with each row's entropy and best alternatives: what a server
 * reports beside the greedy ids, and the loss of a draft model in training.
 * (The pages stop at the ids; this is the library's extension, on the same
 * row, shard and padding conventions.)
 *
 * With x the row's logits of ids below org_vocab, lse = log sum_j e^x_j:
 *   logprob = x_token - lse,   entropy = lse - sum_j e^(x_j - lse) x_j,
 *   alternatives: the top_k best ids in the argmax order, each with x - lse.
 * Sums are kept in fp32 relative to the row's maximum.
 *
 *   logits       as sga_local_argmax, column 0 = global id 0.
 *   vocab        columns of a row, 1 .. SGA_MAX_VOCAB; ld >= vocab.
 *   org_vocab    1 .. SGA_MAX_VOCAB; ids >= org_vocab are padding, not read.
 *   tokens       device int32 [rows] or NULL.  A negative token is no token:
 *                its log probability is 0.  A token >= org_vocab (or one whose
 *                logit is -inf) has log probability -inf.
 *   top_k        0 .. SGA_MAX_TOP.
 *   out_logprob, out_entropy, out_lse   device fp32 [rows], each nullable.
 *   out_top_ids, out_top_logprobs   device int32 / fp32 [rows, top_k], each
 *                nullable: best first, equal logits by ascending id (-inf
 *                logits included); with fewer than top_k ids below org_vocab
 *                the rest are id -1, log probability -inf.
 * A row with no logit above -inf has lse -inf, entropy 0 and every log
 * probability -inf (a negative token's stays 0).  A row holding a NaN or +inf
 * has NaN for lse, entropy and every log probability (a negative token's stays
 * 0); its alternatives' ids keep the argmax order.
 * fp32 and int32 pointers must be 4-byte aligned.  One kernel launch.
 * Errors: SGA_ERR_DTYPE, SGA_ERR_SIZE (rows or top_k), SGA_ERR_VOCAB,
 * SGA_ERR_SHARD (ld < vocab), SGA_ERR_NULL (logits), SGA_ERR_ALIGN.
 */
#define SGA_MAX_TOP 32
int sga_token_logprobs(const void *logits, int dtype, int64_t rows, int64_t ld, int64_t vocab,
                       int64_t org_vocab, const int32_t *tokens, int top_k, float *out_logprob,
                       float *out_entropy, float *out_lse, int32_t *out_top_ids,
                       float *out_top_logprobs, sga_stream stream);

/* A row's statistics over one vocab shard: the maximum, sum_j e^(x_j - max),
 * sum_j (x_j - max) log2(e) e^(x_j - max), and the token's logit (-inf when
 * the token is not an id of the shard).  A shard with no logit above -inf has
 * max -inf (its sums are not used). */
typedef struct sga_logprob_part {
  float max, sum, wsum, token;
} sga_logprob_part;

/*
 * sga_local_logprobs -- the part of sga_token_logprobs that one vocab shard
 * (one tensor-parallel rank) contributes; the parts of all shards, gathered
 * on dim 0, go to sga_logprob_reduce.
 *
 *   logits, dtype, rows, ld, shard_start, shard_width, org_vocab
 *                as sga_local_argmax.
 *   tokens       device int32 [rows] GLOBAL ids, or NULL, as above.
 *   out_parts    device [rows], 4-byte aligned.
 *   out_top      device [rows, top_k], 8-byte aligned: the shard's best
 *                (logit, GLOBAL id), best first; entries past the shard's
 *                non-padding ids are (-inf, 0x7fffffff).  NULL iff top_k is 0.
 */
int sga_local_logprobs(const void *logits, int dtype, int64_t rows, int64_t ld,
                       int64_t shard_start, int64_t shard_width, int64_t org_vocab,
                       const int32_t *tokens, int top_k, sga_logprob_part *out_parts,
                       sga_stat *out_top, sga_stream stream);

/*
 * sga_logprob_reduce -- joins the gathered parts of all shards into the
 * results of sga_token_logprobs.
 *
 *   parts        device, num_shards * rows entries, shard-major.
 *   tops         device, num_shards * rows * top_k entries, shard-major (NULL
 *                iff top_k is 0); shards in ascending id order.
 *   num_shards   1 .. 4096.
 *   tokens       the tokens given to sga_local_logprobs (they tell a row
 *                without a token from one whose token has no probability).
 * Outputs as sga_token_logprobs.
 */
int sga_logprob_reduce(const sga_logprob_part *parts, const sga_stat *tops, int num_shards,
                       int64_t rows, int top_k, const int32_t *tokens, float *out_logprob,
                       float *out_entropy, float *out_lse, int32_t *out_top_ids,
                       float *out_top_logprobs, sga_stream stream);

/*
 * sga_token_logprobs_grad -- gradient of the log probabilities, the entropy
 * and the alternatives' log probabilities with respect to the logits, over
 * the whole vocabulary or one shard of it (no exchange: the row's lse and
 * entropy carry what the other shards hold).  With p_j = e^(x_j - lse):
 *   grad_j = [j = token] g_logprob + sum_i [j = top_ids_i] g_top_i
 *            - p_j (g_logprob + sum_i g_top_i) - g_entropy p_j (x_j - lse + entropy)
 *
 *   logits, dtype, rows, ld, shard_start, shard_width, org_vocab
 *                as sga_local_argmax.
 *   tokens       device int32 [rows] or NULL: global ids, as above (a negative
 *                token has no gradient).
 *   lse, entropy device fp32 [rows] from the forward pass; entropy may be NULL
 *                iff grad_entropy is.
 *   grad_logprob, grad_entropy   device fp32 [rows], nullable (no gradient).
 *   top_ids, grad_top   device [rows, top_k]; NULL iff top_k is 0.  Ids may
 *                repeat and may be the token; a negative id is skipped.
 *   out_grad     device, rows x shard_width elements of `dtype`, row stride
 *                ldg >= shard_width elements, aligned to the element; padding
 *                ids get 0.  May be the logits buffer itself (ldg == ld); any
 *                other overlap is not allowed.
 * A row whose lse is -inf gets 0 everywhere.
 */
int sga_token_logprobs_grad(const void *logits, int dtype, int64_t rows, int64_t ld,
                            int64_t shard_start, int64_t shard_width, int64_t org_vocab,
                            const int32_t *tokens, const float *lse, const float *entropy,
                            const float *grad_logprob, const float *grad_entropy, int top_k,
                            const int32_t *top_ids, const float *grad_top, void *out_grad,
                            int64_t ldg, sga_stream stream);

/*
 * sga_probs -- the probabilities of logits rows at a temperature, over a whole
 * vocabulary: what sga_sampled_verify reads, of the target's rows and of the
 * draft model's.  Here and in the calls below vocab shards are gathered first.
 * (The pages verify greedily; this is the library's extension.)
 *   p_j = e^((x_j - max) / T) / sum_i e^((x_i - max) / T)
 *
 *   logits, dtype, rows, ld, vocab, org_vocab   as sga_token_logprobs.
 *   temperature  device fp32 [rows], finite, or NULL (1 everywhere).  0 is a
 *                greedy row: 1 at its argmax (see "argmax order" above), 0
 *                elsewhere.  A negative or NaN temperature makes the row NaN.
 *   out_probs    device fp32, rows x vocab elements, row stride ldp >= vocab,
 *                4-byte aligned; padding ids get 0.  May be the buffer of fp32
 *                logits itself (ldp == ld); any other overlap is not allowed.
 * At a temperature above 0 a row with no logit above -inf is 0 everywhere, and
 * a row holding a NaN or +inf is NaN (but for its padding ids).  One launch.
 * Equal calls give equal results; the order of a row's sum, and so its last bits,
 * goes by the sizes and alignments.
 * Errors: SGA_ERR_DTYPE, SGA_ERR_SIZE (rows), SGA_ERR_VOCAB, SGA_ERR_SHARD
 * (ld or ldp < vocab), SGA_ERR_NULL, SGA_ERR_ALIGN.
 */
int sga_probs(const void *logits, int dtype, int64_t rows, int64_t ld, int64_t vocab,
              int64_t org_vocab, const float *temperature, float *out_probs, int64_t ldp,
              sga_stream stream);

/*
 * sga_sampled_verify -- verification of drafted tokens by rejection sampling:
 * sga_greedy_verify for requests that are sampled, from the target's and the
 * draft model's probabilities and given uniform random numbers.  The emitted
 * tokens are distributed as the target's, as finely as the uniforms are: fp32
 * numbers of 24 bits step by 6e-8 of a row's sum, and ids of about that probability
 * and less are drawn too often or never (of the 152064 ids of a softmax row with
 * N(0, 2.5^2) logits 17 % never, which have 0.04 % of the probability; the total
 * variation is 0.15 %).
 * (The pages verify greedily; this is the library's extension, on the same
 * request layout and outputs.)
 *
 * Draft t of a row with target probabilities p, draft probabilities q and
 * uniform u is accepted when fl(u q_t) < p_t (fp32), up to the first one that
 * is not.  There a token is drawn from w_j = max(fl(p_j - q_j), 0), or from w = p
 * where those are all 0; with every draft accepted it is drawn from the bonus
 * row's p.  Drawing: weights count in whole units of 2^-38 (w clamped to [0, 1]
 * and rounded to the nearest unit, NaN counts as 0), S_j = w_0 + ... + w_j in
 * 64-bit integers, and the token is the first j with S_j > min(floor(u S), S - 1),
 * S the total and u S a product of doubles (u = sample_u below, counted as 0 when
 * it is negative or NaN).  The sums are exact, so the ids do not depend on how
 * the row is split, and tokens of weight 0 are never drawn.
 * A row of ones and zeros (sga_probs at temperature 0) gives the greedy result
 * of sga_greedy_verify where the draft's rows are of that kind as well (or
 * draft_probs is NULL).
 *
 *   target_probs  device fp32, rows x vocab, row stride ldt >= vocab: row
 *                 cu[i] + i + j is position j of request i, as sga_greedy_verify.
 *   rows          D + num_reqs, D = cu_num_draft[num_reqs] the number of drafts;
 *                 num_reqs .. 2^28.
 *   draft_probs   device fp32, D x vocab, row stride ldd >= vocab: row cu[i] + j
 *                 is what draft j of request i was sampled from.  NULL: drafts
 *                 proposed without probabilities, q = 1 at the draft, 0 elsewhere.
 *   vocab         1 .. SGA_MAX_VOCAB (leave out padding ids, or give them 0).
 *   num_reqs      >= 0 (0: nothing enqueued).
 *   cu_num_draft  device int32 [num_reqs + 1], as sga_greedy_verify.  A request
 *                 with K_i outside [0, max_k] or with rows outside of `rows` emits
 *                 nothing and sets SGA_DEVERR_K_RANGE.
 *   draft_tokens  device int32 [D] (may be NULL when D is 0).  An id outside
 *                 [0, vocab) is a placeholder: not accepted, and q counts as 0.
 *   in_prefill    device uint8 [num_reqs] or NULL, as sga_greedy_verify_prefill.
 *   accept_u      device fp32 [D], uniform in [0, 1) (may be NULL when D is 0).
 *   sample_u      device fp32 [num_reqs], uniform in [0, 1).
 *   max_k         1 .. SGA_MAX_K.
 *   out_sampled   device int32 [num_reqs, max_k + 1]: the a_i accepted drafts,
 *                 the drawn token, then -1.  A row without any weight draws -1.
 *   out_num_sampled, out_num_rejected, out_last   device int32 [num_reqs]:
 *                 a_i + 1, K_i - a_i and the drawn token.
 * All pointers must be 4-byte aligned (in_prefill: none).  One launch.
 * Errors: SGA_ERR_MAXK, SGA_ERR_SIZE (num_reqs, rows), SGA_ERR_VOCAB,
 * SGA_ERR_SHARD (ldt or ldd < vocab), SGA_ERR_NULL, SGA_ERR_ALIGN.
 */
int sga_sampled_verify(const float *target_probs, int64_t rows, int64_t ldt,
                       const float *draft_probs, int64_t ldd, int64_t vocab, int num_reqs,
                       const int32_t *cu_num_draft, const int32_t *draft_tokens,
                       const uint8_t *in_prefill, const float *accept_u, const float *sample_u,
                       int max_k, int32_t *out_sampled, int32_t *out_num_sampled,
                       int32_t *out_num_rejected, int32_t *out_last, sga_stream stream);

/*
 * sga_distill -- the divergence of a draft model's rows from a teacher's top
 * logits (of a target model, as sga_token_logprobs lists them), with or without
 * its gradient with respect to the draft's logits in the same pass.  (The pages
 * take trained draft models as given; this is the library's extension.)
 *
 * With y = x / T of the row's logits x, s_j = e^(y_j - lse) (lse the log-sum-exp
 * of y over ids below org_vocab), and the teacher's entries (id_i, z_i):
 *   without teacher_lse: p_i = e^(z_i / T) / sum of those of the list, p_r = 0;
 *   with teacher_lse:    p_i = e^(z_i / T - teacher_lse), p_r = max(0, 1 - sum p_i),
 *                        the teacher's probability of all ids off the list;
 *   loss = sum_i p_i (log p_i - log s_id_i) + p_r (log p_r - log s_r),
 *   s_r = e^(lse_rest - lse), lse_rest the log-sum-exp of y over ids off the list;
 *   grad_j = grad_loss / T ((sum_i p_i + p_r) s_j - sum over id_i = j of p_i
 *            - [j off the list] p_r e^(y_j - lse_rest)).
 * (Soft targets at T > 1 are often weighted by T^2: give that in grad_loss.)
 *
 *   logits, dtype, rows, ld, vocab, org_vocab   as sga_token_logprobs.
 *   teacher_ids, teacher_logits   device int32 / fp32 [rows, k]: ids in any
 *                order.  An id outside [0, org_vocab) is no entry (it counts to
 *                the rest).  Entries of the same id each count.  A row without
 *                an entry (or whose list has no weight, without teacher_lse)
 *                has loss 0 and gradient 0 whatever its logits are.
 *   k            1 .. SGA_MAX_TEACHER.
 *   teacher_lse  device fp32 [rows] or NULL: log-sum-exp of the teacher's
 *                logits / T (zeros where teacher_logits are log probabilities
 *                and T is 1).
 *   temperature  T, 1e-6 .. 1e6.
 *   out_loss, out_lse, out_lse_rest   device fp32 [rows], each nullable.
 *   grad_loss    device fp32 [rows] or NULL (ones): upstream gradients.
 *   out_grad     device, rows x vocab elements of `dtype`, row stride ldg >=
 *                vocab, or NULL; padding ids get 0.  May be the logits buffer
 *                itself (ldg == ld); any other overlap is not allowed.
 * An entry with p_i > 0 on a logit of -inf makes the loss +inf (its gradient
 * stays finite); p_r is left out (0) where the row has no logit above -inf off
 * the list.  A row with no logit above -inf has lse -inf and gradient 0; one
 * holding a NaN or +inf has NaN for its lse, loss and gradient.  One launch.
 * Equal calls give equal results; the order of a row's sums, and so their last
 * bits, goes by the sizes and alignments and by whether a gradient is asked for.
 * Errors: SGA_ERR_DTYPE, SGA_ERR_SIZE (rows, k, temperature), SGA_ERR_VOCAB,
 * SGA_ERR_SHARD (ld or ldg < vocab), SGA_ERR_NULL, SGA_ERR_ALIGN.
 */
#define SGA_MAX_TEACHER 128
int sga_distill(const void *logits, int dtype, int64_t rows, int64_t ld, int64_t vocab,
                int64_t org_vocab, const int32_t *teacher_ids, const float *teacher_logits, int k,
                const float *teacher_lse, float temperature, float *out_loss, float *out_lse,
                float *out_lse_rest, const float *grad_loss, void *out_grad, int64_t ldg,
                sga_stream stream);

/*
 * sga_distill_grad -- the gradient of sga_distill from the lse and lse_rest
 * that it gave, for losses whose upstream gradient is known later.
 *   lse          device fp32 [rows].
 *   lse_rest     device fp32 [rows]; may be NULL iff teacher_lse is.
 *   out_grad     as sga_distill, not NULL.
 * The sums are rounded to fp32, which costs s_j and the rest's term up to 2^-23
 * (|lse| + |lse_rest|) of themselves.  In a row whose lse (or, with teacher_lse,
 * lse_rest) is above 512 in size, or infinite other than by logits of -inf, they hold too
 * little, or nothing, of the sum of exponentials (a rest masked by -1e9, a low
 * temperature): such a row's sums are taken anew from its logits, by one CTA,
 * which reads the row twice.
 * Other arguments, results and errors as sga_distill.
 */
int sga_distill_grad(const void *logits, int dtype, int64_t rows, int64_t ld, int64_t vocab,
                     int64_t org_vocab, const int32_t *teacher_ids, const float *teacher_logits,
                     int k, const float *teacher_lse, float temperature, const float *lse,
                     const float *lse_rest, const float *grad_loss, void *out_grad, int64_t ldg,
                     sga_stream stream);

/*
 * Device error word of the current device.  Kernels OR bits into it instead
 * of trapping: SGA_DEVERR_K_RANGE (a request's K_i outside [0, max_k], or in
 * sga_sampled_verify its rows outside of the given ones),
 * SGA_DEVERR_D2T_RANGE (a winning id outside the d2t table),
 * SGA_DEVERR_TIMEOUT (a bounded wait inside a pipelined kernel gave up; its
 * outputs are not valid), SGA_DEVERR_LAYOUT (sga_local_argmax_blocks[_shards]:
 * a request of cu_num_draft names rows outside [0, rows) or ends before it
 * starts; that request's statistics are not written, and with a decreasing
 * cu_num_draft the other requests' statistics are not valid either).  sga_device_error synchronises the current device
 * and copies the word to *out_word (host pointer); sga_clear_device_error
 * synchronises and zeroes it.  Both return SGA_OK or SGA_ERR_CUDA.
 */
#define SGA_DEVERR_K_RANGE 1u
#define SGA_DEVERR_D2T_RANGE 2u
#define SGA_DEVERR_TIMEOUT 4u
#define SGA_DEVERR_LAYOUT 8u
int sga_device_error(uint32_t *out_word);
int sga_clear_device_error(void);

/*
 * sga_selftest_wait_timeout -- exercises the bounded waits that the
 * pipelined kernels of this library use (the pages have no counterpart): a
 * thread and a warp, in the two forms of the wait, wait on a shared-memory
 * mbarrier that nothing arrives at; after limit_ns (1 us .. 1 s) they give up,
 * and a second warp leaves its wait on the abort flag that the first raises.
 * If all did, none before limit_ns, SGA_DEVERR_TIMEOUT is OR-ed into the device
 * error word; the kernel returns normally.  waited_ns (device, nullable, 8-byte
 * aligned) receives the time the longest wait took.  The context stays usable:
 * no trap, no fault.
 */
int sga_selftest_wait_timeout(uint64_t limit_ns, uint64_t *waited_ns, sga_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* SGA_H */
