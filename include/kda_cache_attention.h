/*
 * kda_cache_attention.h -- C ABI of causal softmax attention over the 8-bit
 * paged cache that kda_qk_rope.h writes, for the softmax layers that stand
 * between KDA layers: single tokens, multi-token (speculative) steps and
 * prompt chunks of a varlen batch.
 *
 * Sequence i holds query rows t = cu_seqlens[i] .. cu_seqlens[i+1]-1 (n_i of
 * them) and seq_lens[i] cached tokens, the queries' own among them; query j
 * sees the tokens before position
 *   limit = seq_lens[i] - n_i + j + 1.
 * For query head h, with kv head h' = h / (Hq / Hkv) and token position s in
 * block b = block_table[i][s / block_size], row s % block_size:
 *   k_s = k_code[b][h'][row] * k_scale[b][h'],  v_s likewise
 *   out[t][h] = sum_s softmax_s(sm_scale q . k_s) v_s     (s < limit)
 * A query that sees nothing gets zeros.  Rows behind cu_seqlens[B] are left
 * as they were.
 *
 * Method: the e4m3 codes go to the tensor cores as they are (fp32
 * accumulation); the other operand of each product, q and the softmax
 * weights, is split into a leading and a remaining e4m3 part:
 *   - an element of q is exact from 2^-9 of its row's largest up, and below
 *     that off by less than 2^-17 of that largest;
 *   - a weight (V's block scale folded in) is off by at most 2^-8 + 2^-12 of
 *     itself, or by 2^-18 of the largest weight of its 128-token tile where
 *     that is more: smaller weights lose their last bits one by one, and below
 *     2^-18 they add nothing to the output.  All a tile can lose that way is
 *     2^-11 of its largest weight.
 * The softmax sum adds the weights before they are rounded.  Sums, maxima and
 * the output are kept in fp32 and rounded to bf16 once.
 *
 * One kernel serves a whole call, chosen by max_new: single tokens beside a
 * long chunk run in the kernel for chunks, whose tiles they hardly fill.  Where
 * there are many, two calls are faster (a chunk of 512 tokens and 63 single
 * tokens behind 1,000 to 16,384, 48 and 8 heads: 746 us in one call, 87 and
 * 173 us in two).
 */
#ifndef KDA_CACHE_ATTENTION_H
#define KDA_CACHE_ATTENTION_H

#include <stdint.h>

#include "kda_decode.h" /* return codes, KDA_DEVERR_SLOT_RANGE, KDA_DEVERR_TIMEOUT */

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Arguments.  T = query rows of the batch, D = 128.
 *
 *   q, out      bf16 [T][row stride], Hq * D channels; 16-byte aligned, row
 *               strides multiples of 8; they must not overlap
 *   cu_seqlens  int32 [B+1], cu_seqlens[0] = 0, non-decreasing, <= T; a
 *               sequence whose bounds break this is skipped and
 *               KDA_DEVERR_SEQLENS (kda_chunk_metadata.h) is set
 *   seq_lens    int32 [B]; a value below n_i leaves the first queries without
 *               keys
 *   block_table int32 [B][block_table_stride], max_blocks entries per row.
 *               An entry outside [0, num_blocks), or past max_blocks, that a
 *               query would need sets KDA_DEVERR_SLOT_RANGE; its tokens count
 *               as absent.
 *   caches      e4m3 (bytes), strides as in kda_qk_rope.h: multiples of 16,
 *               base 16-byte aligned
 *   scales      fp32 [num_blocks][Hkv].  V scales are positive (below 2^-64
 *               they count as 2^-64) and lie within a factor of 2^96 of one
 *               another in a head.
 *   workspace   workspace_bytes >= kda_cache_attention_workspace_bytes(...),
 *               16-byte aligned; its first
 *               KDA_CACHE_ATTENTION_COUNTER_BYTES bytes are zero before the
 *               first call and every call leaves them zero again.  Calls that
 *               may overlap on the GPU need different workspaces; calls
 *               ordered on one stream may share one.  After
 *               KDA_DEVERR_TIMEOUT they have to be cleared.
 *   max_new     the largest n_i the caller expects (>= 1): chooses the
 *               kernel and its row tile; the result stays the same up to
 *               rounding
 */
typedef struct KdaCacheAttentionArgs {
  uint32_t struct_size;        /* = sizeof(KdaCacheAttentionArgs) */
  int32_t B, T;
  int32_t num_q_heads, num_kv_heads; /* num_q_heads a multiple of num_kv_heads */
  int32_t head_dim;            /* must be 128 */
  int32_t block_size;          /* 16, 32, 64, 128 or 256 */
  int32_t num_blocks, max_blocks, max_new;
  float sm_scale;              /* 0 => 1/sqrt(128) */
  const uint16_t* q;
  int64_t q_row_stride;
  uint16_t* out;
  int64_t out_row_stride;
  const int32_t* cu_seqlens;
  const int32_t* seq_lens;
  const int32_t* block_table;
  int64_t block_table_stride;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  int64_t block_stride, head_stride, token_stride;
  const float* k_scale;
  const float* v_scale;
  void* workspace;
  int64_t workspace_bytes;
  int32_t* err_flag;           /* or NULL */
} KdaCacheAttentionArgs;

#define KDA_CACHE_ATTENTION_COUNTER_BYTES 45056

/* Workspace bytes of a call with these head counts and max_new; -1 for an
 * argument out of range.  It does not grow with B, T or the lengths, and a
 * workspace for a larger max_new serves smaller ones (3 to 41 MB). */
int64_t kda_cache_attention_workspace_bytes(int32_t num_q_heads, int32_t num_kv_heads, int32_t max_new);

/*
 * Enqueue the attention on `stream` (one launch).  Returns KDA_OK or a
 * negative KDA_ERR_* code; on an error nothing is launched and
 * kda_last_error() describes it.  B == 0 or T == 0 is a no-op.  The first
 * call on a device does a once-per-device set-up: make it before any capture.
 */
int kda_cache_attention(const KdaCacheAttentionArgs* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_CACHE_ATTENTION_H */
