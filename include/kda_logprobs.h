/*
 * kda_logprobs.h -- C ABI of the log probabilities of given tokens, with the
 * entropy of their rows and the likeliest alternatives: what a serving step
 * reports beside the tokens that kda_verify.h lets stand, and what scoring a
 * given text needs.
 *
 * Row r holds V logits x (fp32 or bf16), lse = log sum_i exp(x_i):
 *   logprobs[r]        = x_tok - lse,                 tok = tokens[r]
 *   ranks[r]           = tokens ahead of tok (a larger logit, or an equal one
 *                        of a lower index; 0 is the likeliest)
 *   entropy[r]         = lse - sum_i p_i x_i          (p = exp(x - lse), 0 log 0 = 0)
 *   top_ids[r][j]      = token of rank j,             j < num_top
 *   top_logprobs[r][j] = its log probability; past the V-th: -1 and -infinity
 * A logit of -infinity is a token that is ruled out.  A row that is no
 * distribution (it holds a NaN or +infinity, or nothing above -infinity)
 * gives NaN and, for whole numbers, -1.
 * A row whose token is below 0 is not asked for (verification leaves -1
 * behind the tokens that stand): it is not read and gives 0 and, for whole
 * numbers, -1.  A token >= V does the same and sets KDA_DEVERR_TOKEN_RANGE.
 * Without tokens every row is read, and there are no logprobs and ranks.
 * Sums are fp32; results do not depend on the order in which CTAs run.
 */
#ifndef KDA_LOGPROBS_H
#define KDA_LOGPROBS_H

#include <stdint.h>

#include "kda_verify.h" /* return codes, KDA_DEVERR_TOKEN_RANGE */

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_LOGPROBS_BF16 1u /* logits are bf16 (else fp32) */
#define KDA_LOGPROBS_MAX_TOP 32

/* Device pointers, aligned to their elements.  No result may overlap an
 * input or another result. */
typedef struct KdaLogprobsArgs {
  uint32_t struct_size;        /* = sizeof(KdaLogprobsArgs) */
  int32_t R;                   /* rows; 0 is a no-op */
  int32_t V;                   /* vocabulary, 1 .. 2^30 */
  int32_t num_top;             /* 0 .. KDA_LOGPROBS_MAX_TOP */
  uint32_t flags;              /* KDA_LOGPROBS_BF16 */
  const void* logits;          /* [R][logits_row_stride] */
  int64_t logits_row_stride;   /* elements, >= V */
  const int32_t* tokens;       /* [R] or NULL */
  float* logprobs;             /* [R]; NULL exactly when tokens is, as ranks */
  int32_t* ranks;              /* [R] */
  float* entropy;              /* [R] */
  int32_t* top_ids;            /* [R][num_top]; may be NULL when num_top is 0, as top_logprobs */
  float* top_logprobs;         /* [R][num_top] */
  int32_t* err_flag;           /* or NULL */
} KdaLogprobsArgs;

/*
 * Enqueue the operator on `stream` (one launch, no workspace).  Returns
 * KDA_OK or a negative KDA_ERR_* code; on an error nothing is launched and
 * kda_last_error() describes it.  The first call on a device does a
 * once-per-device set-up: make it before any capture.
 */
int kda_logprobs(const KdaLogprobsArgs* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LOGPROBS_H */
