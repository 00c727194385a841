/*
 * kda_verify.h -- C ABI of the verification of drafted tokens against the
 * target's probabilities: the step that follows a multi-token (speculative)
 * decode (kda_decode.h, tokens_per_seq) and says which of its state slots
 * the next step starts from.
 *
 * Sequence n carries T target rows (token rows n*T .. n*T + T - 1 of the
 * multi-token step) and T - 1 drafted tokens d_0 .. d_{T-2}; p_t is target row
 * t, q_t the draft model's row that d_t was drawn from (without draft_probs,
 * q_t is 1 at d_t and 0 elsewhere).  With given uniform numbers:
 *   k = the number of leading drafts with accept_u[t] * q_t(d_t) < p_t(d_t)
 *       (exact comparison)
 *   x ~ max(p_k - q_k, 0) when draft k was refused, by inversion at
 *       sample_u[n]; p_k itself where that difference has no mass, and where
 *       no draft stands at k (all T - 1 accepted, or the drafts end)
 *   tokens[n]       = d_0 .. d_{k-1}, x, -1 ...
 *   num_accepted[n] = k
 *   next_slot[n]    = slot_idx[n][k]: the state and window after the last
 *                     token that stands, the next step's src_slot
 * A draft outside [0, V) ends the sequence's drafts (-1 is the customary
 * mark; a value >= V also sets KDA_DEVERR_TOKEN_RANGE).  A sequence whose
 * src_slot is <= 0 is padding: tokens -1, num_accepted 0, next_slot 0, and
 * its rows are not read.
 *
 * The inversion does not depend on summation order: probabilities are taken
 * into [0, 1] (NaN counts as 0), the weights max(p - q, 0), or p, are integers
 * in units of 2^-60, exact wherever p and q are 0 or at least 2^-37 and else off by at
 * most 3 units, and x is the lowest index whose inclusive running sum exceeds
 * floor(floor(sample_u * 2^31) * total / 2^31); sample_u is taken into
 * [0, 1 - 2^-31], NaN as 0.  Probabilities of a row sum to about 1, at most
 * 7 (of a row that sums to more x is some token in [0, V)).  Where a row has
 * no mass at all x is V - 1.
 */
#ifndef KDA_VERIFY_H
#define KDA_VERIFY_H

#include <stdint.h>

#include "kda_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_DEVERR_TOKEN_RANGE 32 /* a drafted token was >= V; the drafts end before it */

/* Device pointers, 4-byte aligned; probabilities are read fastest when their
 * base and strides are multiples of 16 bytes. */
typedef struct KdaVerifyArgs {
  uint32_t struct_size;        /* = sizeof(KdaVerifyArgs) */
  int32_t N;                   /* sequences */
  int32_t T;                   /* target rows per sequence, 1 .. KDA_MAX_TOKENS_PER_SEQ */
  int32_t V;                   /* vocabulary, 1 .. 2^30 */
  const int32_t* draft_tokens; /* [N][T-1]; may be NULL when T is 1 */
  const float* target_probs;   /* [N*T][target_row_stride] */
  int64_t target_row_stride;   /* elements, >= V */
  const float* draft_probs;    /* [N*(T-1)][draft_row_stride] or NULL */
  int64_t draft_row_stride;
  const float* accept_u;       /* [N][T-1]; may be NULL when T is 1 */
  const float* sample_u;       /* [N] */
  const int32_t* src_slot;     /* [N] or NULL (no padding sequences) */
  const int32_t* slot_idx;     /* [N][T] or NULL, the multi-token step's */
  int32_t* tokens;             /* [N][T] */
  int32_t* num_accepted;       /* [N] */
  int32_t* next_slot;          /* [N]; NULL exactly when slot_idx is; may be src_slot itself, no other
                                * result may overlap an input */
  int32_t* err_flag;           /* or NULL */
} KdaVerifyArgs;

/*
 * Enqueue the verification on `stream` (one launch, no workspace).  Returns
 * KDA_OK or a negative KDA_ERR_* code; on an error nothing is launched and
 * kda_last_error() describes it.  N == 0 is a no-op.
 */
int kda_verify_draft(const KdaVerifyArgs* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_VERIFY_H */
