/*
 * kda_linear.h -- C ABI of a matrix product with a fused epilogue: the
 * projections in front of and behind the KDA and softmax layers, the
 * feed-forward blocks, and the head that makes the logits.
 *
 *   y[m][n]   = x_scale[m] * weight_scale[n] * sum_k x[m][k] weight[n][k] + bias[n]
 *   out[m][n] = act(y[m][n]) + residual[m][n],                n < N
 * with act the identity, silu(y) = y / (1 + e^-y), or gelu(y) = y (1 +
 * erf(y / sqrt 2)) / 2; gated, with H = N / 2:
 *   out[m][n] = silu(y[m][n]) * y[m][H + n] + residual[m][n], n < H
 * x and weight are both bf16 (no scales), or both e4m3 with one scale per row
 * of each, as kda_add_norm.h makes them.  Products are exact and summed in
 * fp32 (by tensor cores, which cut sums towards zero: fp32 results from short
 * sums, so that they are off by no more than about 2^-20 of sums without much
 * cancellation); the epilogue is fp32 and rounded once, to out's type (silu's
 * values below 2^-119 come out as 0).  A row of x that
 * is not finite, or whose scale is NaN, reaches no other row.
 */
#ifndef KDA_LINEAR_H
#define KDA_LINEAR_H

#include <stdint.h>

#include "kda_decode.h" /* return codes, KDA_DEVERR_TIMEOUT */

#ifdef __cplusplus
extern "C" {
#endif

/* activation */
#define KDA_ACT_NONE 0
#define KDA_ACT_SILU 1
#define KDA_ACT_GELU 2
#define KDA_ACT_SILU_GATED 3

/* flags */
#define KDA_LINEAR_E4M3 1u         /* x and weight are e4m3 (else bf16) */
#define KDA_LINEAR_OUT_F32 2u      /* out is fp32 (else bf16) */
/* The kernel directly ahead of this one in the stream does not write weight,
 * weight_scale or bias: they may be read while it still runs.  (Kernels ahead
 * of that one may: they have ended by then, as this library's kernels launch
 * dependents only when all that is ahead of them has.  Behind a kernel of
 * another library that launches dependents sooner than that, the promise is
 * about whatever may still be running ahead of it too.) */
#define KDA_LINEAR_EARLY_WEIGHT 4u

/*
 * Arguments.  x and weight are 16-byte aligned and their row strides
 * multiples of 16 bytes; scales, bias and err_flag 4-byte, residual 2-byte
 * aligned, out to its elements.  (out and residual are accessed fastest when
 * their bases and row strides are multiples of 16 bytes.)  out may be
 * residual itself where both are bf16 and the strides are the same; otherwise
 * out may not overlap an input.
 */
typedef struct KdaLinearArgs {
  uint32_t struct_size;        /* = sizeof(KdaLinearArgs) */
  int32_t M;                   /* rows of x, up to 2^31 - 512; 0 is a no-op */
  int32_t N;                   /* rows of weight, 1 .. 2^24; even with KDA_ACT_SILU_GATED */
  int32_t K;                   /* 1 .. 2^24 */
  int32_t activation;          /* KDA_ACT_* */
  uint32_t flags;
  const void* x;               /* [M][x_row_stride] */
  int64_t x_row_stride;        /* elements, >= K */
  const void* weight;          /* [N][weight_row_stride] */
  int64_t weight_row_stride;   /* elements, >= K */
  const float* x_scale;        /* fp32 [M]; with KDA_LINEAR_E4M3 only, there required */
  const float* weight_scale;   /* fp32 [N]; likewise */
  const float* bias;           /* fp32 [N] or NULL */
  const uint16_t* residual;    /* bf16 [M][residual_row_stride] or NULL */
  int64_t residual_row_stride; /* elements, >= the width of out */
  void* out;                   /* bf16 or fp32 [M][out_row_stride], N wide (N / 2 gated) */
  int64_t out_row_stride;      /* elements */
  int32_t* err_flag;           /* or NULL; KDA_DEVERR_TIMEOUT */
} KdaLinearArgs;

/*
 * Enqueue the product on `stream` (one launch, no workspace).  Returns KDA_OK
 * or a negative KDA_ERR_* code; on an error nothing is launched and
 * kda_last_error() describes it.  The first call on a device does a
 * once-per-device set-up: make it before any capture.
 */
int kda_linear(const KdaLinearArgs* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LINEAR_H */
