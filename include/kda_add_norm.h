/*
 * kda_add_norm.h -- C ABI of the step in front of a layer's projection: the
 * addition of a layer's output to the residual stream, the root-mean-square
 * norm of the sum, and its output in bf16 and / or in 8 bits with one scale
 * per row, as kda_linear.h takes it.
 *
 * For every row t, with channels i < D:
 *   h  = x + residual                      (x alone where residual is NULL)
 *   y  = h / sqrt(mean(h^2) + eps) * weight   (a NULL weight counts as ones)
 *   y  = h                                 with KDA_ADD_NORM_NO_NORM
 *   residual_out = h,  out = y             rounded to bf16
 *   out_scale[t] = max(max|y|, 2^-100) * (1 / 448), the factor rounded to fp32
 *   out_q        = y / out_scale[t]        rounded to fp32, then to e4m3
 * The sum is not rounded before the norm, and y not before its code is made;
 * everything in between is fp32, and squares that fp32 does not hold are made
 * of the row relative to its largest channel, so that any row of finite sums
 * has its norm.  (A sum past fp32's range is infinite.)  A row whose y holds a
 * NaN or an infinity gets the scale NaN, and so does all that is made of it.
 */
#ifndef KDA_ADD_NORM_H
#define KDA_ADD_NORM_H

#include <stdint.h>

#include "kda_decode.h" /* return codes */

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ADD_NORM_NO_NORM 1u /* y = h; weight must be NULL */
#define KDA_ADD_NORM_MAX_D 32768

/*
 * Arguments.  bf16 tensors are passed as 16-bit words, e4m3 as bytes.  x,
 * residual, residual_out, out and weight are 16-byte aligned with row strides
 * of a multiple of 8 elements, out_q 8-byte aligned with a row stride of a
 * multiple of 8, out_scale 4.
 * Results may stand in the place of inputs where pointer and stride are the
 * same: residual_out in residual or x, out in x or residual (but not both in
 * one place); otherwise no result may overlap an input or another result.
 */
typedef struct KdaAddNormArgs {
  uint32_t struct_size;        /* = sizeof(KdaAddNormArgs) */
  int32_t T;                   /* rows; 0 is a no-op */
  int32_t D;                   /* channels, a multiple of 8 up to KDA_ADD_NORM_MAX_D */
  uint32_t flags;              /* KDA_ADD_NORM_NO_NORM */
  float eps;                   /* >= 0 */
  const uint16_t* x;           /* bf16 [T][x_row_stride] */
  int64_t x_row_stride;        /* elements, >= D, as all strides */
  const uint16_t* residual;    /* bf16 [T][residual_row_stride] or NULL */
  int64_t residual_row_stride;
  const float* weight;         /* fp32 [D] or NULL */
  uint16_t* residual_out;      /* bf16 [T][residual_out_row_stride] or NULL */
  int64_t residual_out_row_stride;
  uint16_t* out;               /* bf16 [T][out_row_stride] or NULL */
  int64_t out_row_stride;
  uint8_t* out_q;              /* e4m3 [T][out_q_row_stride] or NULL */
  int64_t out_q_row_stride;
  float* out_scale;            /* fp32 [T]; NULL exactly when out_q is */
} KdaAddNormArgs;

/*
 * Enqueue the step on `stream` (one launch, no workspace).  Returns KDA_OK or
 * a negative KDA_ERR_* code; on an error nothing is launched and
 * kda_last_error() describes it.
 */
int kda_add_norm(const KdaAddNormArgs* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_ADD_NORM_H */
