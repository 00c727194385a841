/*
 * kda_qk_rope.h -- C ABI of the per-head norm and position rotation of
 * queries and keys, with the write of keys and values into an 8-bit paged
 * cache in the same pass: the step in front of kda_cache_attention.h for the
 * softmax layers that stand between KDA layers.
 *
 * For every token row t (position pos = positions[t]) of the packed
 * projections qkv = [q heads | k heads | v heads], each head 128 wide:
 *   x^  = x / sqrt(mean(x^2) + eps) * weight       (q and k; a NULL weight
 *                                                   leaves that part unnormed)
 *   the first rot_dim channels of x^ are rotated in pairs (a_i, b_i), i <
 *   rot_dim / 2, by the angle 2 pi pos freqs[i] / 2^64:
 *     a_i' = a_i cos - b_i sin,  b_i' = b_i cos + a_i sin
 *   with (a_i, b_i) = channels (i, i + rot_dim / 2), or (2i, 2i + 1) with
 *   KDA_ROPE_INTERLEAVED; the other channels pass through.
 * freqs holds turns per position as unsigned 64-bit fractions, so
 * pos * freqs[i] wraps to the exact angle however far the position.
 *
 * Queries are written to q_out (bf16).  Keys are written to k_out (bf16,
 * optional) and, with a cache, keys and values (unrotated) go to the block
 * slot_map[t] / block_size at row slot_map[t] % block_size as e4m3 codes:
 * value = code * scale[block][head], one scale for K and one for V.
 *
 * Block scales.  For a block and head, let amax be the largest finite |x| of
 * the rows this call writes there, and fit = 2^e with the smallest e in
 * [-64, 119] such that amax <= 448 * 2^e (e = -64 for amax = 0).  If the
 * call writes the block's row 0 the scale becomes fit; otherwise older rows
 * stay in the block and the scale becomes max(old scale, fit), the codes of
 * the rows before the first written one being divided by the growth (exact,
 * a power of two, but for codes that fall below e4m3's normal range).
 * Codes are rounded to nearest even from the 32-bit value and saturate at
 * +-448; NaN stays NaN.
 */
#ifndef KDA_QK_ROPE_H
#define KDA_QK_ROPE_H

#include <stdint.h>

#include "kda_decode.h" /* return codes, KDA_DEVERR_SLOT_RANGE */

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ROPE_INTERLEAVED 1u

/*
 * Arguments.  T = token rows, D = 128.  bf16 tensors are passed as 16-bit
 * words, e4m3 as bytes.  qkv, q_out, k_out, the caches and their strides in
 * bytes are multiples of 16 bytes; freqs and slot_map 8 bytes, the weights
 * 16; the rest 4.
 *
 *   qkv        bf16 [T][qkv_row_stride], (Hq + 2 Hkv) * D channels used
 *   q_out      bf16 [T][q_row_stride], Hq * D written per row; may be the q
 *              part of qkv itself (same pointer and stride)
 *   k_out      bf16 [T][k_row_stride] or NULL, Hkv * D written per row; may
 *              be the k part of qkv itself only when there is no cache
 *   positions  int32 [T]
 *   freqs      uint64 [rot_dim / 2]
 *   caches     e4m3, element (block, head, row, d) at block * block_stride +
 *              head * head_stride + row * token_stride + d
 *   scales     fp32 [num_blocks][Hkv]
 *   slot_map   int64 [T]; < 0: the row's k and v are not cached (its q and
 *              k_out rows are still written).  A slot >= num_blocks *
 *              block_size is treated the same and sets KDA_DEVERR_SLOT_RANGE.
 *              The rows of a call that fall in one block are consecutive
 *              rows with consecutive slots.
 */
typedef struct KdaQkRopeArgs {
  uint32_t struct_size;        /* = sizeof(KdaQkRopeArgs) */
  int32_t T;
  int32_t num_q_heads, num_kv_heads;
  int32_t head_dim;            /* must be 128 */
  int32_t rot_dim;             /* 0 .. 128, a multiple of 16 */
  int32_t block_size;          /* 16, 32, 64, 128 or 256 (with a cache) */
  int32_t num_blocks;
  uint32_t flags;              /* KDA_ROPE_INTERLEAVED */
  float eps;
  const uint16_t* qkv;
  int64_t qkv_row_stride;      /* elements */
  uint16_t* q_out;
  int64_t q_row_stride;
  uint16_t* k_out;
  int64_t k_row_stride;
  const int32_t* positions;
  const uint64_t* freqs;       /* may be NULL when rot_dim is 0 */
  const float* q_weight;       /* fp32 [128] or NULL */
  const float* k_weight;       /* fp32 [128] or NULL */
  uint8_t* k_cache;            /* both caches or none */
  uint8_t* v_cache;
  int64_t block_stride, head_stride, token_stride; /* elements (bytes) */
  float* k_scale;
  float* v_scale;
  const int64_t* slot_map;
  int32_t* err_flag;           /* or NULL */
} KdaQkRopeArgs;

/*
 * Enqueue the pass on `stream` (one launch).  Returns KDA_OK or a negative
 * KDA_ERR_* code; on an error nothing is launched and kda_last_error()
 * describes it.  T == 0 is a no-op.
 */
int kda_qk_rope(const KdaQkRopeArgs* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_QK_ROPE_H */
