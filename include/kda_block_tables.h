/*
 * kda_block_tables.h -- C ABI of the device-side step metadata of a paged
 * cache: block tables, slot map, positions and cumulative starts, built on
 * the GPU from the requests' lengths (no device-to-host read, as for the
 * chunk metadata of kda_chunk_metadata.h).
 *
 * Definition, for request i with c_i tokens already cached and n_i new ones,
 * blocks (pages) of bs tokens, and the free list f with `head` entries
 * already taken:
 *   cu_seqlens[i] = n_0 + ... + n_{i-1}   (i = 0 .. B)
 *   seq_lens[i]   = c_i + n_i
 *   need_i        = ceil((c_i + n_i) / bs) - ceil(c_i / bs) new blocks, taken
 *                   from the list in request order: the k-th of request i is
 *                   f[head + need_0 + ... + need_{i-1} + k], stored to
 *                   block_table[i][ceil(c_i / bs) + k]; other entries of the
 *                   table are left as they are
 *   *free_head_out = head + sum need_i
 *   token row t = cu_seqlens[i] + j (j = 0 .. n_i - 1):
 *     positions[t] = c_i + j
 *     slot_map[t]  = block_table[i][positions[t] / bs] * bs + positions[t] % bs
 *   rows t = cu_seqlens[B] .. T - 1 (padding of a captured step):
 *     positions[t] = 0, slot_map[t] = -1
 * A request whose last step was cut back (drafted tokens that did not stand)
 * still holds the blocks it was given for them.  With held_blocks, h_i takes
 * the place of ceil(c_i / bs) above wherever it is larger, so that such blocks
 * are used before the list; held_blocks_out[i] is the count after this step,
 * the next step's h_i (blocks that the list did not have are not counted).
 */
#ifndef KDA_BLOCK_TABLES_H
#define KDA_BLOCK_TABLES_H

#include <stdint.h>

#include "kda_chunk_metadata.h" /* KDA_DEVERR_SEQLENS, KDA_DEVERR_CAPACITY */
#include "kda_decode.h"         /* return codes, KDA_DEVERR_SLOT_RANGE */

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Arguments; every pointer is caller-owned device memory, 4-byte aligned
 * (slot_map 8 bytes).  What a request asks for that cannot be had never
 * faults; it sets bits of *err_flag:
 *   KDA_DEVERR_SEQLENS    a length was negative or c_i + n_i passed 2^31 - 1:
 *                         the request gets no new tokens (a negative c_i
 *                         counts as 0)
 *   KDA_DEVERR_CAPACITY   the free list ran out, a request needs more than
 *                         max_blocks entries, or there are more than T new
 *                         tokens: tokens without a block get slot -1 (and
 *                         their table entry, where there is one, -1); rows
 *                         past T are not written
 *   KDA_DEVERR_SLOT_RANGE a block taken from the list or read from the table
 *                         is outside [0, num_blocks): treated as no block
 * Entries past max_blocks take nothing from the list, and *free_head_out
 * never passes num_free.  Blocks for tokens past row T are taken from the
 * list, stored in the table and counted as held like the others.  No result
 * may overlap an input (seq_lens is not cached_lens, and so on) or another
 * result.
 */
typedef struct KdaBlockTablesArgs {
  uint32_t struct_size;          /* = sizeof(KdaBlockTablesArgs) */
  int32_t B;                     /* requests */
  int32_t max_blocks;            /* entries of a block-table row, >= 1 */
  int32_t block_size;            /* tokens of a block, >= 1 */
  int32_t num_blocks;            /* blocks of the cache, >= 1 */
  int32_t T;                     /* rows of positions and slot_map */
  int32_t num_free;              /* entries of free_blocks */
  const int32_t* cached_lens;    /* [B] */
  const int32_t* new_lens;       /* [B] */
  const int32_t* held_blocks;    /* [B] or NULL: table entries that hold blocks, see below */
  int32_t* held_blocks_out;      /* [B] or NULL, another array than held_blocks */
  int32_t* block_table;          /* [B][block_table_stride] */
  int64_t block_table_stride;    /* elements, >= max_blocks */
  const int32_t* free_blocks;    /* [num_free] */
  const int32_t* free_head;      /* [1] or NULL for 0 */
  int32_t* free_head_out;        /* [1], another word than free_head */
  int32_t* cu_seqlens;           /* [B + 1] */
  int32_t* seq_lens;             /* [B] */
  int32_t* positions;            /* [T] */
  int64_t* slot_map;             /* [T] */
  int32_t* err_flag;             /* or NULL */
} KdaBlockTablesArgs;

/*
 * Enqueue the build on `stream`.  Returns KDA_OK or a negative KDA_ERR_* code
 * (nothing is launched then; kda_last_error() says why).  One launch; nothing
 * is allocated, synchronised or read back, so the call can be captured.
 */
int kda_block_tables(const KdaBlockTablesArgs* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_BLOCK_TABLES_H */
