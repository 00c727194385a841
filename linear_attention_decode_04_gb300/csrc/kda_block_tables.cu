// kda_block_tables.cu -- block tables and slot maps from request lengths
// (definition in include/kda_block_tables.h).
//
// Latency bound: a few bytes per request and 12 per token row.  One launch,
// kThreads token rows per CTA.  Every CTA scans the requests' token and block
// counts itself, a tile of kTile requests at a time in shared memory: the
// lengths are a few KB out of L2, so repeating the scan costs less than a
// second launch or a grid-wide wait.  A row then finds its request by binary search
// among the tile's starts, and forms its block without reading any table
// entry that this launch writes: a block that is new this step comes straight
// from the free list.  The row that opens a block stores its table entry;
// each new block is opened by exactly one row.
//
// Measured on a GB300, back to back: 64 requests 4.4 to 4.7 us, 1,024 requests
// with 48,000 token rows 5.7 to 6.1 us (their bytes take 0.1 us: what is left is the
// launch, two trips to memory and the scan).  Sizes that are powers of two are
// shifted, not divided; sums are 64 bits wide, so that lengths whose total
// passes 2^31 are found rather than wrapped.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_block_tables.h"
#include "kda_internal.h"

namespace {

constexpr int kThreads = 512;
constexpr int kPer = 4;                  // requests per thread and tile
constexpr int kTile = kThreads * kPer;

struct Params {
  int B, max_blocks, bs, num_blocks, T, num_free;
  int log2;  // of bs, or -1
  const int32_t *cached, *fresh, *held;
  int32_t* held_out;
  int32_t* table;
  int64_t table_stride;
  const int32_t *free_blocks, *free_head;
  int32_t *free_head_out, *cu, *seq_lens, *positions;
  int64_t* slot_map;
  int32_t* err;
};

// pos / bs: a shift for the usual sizes (a division takes some 40 instructions)
__device__ __forceinline__ int block_of(const Params& p, int pos) { return p.log2 >= 0 ? pos >> p.log2 : pos / p.bs; }
// A request's lengths with what is out of range taken out: new tokens,
// first and number of new table entries.
struct Request {
  int c, n, first, need;
  bool bad, over;
};
__device__ __forceinline__ Request request(const Params& p, int i) {
  Request r;
  const int c = p.cached[i], n = p.fresh[i];
  r.bad = c < 0 || n < 0 || static_cast<int64_t>(c) + n > 0x7fffffffLL;
  r.c = c < 0 ? 0 : c;
  r.n = r.bad ? 0 : n;
  // ceil without the overflow of c + bs - 1
  const int cb = block_of(p, r.c), eb = block_of(p, r.c + r.n), full = cb + (r.c != cb * p.bs);
  const int have = p.held ? max(full, p.held[i]) : full;
  const int end = eb + (r.c + r.n != eb * p.bs);
  r.first = have;
  r.over = r.n > 0 && end > p.max_blocks;
  r.need = max(min(end, p.max_blocks) - min(have, p.max_blocks), 0);
  return r;
}

// Entry f of the free list: a block, or -1 and the reason among `errors`.
__device__ __forceinline__ int listed_block(const Params& p, int64_t f, int& errors) {
  if (f < 0 || f >= p.num_free) {
    errors |= KDA_DEVERR_CAPACITY;
    return -1;
  }
  const int b = p.free_blocks[f];
  if (b >= 0 && b < p.num_blocks) return b;
  errors |= KDA_DEVERR_SLOT_RANGE;
  return -1;
}

__global__ void __launch_bounds__(kThreads) block_tables_kernel(const Params p) {
  __shared__ int64_t tok_s[kTile + 1], blk_s[kTile];
  __shared__ int64_t warp_tok[kThreads / 32], warp_blk[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kThreads + tid;
  const int64_t row_end = static_cast<int64_t>(blockIdx.x + 1) * kThreads;
  const bool first_cta = blockIdx.x == 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t head = p.free_head ? *p.free_head : 0;
  int64_t tok = 0, blk = 0;  // tokens and new blocks of the requests before the tile
  int errors = 0;
  for (int base = 0; base < p.B; base += kTile) {
    int64_t n[kPer], need[kPer], nsum = 0, bsum = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = base + tid * kPer + k;
      n[k] = need[k] = 0;
      if (i < p.B) {
        const Request r = request(p, i);
        n[k] = r.n;
        need[k] = r.need;
        if (first_cta) {
          if (r.bad) errors |= KDA_DEVERR_SEQLENS;
          if (r.over) errors |= KDA_DEVERR_CAPACITY;
          p.seq_lens[i] = r.c + r.n;
        }
      }
      nsum += n[k];
      bsum += need[k];
    }
    int64_t nx = nsum, bx = bsum;  // inclusive over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, nx, o), b = __shfl_up_sync(0xffffffffu, bx, o);
      if (lane >= o) nx += a, bx += b;
    }
    if (lane == 31) warp_tok[warp] = nx, warp_blk[warp] = bx;
    __syncthreads();
    int64_t nbase = 0, bbase = 0, ntile = 0, btile = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w == warp) nbase = ntile, bbase = btile;
      ntile += warp_tok[w];
      btile += warp_blk[w];
    }
    int64_t ns = tok + nbase + nx - nsum, bo = blk + bbase + bx - bsum;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int j = tid * kPer + k;
      tok_s[j] = ns;
      blk_s[j] = bo;
      if (first_cta && base + j < p.B) {
        p.cu[base + j] = static_cast<int32_t>(ns < 0x7fffffff ? ns : 0x7fffffff);
        if (p.held_out) {  // what the request held, and of the new blocks those that the list had
          const int64_t from = head + bo, got = from < 0 ? 0 : min(max(p.num_free - from, int64_t{0}), need[k]);
          p.held_out[base + j] = min(request(p, base + j).first, p.max_blocks) + static_cast<int>(got);
        }
      }
      ns += n[k];
      bo += need[k];
    }
    __syncthreads();
    if (first_cta && tok + ntile > p.T) {
      // blocks that rows past the end would open: taken and counted, so stored as well; a warp per request
      for (int j = warp; j < min(kTile, p.B - base); j += kThreads / 32) {
        if ((j + 1 < kTile ? tok_s[j + 1] : tok + ntile) <= p.T) continue;
        const Request r = request(p, base + j);
        for (int e = lane; e < r.need; e += 32) {
          const int page = r.first + e;
          if (tok_s[j] + (static_cast<int64_t>(page) * p.bs - r.c) >= p.T)
            p.table[(base + j) * p.table_stride + page] = listed_block(p, head + blk_s[j] + e, errors);
        }
      }
    }
    if (row >= tok && row < tok + ntile && row < p.T) {
      // the last request of the tile that starts at or before the row; it is
      // not empty, because the next one starts behind the row
      int lo = 0, hi = min(kTile, p.B - base);
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tok_s[mid] <= row) lo = mid;
        else hi = mid;
      }
      const int i = base + lo;
      const Request r = request(p, i);
      const int pos = r.c + static_cast<int>(row - tok_s[lo]);
      const int page = block_of(p, pos), at = pos - page * p.bs;
      int b = -1;
      if (page < p.max_blocks) {
        int32_t* entry = p.table + i * p.table_stride + page;
        if (page >= r.first) {
          b = listed_block(p, head + blk_s[lo] + (page - r.first), errors);
          if (at == 0) *entry = b;
        } else {
          b = *entry;
          if (b < 0 || b >= p.num_blocks) b = -1, errors |= KDA_DEVERR_SLOT_RANGE;
        }
      }
      p.positions[row] = pos;
      p.slot_map[row] = b < 0 ? -1 : static_cast<int64_t>(b) * p.bs + at;
    }
    tok += ntile;
    blk += btile;
    if (!first_cta && tok >= row_end) break;
    __syncthreads();
  }
  if (row >= tok && row < p.T) {
    p.positions[row] = 0;
    p.slot_map[row] = -1;
  }
  if (first_cta && tid == 0) {
    p.cu[p.B] = static_cast<int32_t>(tok < 0x7fffffff ? tok : 0x7fffffff);
    const int64_t used = head + blk;
    *p.free_head_out = static_cast<int32_t>(used < p.num_free ? used : max(head, static_cast<int64_t>(p.num_free)));
    if (tok > p.T) errors |= KDA_DEVERR_CAPACITY;
  }
  if (errors && p.err) atomicOr(p.err, errors);
}

bool misaligned(const void* ptr, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(ptr) & mask) != 0; }

}  // namespace

extern "C" int kda_block_tables(const KdaBlockTablesArgs* a, void* stream) {
  kda_internal_clear_error();
  if (!a) return kda_internal_fail(KDA_ERR_NULLPTR, "args is NULL");
  if (a->struct_size != sizeof(KdaBlockTablesArgs))
    return kda_internal_fail(KDA_ERR_ABI, "struct_size %u, library expects %zu", a->struct_size,
                             sizeof(KdaBlockTablesArgs));
  if (a->B < 0 || a->max_blocks < 1 || a->block_size < 1 || a->num_blocks < 1 || a->T < 0 || a->num_free < 0 ||
      a->block_table_stride < a->max_blocks)
    return kda_internal_fail(KDA_ERR_SHAPE, "B=%d max_blocks=%d block_size=%d num_blocks=%d T=%d num_free=%d", a->B,
                             a->max_blocks, a->block_size, a->num_blocks, a->T, a->num_free);
  if (!a->cu_seqlens || !a->free_head_out ||
      (a->B > 0 && (!a->cached_lens || !a->new_lens || !a->block_table || !a->seq_lens)) ||
      (a->num_free > 0 && !a->free_blocks) || (a->T > 0 && (!a->positions || !a->slot_map)))
    return kda_internal_fail(KDA_ERR_NULLPTR, "a required pointer is NULL");
  if (a->free_head == a->free_head_out)
    return kda_internal_fail(KDA_ERR_SHAPE, "free_head and free_head_out must be two words");
  if (a->held_blocks && a->held_blocks == a->held_blocks_out)
    return kda_internal_fail(KDA_ERR_SHAPE, "held_blocks and held_blocks_out must be two arrays");
  // every CTA reads all lengths for itself, some after others have written
  const void* const in[] = {a->cached_lens, a->new_lens, a->held_blocks, a->free_blocks, a->free_head};
  const void* const results[] = {a->seq_lens, a->cu_seqlens, a->held_blocks_out, a->positions, a->block_table};
  for (const void* x : in)
    for (const void* y : results)
      if (x && x == y) return kda_internal_fail(KDA_ERR_SHAPE, "a result may not take the place of an input");
  if (misaligned(a->held_blocks, 3) || misaligned(a->held_blocks_out, 3) || misaligned(a->cached_lens, 3) ||
      misaligned(a->new_lens, 3) || misaligned(a->block_table, 3) ||
      misaligned(a->free_blocks, 3) || misaligned(a->free_head, 3) || misaligned(a->free_head_out, 3) ||
      misaligned(a->cu_seqlens, 3) || misaligned(a->seq_lens, 3) || misaligned(a->positions, 3) ||
      misaligned(a->slot_map, 7) || misaligned(a->err_flag, 3))
    return kda_internal_fail(KDA_ERR_ALIGN, "a pointer is not aligned as required");
  int log2 = -1;
  if ((a->block_size & (a->block_size - 1)) == 0)
    for (log2 = 0; (1 << log2) < a->block_size;) ++log2;
  const Params p{a->B, a->max_blocks, a->block_size, a->num_blocks, a->T, a->num_free, log2, a->cached_lens, a->new_lens,
                 a->held_blocks, a->held_blocks_out,
                 a->block_table, a->block_table_stride, a->free_blocks, a->free_head, a->free_head_out,
                 a->cu_seqlens, a->seq_lens, a->positions, a->slot_map, a->err_flag};
  const unsigned grid = a->T > kThreads ? static_cast<unsigned>((static_cast<int64_t>(a->T) + kThreads - 1) / kThreads) : 1u;
  const cudaError_t e = kda_internal_launch(block_tables_kernel, dim3(grid), dim3(kThreads), 0, stream, p);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
  return KDA_OK;
}
