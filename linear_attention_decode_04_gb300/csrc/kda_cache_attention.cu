// kda_cache_attention.cu -- causal softmax attention over the 8-bit paged
// cache (definition in include/kda_cache_attention.h).
//
// Single tokens and multi-token steps are bound by HBM (the cache is read
// once); prompt chunks by the softmax between the two products.  There are
// two kernels: one for up to 96 query rows per kv head and sequence, one
// (at the end) for more.
//
// Measured on a GB300 against a copy's 6795 GB/s: one token behind 260,000
// cached ones, 96 q and 8 kv heads, 91 us (78 at a copy's rate); 64 sequences of
// 4 tokens behind 1,000 to 16,384, 48 heads, 134 us (110); a small batch 7 us, of
// which the launch, the plan and the trip to the first tile take most.  4 prompt chunks
// of 515 tokens, 48 heads, 90 us; long ones reach 860 TFLOP/s of useful work.
// 33 to 96 rows are far from the copy's rate: 64 sequences of 8 tokens, 64 heads, 234
// us (112); their variants share maxima between groups and spill registers.
//
// Products of the first kernel.  Both are formed transposed, so that the
// cache's codes are the 128-row operand and the few queries the narrow one:
//   S^T [token][row]   = K [token][d]   Q^T [d][row]      (128 x R, k = 128)
//   O^T [d][row]       = V^T [d][token] P^T [token][row]  (128 x R, k = 128)
// with R query rows (tokens x heads of one kv head).  K and V tiles of 128
// tokens go from the paged cache to shared memory by TMA (128-byte swizzle)
// and from there to tcgen05 kind::f8f6f4 untouched: K as a K-major operand, V
// as an M-major one.  The narrow operand is split into two e4m3 parts (leading
// and remainder), each a product of its own into the same accumulator; the
// tensor cores have time for that, and no code of the cache is ever converted.
// What that rounds: the parts end at e4m3's smallest step, 2^-9, below a largest
// value of 2^8 (of a tile's weights) or 224 to 448 (of a query row).  So a weight is
// off by 2^-8 of itself at most, or 2^-18 of its tile's largest; its rounding to
// fp16 on the way (2^-12) is small beside that and lets conversions and the remainder's
// subtraction work on pairs.  The output is rounded to bf16's 2^-8 in the end; a third part would cost
// half as many products again for bits that are lost there.  The softmax sum adds the
// unrounded weights: the roundings, as often up as down, then stay in the numerator
// alone, where they average out, and no sum has to wait for the parts.
//
// Block scales.  k_scale multiplies S.  v_scale is folded into the weights:
// with z = s + log2(v_scale) a token's weight is w = 2^(z - M), M the largest
// z of the tile, so a row's weights use e4m3's range whatever the scales are;
// the softmax sum adds w / v_scale.  Every tile has its own M and its own
// accumulator, which is added to the row's fp32 sum in registers with the
// factor 2^(M - running max): an accumulator never has to be rescaled, and
// a tile of small weights loses no bits beside a large one.
//
// Work split.  The tiles of all (sequence, row tile, kv head) units in one
// row are dealt out evenly to the resident CTAs, whatever the lengths; a unit
// that several CTAs share leaves partial sums in the workspace, and the CTA
// that arrives last joins them in order of position (the result does not
// depend on who is last).
//
// Roles.  One producer warp (block table and scales two tiles ahead, TMA
// into a ring), one warp whose lane 0 issues the products, and groups of one
// warpgroup for 8, 16 or 24 query rows each (Cfg).  A thread holds 4 tokens of
// a quarter of the group's rows, so a row's maximum takes shuffles and one trip
// through shared memory per tile; up to 24 rows one group is enough (two CTAs
// an SM hide one another's waits), above it several groups of 16 share the
// tile: more warps hide the chain of one tile better than longer columns do
// (64 sequences x 8 tokens x 64 heads: 244 us with groups of 16 when that was chosen,
// 295 with 32).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "kda_cache_attention.h"
#include "kda_chunk_metadata.h"
#include "kda_internal.h"

namespace {

constexpr int kD = KDA_HEAD_DIM;
constexpr int kTile = 128;                 // tokens per tile
constexpr int kTileBytes = kTile * kD;     // of K, and of V
constexpr int kMaxPages = 8;               // blocks of a tile, at block size 16
constexpr int kMaxCtas = 304;              // 2 x 152
// What beginning and ending a unit costs, in tiles: the work is dealt out by
// tiles + kUnitCost per unit, so that CTAs with many short units end with the rest.
// One value for all variants, measured with 2, 4 and 8: prompt chunks 101, 90 and 94 us;
// 64 sequences behind 1,000 to 16,384 tokens, 8 rows 120, 121 and 124, 16 rows 117, 117
// and 121, 24 rows 135, 134 and 137, 32 rows 163, 156 and 158, 64 rows 245, 234 and 246,
// 96 rows 363, 339 and 343; one long sequence 91 with any.  Only many short units of few
// rows want less: 500 sequences of 10 to 2,000 tokens, 8 rows, 114, 124 and 141.
constexpr int kUnitCost = 4;
constexpr int kCounters = 4 * 6 * 152;     // of each kind: CTAs x warps that join, at most
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kLog2e = 1.44269504088896340736f;

struct Params {
  int B, T, Hq, Hkv, G, bs_log2, num_blocks, max_blocks;
  uint32_t g_mul;  // ceil(2^32 / G), or 0 where that is not exact for every row
  float scale;  // sm_scale * log2(e)
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  int64_t out_stride;
  const int32_t *cu, *lens, *table;
  int64_t table_stride;
  const float *k_scale, *v_scale;
  int32_t* counters;
  float* partial;
  int32_t* err;
};

// A variant: `GROUPS` softmax warpgroups of `COLS` query rows each.
template <int COLS, int GROUPS>
struct Cfg {
  static constexpr int kCols = COLS, kGroups = GROUPS;
  static constexpr int kRows = COLS * GROUPS;            // query rows of a tile
  static constexpr int kN = (kRows + 15) / 16 * 16;      // width of the products
  static constexpr int kThreads = 128 * GROUPS + 64;
  static constexpr int kCtasPerSm = kRows > 32 ? 1 : 2;
  // a group's pairs of 8-column blocks share 16 columns of the weights
  static_assert(COLS % 16 == 0 || COLS == 8 || GROUPS == 1, "groups");
  // Ring depths in tiles.  A K tile is free after its S product, about a tile's
  // time before its V tile is; at 32 rows two CTAs fit an SM with K two deep.
  static constexpr int kK = kRows > 32 ? 3 : kN > 16 ? 2 : 3;
  static constexpr int kV = kRows > 32 ? 4 : 3;
  static constexpr int kNan = GROUPS > 1 ? 4 : 1;
  static constexpr int kTmemCols = kN > 64 ? 512 : 4 * kN;  // S and O, two buffers each; a power of two
  static constexpr int kPartial = COLS * (32 + 2);       // floats of a warp's partial record: maxima, sums, 32 channels
  // parts that one warp joins (one token behind 260,000: 92 us with 8, 94 with 16, 99 with all in one)
  static constexpr int kJoinFan = 8;
  static constexpr int kBlocks = COLS / 8;               // 8-column blocks of a group's tensor-memory loads
  static constexpr int kMine = COLS / 4;                 // rows that a thread holds elements of
};

// The variant for prompts: two softmax warpgroups of 128 query rows each.  Four
// warps beside them, producer, issuer and two that wait, so that whole warpgroups
// can trade registers.
struct Wide {
  static constexpr int kGroups = 2, kRows = 256;
  static constexpr int kThreads = 128 * kGroups + 128;
  static constexpr int kCtasPerSm = 1, kK = 3, kV = 3;
  static constexpr int kPartial = 32 * (kD + 2);         // floats of a warp's partial record: maxima, sums, 32 rows
  static constexpr int kJoinFan = 8;
};

template <class C>
struct alignas(1024) Smem {
  uint8_t p[2][C::kN * kTile];            // leading part, remainder; [row' / 16][token][row' % 16]
  uint8_t q[2][C::kN * kD];               // likewise; core matrices of 8 rows x 16 bytes
  uint8_t k[C::kK][kTileBytes], v[C::kV][kTileBytes];
  uint64_t k_full[C::kK], k_empty[C::kK], v_full[C::kV], v_empty[C::kV], sc_full[C::kV];
  uint64_t s_full[2], o_full[2], p_full, q_full, done;
  float4 sc[C::kV][kMaxPages];            // k_scale, log2(v_scale), 1 / v_scale of a tile's blocks; lives as V does
  float row_scale[C::kRows];
  int limit[C::kRows];
  float wmax[2][C::kGroups][4][C::kCols];
  float wsum[C::kGroups][4][C::kCols];
  int nan_at[C::kNan][kD];                // per unit and channel: first position that holds a NaN value
  int64_t total;                          // cost of all work, for the few places that need it again
  int walk[7];                            // where this CTA's tiles start
  int64_t scan[C::kThreads / 32], beyond[C::kThreads / 32];
  uint32_t tmem;
  int failed;
};
// Per warp, broadcast to its lanes: the tile's maxima, and the two factors per
// row of the tile and of the one before.
template <class C>
struct alignas(16) Bcast {
  float mt[C::kCols];
  float alpha[2][C::kCols], beta[2][C::kCols];
};

struct alignas(1024) WideSmem {
  uint8_t q[2][2][128 * kD], p[2][2][128 * kTile];  // [group][leading part, remainder], rows of 128 bytes, swizzled as K is
  uint8_t k[Wide::kK][kTileBytes], v[Wide::kV][kTileBytes];
  uint64_t k_full[Wide::kK], k_empty[Wide::kK], v_full[Wide::kV], v_empty[Wide::kV], sc_full[Wide::kV];
  uint64_t s_full[2], o_full[2], p_full[2], q_full[2], done;
  float4 sc[Wide::kV][kMaxPages];
  int nan_at[kD];                         // of the unit, as above
  int nan_seen;
  int64_t total;
  int walk[7];
  int64_t scan[Wide::kThreads / 32], beyond[Wide::kThreads / 32];
  uint32_t tmem;
  int failed;
};

__device__ __forceinline__ uint32_t s32(const void* ptr) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(ptr));
}
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(s32(b)), "r"(count));
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(s32(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(s32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(s32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase, at most kWaitLimitNs; after any thread of the CTA has
// given up, no thread waits any more.
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, int* failed) {
  if (bar_try(b, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    if (bar_try(b, parity)) return true;
    if (*reinterpret_cast<volatile int*>(failed)) return false;
    uint64_t now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
    if (it == 0) t0 = now;
    else if (now - t0 > kWaitLimitNs) {
      *reinterpret_cast<volatile int*>(failed) = 1;
      return false;
    }
  }
}
// The same without regard to others that gave up: for copies already on their way.
__device__ __forceinline__ void bar_drain(uint64_t* b, uint32_t parity) {
  uint64_t t0, now;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  do asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
  while (!bar_try(b, parity) && now - t0 < kWaitLimitNs);
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(s32(b)) : "memory");
}
// Shared-memory matrix descriptor: start, leading and stride byte offsets in
// 16-byte units, version 1, swizzle (0 none, 2 = 128 bytes).
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFF) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFF) << 32) | (1ull << 46) | (static_cast<uint64_t>(swizzle) << 61);
}
// Instruction descriptor, kind::f8f6f4: f32 accumulator, e4m3 operands, M = 128, N = n.
__host__ __device__ constexpr uint32_t idesc(uint32_t n, bool a_m_major, bool b_n_major) {
  return (1u << 4) | (static_cast<uint32_t>(a_m_major) << 15) | (static_cast<uint32_t>(b_n_major) << 16) |
         ((n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int tok, int head, int block, uint64_t* b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(map), "r"(0), "r"(tok), "r"(head), "r"(block), "r"(s32(b))
      : "memory");
}
// BLOCKS * 8 consecutive columns of this warp's 32 lanes, as fragments: thread
// i gets of block b, in r[j][2b], r[j][2b + 1], lane i / 4 + 8 j, columns
// 8 b + 2 (i % 4) and the next.  The load writes the registers of all 32
// threads, so the warp has to be together: a thread still on a branch of its
// own would find its registers overwritten.  Load and wait are one statement,
// so that nothing can come between them.
template <int BLOCKS>
__device__ __forceinline__ void tm_ld(uint32_t addr, float (&r)[4][2 * BLOCKS]) {
  __syncwarp();
  const uint32_t up = addr + (16u << 16);  // the upper 16 lanes
  if constexpr (BLOCKS == 1) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%8];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%4,%5,%6,%7}, [%9];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0][0]), "=f"(r[0][1]), "=f"(r[1][0]), "=f"(r[1][1]), "=f"(r[2][0]), "=f"(r[2][1]), "=f"(r[3][0]),
          "=f"(r[3][1])
        : "r"(addr), "r"(up)
        : "memory");
  } else if constexpr (BLOCKS == 2) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0][0]), "=f"(r[0][1]), "=f"(r[1][0]), "=f"(r[1][1]), "=f"(r[0][2]), "=f"(r[0][3]), "=f"(r[1][2]),
          "=f"(r[1][3]), "=f"(r[2][0]), "=f"(r[2][1]), "=f"(r[3][0]), "=f"(r[3][1]), "=f"(r[2][2]), "=f"(r[2][3]),
          "=f"(r[3][2]), "=f"(r[3][3])
        : "r"(addr), "r"(up)
        : "memory");
  } else if constexpr (BLOCKS == 3) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%24];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%8,%9,%10,%11}, [%25];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%12,%13,%14,%15,%16,%17,%18,%19}, [%26];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%20,%21,%22,%23}, [%27];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0][0]), "=f"(r[0][1]), "=f"(r[1][0]), "=f"(r[1][1]), "=f"(r[0][2]), "=f"(r[0][3]), "=f"(r[1][2]),
          "=f"(r[1][3]), "=f"(r[0][4]), "=f"(r[0][5]), "=f"(r[1][4]), "=f"(r[1][5]), "=f"(r[2][0]), "=f"(r[2][1]),
          "=f"(r[3][0]), "=f"(r[3][1]), "=f"(r[2][2]), "=f"(r[2][3]), "=f"(r[3][2]), "=f"(r[3][3]), "=f"(r[2][4]),
          "=f"(r[2][5]), "=f"(r[3][4]), "=f"(r[3][5])
        : "r"(addr), "r"(addr + 16), "r"(up), "r"(up + 16)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
        "[%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0][0]), "=f"(r[0][1]), "=f"(r[1][0]), "=f"(r[1][1]), "=f"(r[0][2]), "=f"(r[0][3]), "=f"(r[1][2]),
          "=f"(r[1][3]), "=f"(r[0][4]), "=f"(r[0][5]), "=f"(r[1][4]), "=f"(r[1][5]), "=f"(r[0][6]), "=f"(r[0][7]),
          "=f"(r[1][6]), "=f"(r[1][7]), "=f"(r[2][0]), "=f"(r[2][1]), "=f"(r[3][0]), "=f"(r[3][1]), "=f"(r[2][2]),
          "=f"(r[2][3]), "=f"(r[3][2]), "=f"(r[3][3]), "=f"(r[2][4]), "=f"(r[2][5]), "=f"(r[3][4]), "=f"(r[3][5]),
          "=f"(r[2][6]), "=f"(r[2][7]), "=f"(r[3][6]), "=f"(r[3][7])
        : "r"(addr), "r"(up)
        : "memory");
  }
}
// A thread's column pairs reduced over the 8 threads that hold the same columns
// (lane bits 2 to 4), each of them ending with one column: afterwards lane i
// holds local column own_column(i).
struct Max {
  __device__ __forceinline__ static float of(float a, float b) { return fmaxf(a, b); }
};
struct Sum {
  __device__ __forceinline__ static float of(float a, float b) { return a + b; }
};
template <class Op, int N>
__device__ __forceinline__ float reduce_columns(const float (&in)[N], int lane) {
  constexpr int P = N > 4 ? 8 : N;  // 2, 4 or 8 (6 is padded)
  float v[P];
#pragma unroll
  for (int i = 0; i < P; ++i) v[i] = i < N ? in[i < N ? i : 0] : 0.f;
#pragma unroll
  for (int o = 16, h = P / 2; o >= 4; o >>= 1, h >>= 1) {
    if (h >= 1) {
#pragma unroll
      for (int i = 0; i < (h > 0 ? h : 1); ++i) {
        const float send = lane & o ? v[i] : v[i + h], keep = lane & o ? v[i + h] : v[i];
        v[i] = Op::of(keep, __shfl_xor_sync(0xffffffffu, send, o));
      }
    } else {
      v[0] = Op::of(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
  }
  return v[0];
}
template <int N>
__device__ __forceinline__ int own_column(int lane) {  // the group's column, >= the width for padding
  constexpr int P = N > 4 ? 8 : N;
  const int i = P == 8 ? (lane >> 4) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1)
              : P == 4 ? (lane >> 4) * 2 + ((lane >> 3) & 1) : lane >> 4;
  return 8 * (i >> 1) + 2 * (lane & 3) + (i & 1);
}
// The weights' columns are kept in an order of their own within 16 so that a
// thread's two pairs are four neighbouring bytes; the accumulator's column
// 8 b + 2 (lane % 4) then belongs to this row (and the next to the next).
template <int BLOCKS>
__device__ __forceinline__ int row_of_column(int b, int lane) {
  const int a = lane & 3;
  if (BLOCKS & 1 && b == BLOCKS - 1) return 8 * b + 2 * a;  // an 8-column end keeps its order
  return (b >> 1) * 16 + 8 * (a & 1) + 4 * (b & 1) + 2 * (a >> 1);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 0xff in the bytes that are NaN codes (0x7f, 0xff)
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }
// Clears the NaN codes of this thread's row of a swizzled tile and notes the
// position per channel.  Rare; all threads of the warp call it.
__device__ __forceinline__ void take_out_nan(uint8_t* row, bool mine, int t, int pos, int* nan_at) {
  if (mine)
#pragma unroll 1
    for (int c = 0; c < kD / 4; ++c) {  // four channels at a time, from their swizzled place
      uint32_t* w = reinterpret_cast<uint32_t*>(row + ((c >> 2) ^ (t & 7)) * 16 + (c & 3) * 4);
      const uint32_t m = nan_bytes(*w);
      if (m) {
        *w &= ~m;
#pragma unroll 1
        for (int j = 0; j < 4; ++j)
          if ((m >> (8 * j)) & 1) atomicMin(nan_at + 4 * c + j, pos);
      }
    }
  __syncwarp();
}
template <int GROUP_THREADS>
__device__ __forceinline__ void group_sync(int g) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(g + 1), "n"(GROUP_THREADS) : "memory");
}

// ------------------------------------------------------------------ the walk
// Units in the order sequence, row tile, kv head; a unit's tiles in order.
struct Walk {
  int seq, rt, h;        // current unit
  int n, len, q0;        // the sequence's queries, length, first query row
  int rts, nt;           // its row tiles; tiles of the current unit
};
// row / G for row < n * G
__device__ __forceinline__ int token_of(const Params& p, int row) {
  return p.g_mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(row), p.g_mul)) : row / p.G;
}
template <class C>
__device__ __forceinline__ int tiles_of(const Params& p, int n, int len, int rt) {
  const int rows = n * p.G;
  const int last = min(rows, (rt + 1) * C::kRows) - 1;  // last query row of the tile
  const int limit = len - n + token_of(p, last) + 1;    // tokens it sees
  return limit <= kTile ? 1 : (limit + kTile - 1) / kTile;
}
template <class C>
__device__ __forceinline__ int rows_to_tiles(const Params& p, int n) {
  return static_cast<int>((static_cast<int64_t>(n) * p.G + C::kRows - 1) / C::kRows);
}
template <class C>
__device__ __forceinline__ bool load_seq(const Params& p, Walk& w) {  // false: nothing to do in this sequence
  if (w.seq < 0 || w.seq >= p.B) {  // cannot be; an empty end of the walk rather than a stray read
    w.q0 = w.n = w.len = w.rt = w.h = 0;
    w.rts = 1;
    return true;
  }
  const int a = p.cu[w.seq], b = p.cu[w.seq + 1];
  w.q0 = a;
  w.n = b - a;
  w.len = p.lens[w.seq];
  if (a < 0 || b < a || b > p.T) w.n = 0;
  if (w.len > 0x7fffff00) w.len = 0x7fffff00;
  if (w.len < 0) w.len = 0;
  w.rt = w.h = 0;
  w.rts = rows_to_tiles<C>(p, w.n);
  return w.n > 0;
}
template <class C>
__device__ __forceinline__ void next_unit(const Params& p, Walk& w) {  // only called while units are left
  if (++w.h < p.Hkv) return;
  w.h = 0;
  if (++w.rt >= w.rts) {
    do ++w.seq;
    while (!load_seq<C>(p, w));
  }
  w.nt = tiles_of<C>(p, w.n, w.len, w.rt);
}
template <class C>
__device__ __forceinline__ int64_t seq_cost(const Params& p, int i) {
  Walk w;
  w.seq = i;
  if (!load_seq<C>(p, w)) return 0;
  int64_t s = 0;
  for (int rt = 0; rt < w.rts; ++rt) s += tiles_of<C>(p, w.n, w.len, rt) + kUnitCost;
  return s * p.Hkv;
}
// A CTA's share: the units it has tiles of, one after another.  Positions are
// in cost; a unit's cost is kUnitCost, then its tiles.
struct Share {
  Walk w;
  int64_t us, left;  // where the unit begins; cost left of the share, this unit's included
  int off;           // where the share begins in the unit
  int t0, take;      // the unit's tiles here
  __device__ __forceinline__ int span() const {
    return static_cast<int>(min(static_cast<int64_t>(kUnitCost + w.nt - off), left));
  }
  __device__ __forceinline__ void tiles() {
    t0 = max(off - kUnitCost, 0);
    take = max(off + span() - kUnitCost, 0) - t0;
  }
};
template <class C>
__device__ __forceinline__ bool next_share(const Params& p, Share& s) {  // false: the share is done
  do {
    s.left -= s.span();
    if (s.left <= 0) return false;
    s.us += kUnitCost + s.w.nt;
    s.off = 0;
    next_unit<C>(p, s.w);
    s.tiles();
  } while (s.take == 0);
  return true;
}

// Where this CTA's tiles lie: the total, then the sequence they start in.  All
// threads; false where the CTA has none.  The tensor memory that warp 0 asked for
// is there afterwards.
template <class C, class M>
__device__ __forceinline__ bool plan(const Params& p, M& S, Share& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t mine = 0, beyond = 0;  // cost of sequence tid, and of those past the first kThreads
  bool bad = false;
  for (int i = tid; i < p.B; i += C::kThreads) {
    const int64_t c = seq_cost<C>(p, i);
    if (i == tid) mine = c;
    else beyond += c;
    const int a = p.cu[i], b = p.cu[i + 1];
    bad |= a < 0 || b < a || b > p.T;
  }
  if (bad && blockIdx.x == 0 && p.err) atomicOr(p.err, KDA_DEVERR_SEQLENS);
  auto warp_scan = [&](int64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    return v;
  };
  int64_t incl = warp_scan(mine);
  if (p.B > C::kThreads) beyond = warp_scan(beyond);
  if (lane == 31) S.scan[warp] = incl, S.beyond[warp] = beyond;
  tc_before();
  __syncthreads();
  tc_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int64_t prior = 0, all = 0, total = 0;
#pragma unroll
  for (int w = 0; w < C::kThreads / 32; ++w) {
    if (w < warp) prior += S.scan[w];
    all += S.scan[w];
    total += S.beyond[w];
  }
  total += all;
  if (tid == 0) S.total = total;
  // one position at least for each CTA that takes part, so that every CTA between
  // a unit's first and last leaves a part of it
  const int64_t cta = blockIdx.x, ctas = max(min(static_cast<int64_t>(gridDim.x), total), int64_t{1});
  // (32-bit division where it is enough: 64-bit ones take longer than the scan)
  auto share_of = [&](int64_t c) {
    return total < (1 << 22) ? static_cast<int64_t>(static_cast<uint32_t>(c * total) / static_cast<uint32_t>(ctas))
                             : c * total / ctas;
  };
  const int64_t begin = cta < ctas ? share_of(cta) : 0, end = cta < ctas ? share_of(cta + 1) : 0;
  if (begin >= end) return false;
  auto look = [&](int i, int64_t from, int64_t cost) {  // whether the share begins in sequence i
    if (cost == 0 || begin < from || begin >= from + cost) return;
    Walk w;
    w.seq = i;
    load_seq<C>(p, w);
    int64_t off = begin - from;
    int c = tiles_of<C>(p, w.n, w.len, 0) + kUnitCost;
    while (off >= static_cast<int64_t>(c) * p.Hkv) {
      off -= static_cast<int64_t>(c) * p.Hkv;
      c = tiles_of<C>(p, w.n, w.len, ++w.rt) + kUnitCost;
    }
    S.walk[0] = i;
    S.walk[4] = w.n, S.walk[5] = w.len, S.walk[6] = w.q0;
    S.walk[1] = w.rt;
    const bool small = off < 0x7fffffff;
    S.walk[2] = small ? static_cast<int>(off) / c : static_cast<int>(off / c);
    S.walk[3] = small ? static_cast<int>(off) % c : static_cast<int>(off % c);
  };
  look(tid, prior + incl - mine, mine);
  for (int base = C::kThreads; all <= begin; base += C::kThreads) {  // larger batches
    __syncthreads();
    const int i = base + tid;
    mine = i < p.B ? seq_cost<C>(p, i) : 0;
    incl = warp_scan(mine);
    if (lane == 31) S.scan[warp] = incl;
    __syncthreads();
    prior = all;
#pragma unroll
    for (int w = 0; w < C::kThreads / 32; ++w) {
      if (w < warp) prior += S.scan[w];
      all += S.scan[w];
    }
    look(i, prior + incl - mine, mine);
  }
  __syncthreads();
  Walk& w = sh.w;
  w.seq = S.walk[0];
  w.n = S.walk[4], w.len = S.walk[5], w.q0 = S.walk[6];
  w.rts = rows_to_tiles<C>(p, w.n);
  w.rt = S.walk[1];
  w.h = S.walk[2];
  w.nt = tiles_of<C>(p, w.n, w.len, w.rt);
  sh.off = S.walk[3];
  sh.us = begin - sh.off;
  sh.left = end - begin;
  sh.tiles();
  return true;
}
// One warp: tables and scales two tiles ahead, then the tiles into the rings.
template <class C, class M>
__device__ __forceinline__ void produce(const Params& p, M& S, Share& sh, bool more, const CUtensorMap& k_map,
                                        const CUtensorMap& v_map) {
  const int lane = threadIdx.x & 31;
  Walk& w = sh.w;
  const int log2 = p.bs_log2, rows = min(1 << log2, kTile), ppt = kTile / rows;  // rows of a copy, copies of a tile
  struct Ref {
    int block, head, tok;
    bool valid;
  };
  int t = sh.t0;       // next tile
  auto take = [&]() {  // the next tile of the share: this lane's block id in it
    Ref r;
    r.valid = more;
    r.block = -1;
    r.head = r.tok = 0;
    if (!more) return r;
    r.head = w.h;
    const int pos = t * kTile + (lane < ppt ? lane * rows : 0);  // (lengths end below 2^31 - 256)
    r.tok = pos & ((1 << log2) - 1);
    const int last = min(w.n * p.G, (w.rt + 1) * C::kRows) - 1;
    const int limit = w.len - w.n + token_of(p, last) + 1;
    if (lane < ppt && pos < limit) {
      const int e = pos >> log2;
      int b = -1;
      if (e < p.max_blocks) b = p.table[w.seq * p.table_stride + e];
      if (b < 0 || b >= p.num_blocks) {
        b = -1;
        if (p.err) atomicOr(p.err, KDA_DEVERR_SLOT_RANGE);
      }
      r.block = b;
    }
    if (++t == sh.t0 + sh.take) {
      more = next_share<C>(p, sh);
      t = sh.t0;
    }
    return r;
  };
  auto scales = [&](const Ref& r) {
    if (r.block < 0) return make_float2(0.f, 0.f);
    const int64_t at = static_cast<int64_t>(r.block) * p.Hkv + r.head;
    return make_float2(p.k_scale[at], p.v_scale[at]);
  };
  Ref a = take(), b = take();
  float2 sa = scales(a);
  uint32_t k_sent = 0, v_sent = 0;
  // The lanes leave together: one that gave up alone would leave the others at a __syncwarp().
  auto gave_up = [&](uint64_t* empty, uint32_t parity) { return __any_sync(0xffffffffu, !bar_wait(empty, parity, &S.failed)); };
  for (uint32_t it = 0; a.valid; ++it) {
    const float2 sb = scales(b);
    const Ref c = take();
    const uint32_t ks = it % C::kK, vs = it % C::kV, kr = it / C::kK, vr = it / C::kV;
    if (kr > 0 && gave_up(&S.k_empty[ks], (kr - 1) & 1)) break;
    if (lane == 0) bar_expect(&S.k_full[ks], kTileBytes);
    __syncwarp();
    if (lane < ppt) tma_tile(s32(S.k[ks]) + lane * rows * kD, &k_map, a.tok, a.head, a.block, &S.k_full[ks]);
    ++k_sent;
    if (vr > 0 && gave_up(&S.v_empty[vs], (vr - 1) & 1)) break;
    if (lane == 0) bar_expect(&S.v_full[vs], kTileBytes);
    __syncwarp();
    if (lane < ppt) tma_tile(s32(S.v[vs]) + lane * rows * kD, &v_map, a.tok, a.head, a.block, &S.v_full[vs]);
    ++v_sent;
    if (lane < ppt) {
      const float sv = fmaxf(sa.y, 0x1p-64f);
      S.sc[vs][lane] = a.block < 0 ? make_float4(0.f, -INFINITY, 0.f, 0.f)
                                   : make_float4(sa.x, log2f(sv), 1.f / sv, 0.f);
    }
    __syncwarp();
    if (lane == 0) bar_arrive(&S.sc_full[vs]);
    a = b, b = c, sa = sb;
  }
  // Nothing may land in shared memory after the CTA is gone.  (Where all went well the
  // last copies have been waited for by who used them, or are about to be; where another
  // role gave up, here or at the end, nobody else waits for them.)
  for (uint32_t j = k_sent > C::kK ? k_sent - C::kK : 0; j < k_sent; ++j) bar_drain(&S.k_full[j % C::kK], (j / C::kK) & 1);
  for (uint32_t j = v_sent > C::kV ? v_sent - C::kV : 0; j < v_sent; ++j) bar_drain(&S.v_full[j % C::kV], (j / C::kV) & 1);
}

// ---------------------------------------------------------------- the kernel
template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtasPerSm)
    cache_attention_kernel(const Params p, const __grid_constant__ CUtensorMap k_map,
                           const __grid_constant__ CUtensorMap v_map) {
  constexpr int kCols = C::kCols, kN = C::kN, kBlocks = C::kBlocks, kMine = C::kMine;
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem<C>& S = *reinterpret_cast<Smem<C>*>(raw);
  Bcast<C>* bcast = reinterpret_cast<Bcast<C>*>(raw + sizeof(Smem<C>));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < C::kK; ++i) bar_init(&S.k_full[i], 1), bar_init(&S.k_empty[i], 1);
    for (int i = 0; i < C::kV; ++i) bar_init(&S.v_full[i], 1), bar_init(&S.v_empty[i], 1);
    for (int i = 0; i < C::kV; ++i) bar_init(&S.sc_full[i], 1);
    for (int i = 0; i < 2; ++i) bar_init(&S.s_full[i], 1), bar_init(&S.o_full[i], 1);
    bar_init(&S.p_full, 128 * C::kGroups);
    bar_init(&S.q_full, 128 * C::kGroups);
    bar_init(&S.done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    S.failed = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&k_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&v_map) : "memory");
  }
  __syncwarp();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s32(&S.tmem)),
                 "n"(C::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  Share sh;
  const bool any = plan<C>(p, S, sh);
  const uint32_t tmem = S.tmem;
  if (any) {
    Walk& w = sh.w;
    bool more = sh.take > 0 || next_share<C>(p, sh);
    if (warp == 4 * C::kGroups) {
      // ================================================================ producer
      produce<C>(p, S, sh, more, k_map, v_map);
    } else if (warp == 4 * C::kGroups + 1) {
      // ======================================================== product issuer
      if (lane == 0) {
        constexpr uint32_t id_s = idesc(kN, false, false), id_o = idesc(kN, true, true);
        uint32_t it = 0, unit = 0;
        bool ok = true;
        auto weigh = [&](uint32_t j) {  // O^T of tile j
          const uint32_t st = j % C::kV;
          ok = ok && bar_wait(&S.p_full, j & 1, &S.failed) && bar_wait(&S.v_full[st], (j / C::kV) & 1, &S.failed);
          if (!ok) return;
          tc_after();
          const uint32_t v = s32(S.v[st]), d = tmem + (2 + (j & 1)) * kN;
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k)
              mma(d, sdesc(v + k * 32 * kD, 0, 1024, 2), sdesc(s32(S.p[part]) + k * 512, 128, 2048, 0), id_o,
                  part + k > 0);
          commit(&S.v_empty[st]);
          commit(&S.o_full[j & 1]);
        };
        for (; more && ok; ++unit) {
          for (int k0 = 0; k0 < sh.take && ok; ++k0, ++it) {
            if (k0 == 0) {
              // the rows of a new unit are in place only after the old unit's last tile is weighed
              if (it > 0) weigh(it - 1);
              ok = ok && bar_wait(&S.q_full, unit & 1, &S.failed);
            }
            const uint32_t st = it % C::kK;
            ok = ok && bar_wait(&S.k_full[st], (it / C::kK) & 1, &S.failed);
            if (!ok) break;
            tc_after();
            const uint32_t kk = s32(S.k[st]), d = tmem + (it & 1) * kN;
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int k = 0; k < kD / 32; ++k)
                mma(d, sdesc(kk + k * 32, 0, 1024, 2), sdesc(s32(S.q[part]) + k * 32 * kN, 16 * kN, 128, 0), id_s,
                    part + k > 0);
            commit(&S.s_full[it & 1]);
            commit(&S.k_empty[st]);
            if (k0 > 0) weigh(it - 1);
          }
          more = next_share<C>(p, sh);
        }
        if (ok && it > 0) weigh(it - 1);
        commit(&S.done);
      }
      __syncwarp();
    } else {
      // ================================================================ softmax
      const int g = warp >> 2, wq = warp & 3, t = tid & 127;  // warpgroup, warp in it, thread in it
      const int col0 = g * kCols;
      const int r8 = lane >> 2, pair = 2 * (lane & 3);  // of the thread's elements: lanes r8 + 8 j, columns 8 b + pair
      const int own = own_column<kMine>(lane);
      const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * wq) << 16) + col0;
      Bcast<C>& bc = bcast[warp];
      float o[4][kMine], l[kMine], rs[kMine];
      uint32_t it = 0, unit = 0;
      const int page0 = 32 * wq >> p.bs_log2, page1 = (32 * wq + 16) >> p.bs_log2;  // 0 for blocks of 128 and more
      // The rows of a unit in registers: 16 threads per row, 8 channels each.  They
      // are asked for before the unit ahead of it ends.
      uint4 v[kBlocks];
      auto load_rows = [&](const Walk& u) {
        const int row0 = u.rt * C::kRows + col0, rows = u.n * p.G - row0;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          const int c = 8 * i + (t >> 4), row = row0 + c;
          v[i] = make_uint4(0, 0, 0, 0);
          if (c < rows) {
            const int tok = token_of(p, row);
            v[i] = *reinterpret_cast<const uint4*>(p.q + (u.q0 + tok) * p.q_stride +
                                                   (static_cast<int64_t>(u.h) * p.G + row - tok * p.G) * kD + (t & 15) * 8);
          }
        }
      };
      if (more) load_rows(w);
      for (; more; ++unit) {
        const int t0 = sh.t0, take = sh.take;
        const int row0 = w.rt * C::kRows + col0;                // first of the group's query rows
        const int rows = min(max(w.n * p.G - row0, 0), kCols);  // rows that exist
        const int ctx = w.len - w.n;
        // ---- the unit's rows: scaled to e4m3's range by a power of two per row, split in two parts
        {
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) {
            const int c = 8 * i + (t >> 4), d = (t & 15) * 8;
            const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            float f[8], amax = 0.f;
            bool finite = true;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              f[2 * k] = __uint_as_float(u[k] << 16);
              f[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              finite &= fabsf(f[k]) <= FLT_MAX;
              amax = fmaxf(amax, fabsf(f[k]));
            }
#pragma unroll
            for (int s = 1; s < 16; s <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
            const uint32_t who = __ballot_sync(0xffffffffu, finite);
            finite = ((who >> (lane & 16)) & 0xffffu) == 0xffffu;
            // 2^e with amax 2^-e in (224, 448]
            const uint32_t bits = __float_as_uint(amax);
            int e = static_cast<int>(bits >> 23) - 126 - 9 + ((bits & 0x7fffffu) > 0x600000u);
            e = min(max(e, -100), 119);
            const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 y = make_float2(f[2 * k] * inv, f[2 * k + 1] * inv);
              const __nv_fp8x2_storage_t h8 = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
              const float2 back = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(h8, __NV_E4M3)));
              const __nv_fp8x2_storage_t l8 =
                  __nv_cvt_float2_to_fp8x2(make_float2(y.x - back.x, y.y - back.y), __NV_SATFINITE, __NV_E4M3);
              hi[k >> 1] |= static_cast<uint32_t>(h8) << (16 * (k & 1));
              lo[k >> 1] |= static_cast<uint32_t>(l8) << (16 * (k & 1));
            }
            const uint32_t off = (d >> 4) * (16 * kN) + (col0 + c) * 16 + (d & 8);
            *reinterpret_cast<uint2*>(S.q[0] + off) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(S.q[1] + off) = make_uint2(lo[0], lo[1]);
            if ((t & 15) == 0) {
              S.row_scale[col0 + c] = finite ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) * p.scale
                                             : __uint_as_float(0x7fc00000u);
              S.limit[col0 + c] = c < rows ? ctx + token_of(p, row0 + c) + 1 : 0;
            }
          }
        }
        if (g == 0) S.nan_at[unit & (C::kNan - 1)][t] = 0x7fffffff;
        fence_async();
        bar_arrive(&S.q_full);
        group_sync<128>(g);
        const int first_limit = ctx + token_of(p, row0) + 1;  // of the group's rows, the one that sees least
        const int tile_rows = min(w.n * p.G, (w.rt + 1) * C::kRows);
        const int least = ctx + token_of(p, w.rt * C::kRows) + 1, most = ctx + token_of(p, tile_rows - 1) + 1;  // of all groups
        float run = -INFINITY;  // running maximum of row `own`
#pragma unroll
        for (int c = 0; c < kMine; ++c) {
          rs[c] = S.row_scale[col0 + 8 * (c >> 1) + pair + (c & 1)];
          l[c] = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j][c] = 0.f;
        }

        auto add_tile = [&](uint32_t i) {  // the products of tile i join the sums
          bar_wait(&S.o_full[i & 1], (i >> 1) & 1, &S.failed);
          tc_after();
          float v[4][kMine];
          tm_ld<kBlocks>(lanes + (2 + (i & 1)) * kN, v);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            const int row = row_of_column<kBlocks>(b, lane);
            const float2 al = *reinterpret_cast<const float2*>(bc.alpha[i & 1] + row);
            const float2 be = *reinterpret_cast<const float2*>(bc.beta[i & 1] + row);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              o[j][2 * b] = o[j][2 * b] * al.x + v[j][2 * b] * be.x;
              o[j][2 * b + 1] = o[j][2 * b + 1] * al.y + v[j][2 * b + 1] * be.y;
            }
          }
        };

        for (int k = 0; k < take; ++k, ++it) {
          const uint32_t vs = it % C::kV, buf = it & 1;
          const int tile0 = (t0 + k) * kTile;
          bar_wait(&S.s_full[buf], (it >> 1) & 1, &S.failed);
          bar_wait(&S.sc_full[vs], (it / C::kV) & 1, &S.failed);
          tc_after();
          float z[4][kMine];
          tm_ld<kBlocks>(lanes + buf * kN, z);
          // a block is at least 16 tokens: lanes 0 .. 15 lie in one, 16 .. 31 in one
          const float4 sc0 = S.sc[vs][page0];
          const float4 sc1 = S.sc[vs][page1];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < kMine; ++c)
              z[j][c] = j < 2 ? fmaf(z[j][c] * sc0.x, rs[c], sc0.y) : fmaf(z[j][c] * sc1.x, rs[c], sc1.y);
          if (tile0 + kTile > first_limit) {
            const int pos = tile0 + 32 * wq + r8;
#pragma unroll
            for (int c = 0; c < kMine; ++c) {
              const int limit = S.limit[col0 + 8 * (c >> 1) + pair + (c & 1)];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (pos + 8 * j >= limit) z[j][c] = -INFINITY;
            }
          }
          // ---- the tile's maximum of every row: over the thread's tokens, the warp's, the group's
          float top;
          {
            float m[kMine];
#pragma unroll
            for (int c = 0; c < kMine; ++c) m[c] = fmaxf(fmaxf(z[0][c], z[1][c]), fmaxf(z[2][c], z[3][c]));
            top = reduce_columns<Max>(m, lane);
          }
          if (own < kCols) S.wmax[buf][g][wq][own] = top;
          group_sync<128>(g);
          if (own < kCols) {
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, S.wmax[buf][g][i][own]);
            const float next = fmaxf(run, top);
            const float ref = next == -INFINITY ? 0.f : next;
            bc.alpha[buf][own] = ex2(run - ref);
            bc.beta[buf][own] = ex2(top - ref);
            bc.mt[own] = (top == -INFINITY ? 0.f : top) - 8.f;  // weights up to 2^8
            run = next;
          }
          __syncwarp();
          // ---- weights, their sum, their two e4m3 parts (16 bits per token and pair of rows)
          uint32_t hi[4][kBlocks], lo[4][kBlocks];
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            const float2 mt = *reinterpret_cast<const float2*>(bc.mt + 8 * b + pair);
            const float2 al = *reinterpret_cast<const float2*>(bc.alpha[buf] + 8 * b + pair);
            const float2 be = *reinterpret_cast<const float2*>(bc.beta[buf] + 8 * b + pair);
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float w0 = ex2(z[j][2 * b] - mt.x), w1 = ex2(z[j][2 * b + 1] - mt.y);
              const float rv = j < 2 ? sc0.z : sc1.z;
              s0 = fmaf(w0, rv, s0);
              s1 = fmaf(w1, rv, s1);
              const __half2 x = __floats2half2_rn(w0, w1);
              const __nv_fp8x2_storage_t h = __nv_cvt_halfraw2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
              hi[j][b] = h;
              lo[j][b] = __nv_cvt_halfraw2_to_fp8x2(__hsub2(x, __half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3))),
                                                    __NV_SATFINITE, __NV_E4M3);
            }
            l[2 * b] = l[2 * b] * al.x + s0 * be.x;
            l[2 * b + 1] = l[2 * b + 1] * al.y + s1 * be.y;
          }
          if (it > 0) bar_wait(&S.o_full[(it - 1) & 1], ((it - 1) >> 1) & 1, &S.failed);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int tok = 32 * wq + r8 + 8 * j;
#pragma unroll
            for (int b = 0; b + 1 < kBlocks; b += 2) {
              const int off = (col0 / 16 + b / 2) * (16 * kTile) + tok * 16 + 2 * pair;
              *reinterpret_cast<uint32_t*>(S.p[0] + off) = hi[j][b] | (hi[j][b + 1] << 16);
              *reinterpret_cast<uint32_t*>(S.p[1] + off) = lo[j][b] | (lo[j][b + 1] << 16);
            }
            if constexpr (kBlocks & 1) {
              const int off = (col0 + 8 * (kBlocks - 1)) / 16 * (16 * kTile) + tok * 16 + (col0 + 8 * (kBlocks - 1)) % 16 + pair;
              *reinterpret_cast<uint16_t*>(S.p[0] + off) = static_cast<uint16_t>(hi[j][kBlocks - 1]);
              *reinterpret_cast<uint16_t*>(S.p[1] + off) = static_cast<uint16_t>(lo[j][kBlocks - 1]);
            }
          }
          // ---- values that some row does not see: a zero weight times NaN is
          // NaN, so what no row sees is cleared, and a NaN that only some rows
          // see is taken out here and put back into their results
          if (g == 0 && tile0 + kTile > least) {
            const int pos = tile0 + t;
            bar_wait(&S.v_full[vs], (it / C::kV) & 1, &S.failed);
            __syncwarp();
            uint4* v = reinterpret_cast<uint4*>(S.v[vs] + t * kD);
            uint32_t nan = 0;
            if (pos >= most) {
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i ^ (t & 7)] = make_uint4(0, 0, 0, 0);  // 8 threads, 8 different banks
            } else if (pos >= least) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint4 u = v[i ^ (t & 7)];
                nan |= nan_bytes(u.x) | nan_bytes(u.y) | nan_bytes(u.z) | nan_bytes(u.w);
              }
            }
            if (__any_sync(0xffffffffu, nan != 0)) take_out_nan(S.v[vs] + t * kD, nan != 0, t, pos, S.nan_at[unit & (C::kNan - 1)]);
          }
          __syncwarp();
          fence_async();
          tc_before();
          bar_arrive(&S.p_full);
          if (k > 0) add_tile(it - 1);
        }
        Share nx = sh;
        const bool then = next_share<C>(p, nx);
        if (then) load_rows(nx.w);
        add_tile(it - 1);

        // ---- the unit's end: sums over the tokens of every row
        float lsum = reduce_columns<Sum>(l, lane);
        if (own < kCols) S.wsum[g][wq][own] = lsum;
        group_sync<128>(g);
        if (own < kCols) {
          lsum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) lsum += S.wsum[g][i][own];
          const float f = S.row_scale[col0 + own];
          if (f != f && S.limit[col0 + own] > 0) lsum = f;  // a row that is not finite (one that sees nothing stays zero)
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int nan_at = S.nan_at[unit & (C::kNan - 1)][32 * wq + r8 + 8 * j];
#pragma unroll
          for (int c = 0; c < kMine; ++c)
            if (nan_at < S.limit[col0 + row_of_column<kBlocks>(c >> 1, lane) + (c & 1)])
              o[j][c] = __uint_as_float(0x7fc00000u);
        }
        // A thread and its neighbour four lanes on hold channels d, d + 1 of the
        // same two rows: each takes one row and writes both channels.
        const bool odd = r8 & 1;
        auto two_channels = [&](int j, int b) {
          const float got = __shfl_xor_sync(0xffffffffu, odd ? o[j][2 * b] : o[j][2 * b + 1], 4);
          return odd ? make_float2(got, o[j][2 * b + 1]) : make_float2(o[j][2 * b], got);
        };
        const int d0 = 32 * wq + (r8 & ~1);
        if (take == w.nt) {
          if (own < kCols) bc.mt[own] = lsum == 0.f ? 0.f : 1.f / lsum;
          __syncwarp();
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            const int c = row_of_column<kBlocks>(b, lane) + odd, row = row0 + c;
            const int tok = token_of(p, row);
            const float f = bc.mt[c];
            uint16_t* out = p.out + (w.q0 + tok) * p.out_stride +
                            (static_cast<int64_t>(w.h) * p.G + row - tok * p.G) * kD + d0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 x = two_channels(j, b);
              if (c < rows) *reinterpret_cast<__nv_bfloat162*>(out + 8 * j) = __floats2bfloat162_rn(x.x * f, x.y * f);
            }
          }
        } else if (rows > 0) {
          // a part of the unit: a record for the CTA that arrives last
          const int64_t first = sh.us + kUnitCost, cost = S.total;  // first: of the unit's tiles
          const int64_t parties = min(static_cast<int64_t>(gridDim.x), cost);
          const int c0 = static_cast<int>(((first + 1) * parties - 1) / cost);
          const int c1 = static_cast<int>(((first + w.nt) * parties - 1) / cost);
          // Records belong to a warp, its 32 channels of all rows: the warps of a group
          // join apart from one another, and none waits for the rest of its CTA.
          auto record = [&](int c) {  // of CTA c: its tail for the unit's first part, else its head
            return p.partial + ((static_cast<int64_t>(c) * 2 + (c == c0 ? 1 : 0)) * 4 * C::kGroups + 4 * g + wq) * C::kPartial;
          };
          float* rec = record(static_cast<int>(blockIdx.x));
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            const int c = row_of_column<kBlocks>(b, lane) + odd;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 x = two_channels(j, b);
              if (c < rows) *reinterpret_cast<float2*>(rec + 2 * kCols + c * 32 + (r8 & ~1) + 8 * j) = x;
            }
          }
          if (own < kCols) rec[own] = run, rec[kCols + own] = lsum;
          // Joins the records of CTAs from, from + step .. to in this order, into the
          // first of them or into the output: 8 lanes per row, four channels each.  Eight
          // parts at a time: lane = part for the maxima and sums, so that they take one
          // trip to memory, and the channels of four parts are on their way together.
          auto join = [&](int from, int step, int to, bool into_out) {
            constexpr int kAhead = C::kGroups > 1 ? 1 : kMine > 4 ? 2 : 4;
            const int sub = lane >> 3, l4 = lane & 7, parts = (to - from) / step + 1;
            float top[kMine], sum[kMine];
            float4 acc[kMine];
#pragma unroll
            for (int i = 0; i < kMine; ++i) top[i] = -INFINITY, sum[i] = 0.f, acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int n0 = 0; n0 < parts; n0 += 8) {
              const bool mine = n0 + l4 < parts;
              const float* rm = record(from + min(n0 + l4, parts - 1) * step) + sub;
              float f[kMine], part_sum[kMine];
#pragma unroll
              for (int i = 0; i < kMine; ++i) {
                f[i] = mine ? __ldcg(rm + 4 * i) : -INFINITY;
                part_sum[i] = mine ? __ldcg(rm + kCols + 4 * i) : 0.f;
              }
#pragma unroll
              for (int i = 0; i < kMine; ++i) {
                float next = fmaxf(top[i], f[i]);
#pragma unroll
                for (int s = 1; s < 8; s <<= 1) next = fmaxf(next, __shfl_xor_sync(0xffffffffu, next, s));
                const float ref = next == -INFINITY ? 0.f : next, old = ex2(top[i] - ref);
                f[i] = ex2(f[i] - ref);
                float more_sum = f[i] * part_sum[i];
#pragma unroll
                for (int s = 1; s < 8; s <<= 1) more_sum += __shfl_xor_sync(0xffffffffu, more_sum, s);
                top[i] = next;
                sum[i] = sum[i] * old + more_sum;
                acc[i].x *= old, acc[i].y *= old, acc[i].z *= old, acc[i].w *= old;
              }
#pragma unroll 1
              for (int n = 0; n < 8 && n0 + n < parts; n += kAhead) {
                float4 x[kAhead][kMine];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                  const float* rp = record(from + min(n0 + n + k, parts - 1) * step) + 2 * kCols + sub * 32;
#pragma unroll
                  for (int i = 0; i < kMine; ++i) x[k][i] = __ldcg(reinterpret_cast<const float4*>(rp + 128 * i) + l4);
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
#pragma unroll
                  for (int i = 0; i < kMine; ++i) {
                    const float w8 = __shfl_sync(0xffffffffu, f[i], (lane & 24) | (n + k));
                    if (n0 + n + k >= parts) continue;  // the warp as one
                    acc[i].x += w8 * x[k][i].x, acc[i].y += w8 * x[k][i].y;
                    acc[i].z += w8 * x[k][i].z, acc[i].w += w8 * x[k][i].w;
                  }
              }
            }
            __syncwarp();  // the warp has read the record that it may now write
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
              const int cc = sub + 4 * i;
              if (cc >= rows) continue;
              if (into_out) {
                const int row = row0 + cc, tok = token_of(p, row);
                const float f = sum[i] == 0.f ? 0.f : 1.f / sum[i];
                const __nv_bfloat162 x = __floats2bfloat162_rn(acc[i].x * f, acc[i].y * f),
                                     y = __floats2bfloat162_rn(acc[i].z * f, acc[i].w * f);
                *reinterpret_cast<uint2*>(p.out + (w.q0 + tok) * p.out_stride +
                                          (static_cast<int64_t>(w.h) * p.G + row - tok * p.G) * kD + 32 * wq + 4 * l4) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
              } else {
                float* rp = record(from);
                reinterpret_cast<float4*>(rp + 2 * kCols + cc * 32)[l4] = acc[i];
                if (l4 == 0) rp[cc] = top[i], rp[kCols + cc] = sum[i];
              }
            }
          };
          // Whether this warp is the last of `parts` to arrive at a counter, whose
          // records it then sees; the counter is left at zero.
          auto arrive = [&](int32_t* counter, int parts) {
            __syncwarp();
            int before = 0;
            if (lane == 0) {
              asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
              if (before == parts - 1) *counter = 0;
            }
            __syncwarp();  // what lane 0 acquired, the others may read (a shuffle passes the value, not the order)
            return __shfl_sync(0xffffffffu, before, 0) == parts - 1;
          };
          // Up to kJoinFan parts are joined by the last to arrive; of more, every fan
          // of neighbours by the last of them, and those by the last of all.  (One
          // place for both: code that runs once per unit costs instruction fetches.)
          const int fan = (static_cast<int>(blockIdx.x) - c0) / C::kJoinFan, fans = (c1 - c0) / C::kJoinFan + 1;
          int from = c0 + fan * C::kJoinFan, step = 1, to = min(from + C::kJoinFan - 1, c1);
          int32_t* counter = p.counters + (fan ? kCounters : 0) + (from * C::kGroups + g) * 4 + wq;
#pragma unroll 1
          for (int n = to - from + 1; arrive(counter, n); n = fans) {
            const bool all_parts = fans == 1 || step > 1;
            join(from, step, to, all_parts);
            if (all_parts) break;
            from = c0, step = C::kJoinFan, to = c1;
            counter = p.counters + 2 * kCounters + (c0 * C::kGroups + g) * 4 + wq;
          }
        }
        group_sync<128>(g);  // row_scale and limit are read: the next unit may write them
        sh = nx;
        more = then;
      }
    }
    // every product has ended before the accumulators are given back, given up or not
    if (warp == 0 && !bar_wait(&S.done, 0, &S.failed)) bar_drain(&S.done, 0);
  }
  tc_before();
  __syncthreads();
  if (tid == 0 && S.failed && p.err) atomicOr(p.err, KDA_DEVERR_TIMEOUT);
  __syncwarp();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kTmemCols));
}

// ------------------------------------------------------------ the kernel, prompts
// Here the query rows are many, so they are the 128-row operand:
//   S [row][token] = Q [row][d] K^T,   O [row][d] = P [row][token] V
// and a thread has a row of its own: its maximum, its sum and its 128 output
// channels (in registers) take no exchange with others.  The scores are read
// from tensor memory twice, for the maximum and for the weights, a row at 32
// tokens a time.  Scales, parts and one accumulator per tile as above.  The
// two warpgroups work on rows of their own, and one's arithmetic runs while
// the other waits for its products.
//
// What bounds long chunks: the chain weights -> products -> maximum -> weights of
// each group (with next to no arithmetic left between them a tile still takes
// 3,500 cycles for both groups; 5,400 with it, of which the tensor cores are
// busy 2,100).  Short ones spend less than half their time there (4 chunks of up to
// 515 tokens behind up to 4,100: 15 tiles an SM, some 40 of 90 us); by inference, not
// by a profile, the rest is what beginning, cutting and joining their units costs.  4,096 tokens behind 12,000, 64 heads: 2.17 ms (3.57 with the
// kernel above; its threads exchange maxima over shared memory).  Measured and
// left out: two threads per row (registers: 4.6 ms), products in halves of 64
// tokens (2.45 ms), 64 tokens at a time (2.2 to 2.4 ms).
//
// Two floats in one instruction.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 32 consecutive columns of this thread's lane.
__device__ __forceinline__ void tm_row(uint32_t addr, float (&r)[32]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(addr)
      : "memory");
}
// Two weights (or scaled queries) in two e4m3 parts each, 16 bits per part.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 v = __floats2half2_rn(x, y);
  hi = __nv_cvt_halfraw2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
  lo = __nv_cvt_halfraw2_to_fp8x2(
      __hsub2(v, __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(hi), __NV_E4M3))), __NV_SATFINITE,
      __NV_E4M3);
}

// SCALES: scales that 32 tokens may have (2 for blocks of 16).
template <int SCALES>
__global__ void __launch_bounds__(Wide::kThreads, 1)
    prompt_attention_kernel(const Params p, const __grid_constant__ CUtensorMap k_map,
                            const __grid_constant__ CUtensorMap v_map) {
  using C = Wide;
  extern __shared__ __align__(1024) uint8_t raw[];
  WideSmem& S = *reinterpret_cast<WideSmem*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < C::kK; ++i) bar_init(&S.k_full[i], 1), bar_init(&S.k_empty[i], 1);
    for (int i = 0; i < C::kV; ++i) bar_init(&S.v_full[i], 1), bar_init(&S.v_empty[i], 1);
    for (int i = 0; i < C::kV; ++i) bar_init(&S.sc_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      bar_init(&S.s_full[i], 1), bar_init(&S.o_full[i], 1);
      bar_init(&S.p_full[i], 128), bar_init(&S.q_full[i], 128);
    }
    bar_init(&S.done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    S.failed = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&k_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&v_map) : "memory");
  }
  __syncwarp();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(s32(&S.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  Share sh;
  const bool any = plan<C>(p, S, sh);
  const uint32_t tmem = S.tmem;
  if (any) {
    Walk& w = sh.w;
    bool more = sh.take > 0 || next_share<C>(p, sh);
    // groups that have rows of the unit
    auto active = [&](const Walk& u) { return u.n * p.G - u.rt * C::kRows > 128 ? 2 : 1; };
    if (warp >= 8) {
      // 168 a thread at launch: 256 x 216 + 128 x 72 = 384 x 168.  (More for the rows
      // and fewer here spills in the producer: 90 us against 94.)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      if (warp == 8) {
        produce<C>(p, S, sh, more, k_map, v_map);
      } else if (warp == 9) {
        // ======================================================== product issuer
        if (lane == 0) {
          constexpr uint32_t id_s = idesc(128, false, false), id_o = idesc(128, false, true);
          uint32_t it = 0, p_seen[2] = {0, 0}, units[2] = {0, 0};
          bool ok = true;
          auto weigh = [&](int g, uint32_t j) {  // O of group g for tile j, whose weights are there
            const uint32_t v = s32(S.v[j % C::kV]), d = tmem + 256 + 128 * g;
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int k = 0; k < kTile / 32; ++k)
                mma(d, sdesc(s32(S.p[g][part]) + k * 32, 0, 1024, 2), sdesc(v + k * 32 * kD, 0, 1024, 2), id_o, part + k > 0);
            commit(&S.o_full[g]);
          };
          while (more && ok) {
            const int groups = active(w);
            for (int k0 = 0; k0 <= sh.take && ok; ++k0) {  // the scores of tile k0 and the sums of the one before
              const uint32_t st = it % C::kK;
              for (int g = 0; g < groups; ++g) {
                ok = ok && (k0 > 0 ? bar_wait(&S.p_full[g], p_seen[g]++ & 1, &S.failed)
                                   : bar_wait(&S.q_full[g], units[g]++ & 1, &S.failed));
                if (k0 < sh.take && g == 0) ok = ok && bar_wait(&S.k_full[st], (it / C::kK) & 1, &S.failed);
                if (!ok) break;
                tc_after();
                if (k0 < sh.take) {
                  const uint32_t kk = s32(S.k[st]), d = tmem + 128 * g;
#pragma unroll
                  for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int k = 0; k < kD / 32; ++k)
                      mma(d, sdesc(s32(S.q[g][part]) + k * 32, 0, 1024, 2), sdesc(kk + k * 32, 0, 1024, 2), id_s, part + k > 0);
                  commit(&S.s_full[g]);
                  if (g == groups - 1) commit(&S.k_empty[st]);
                }
                if (k0 > 0) {
                  if (g == 0) ok = bar_wait(&S.v_full[(it - 1) % C::kV], ((it - 1) / C::kV) & 1, &S.failed);
                  if (!ok) break;
                  weigh(g, it - 1);
                  if (g == groups - 1) commit(&S.v_empty[(it - 1) % C::kV]);
                }
              }
              if (k0 < sh.take) ++it;
            }
            more = next_share<C>(p, sh);
          }
          commit(&S.done);
        }
        __syncwarp();
      }
    } else {
      // ================================================================ softmax
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
      const int g = warp >> 2, wq = warp & 3, t = tid & 127;  // warpgroup, warp in it, row in it
      const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * wq) << 16);
      const uint32_t s_at = lanes + 128 * g, o_at = lanes + 256 + 128 * g;
      uint8_t* const q_row = S.q[g][0] + t * 128;  // the remainders' row: 128 * kD bytes on
      uint8_t* const p_row = S.p[g][0] + t * 128;
      uint32_t it = 0, tiles = 0;                  // tiles of the share; of them those that this group took part in
      for (; more; more = next_share<C>(p, sh)) {
        const int t0 = sh.t0, take = sh.take, ctx = w.len - w.n;
        const int row0 = w.rt * C::kRows, row = row0 + 128 * g + t;
        const int tile_rows = min(w.n * p.G, row0 + C::kRows);  // end of the unit's rows
        const int least = ctx + token_of(p, row0) + 1, most = ctx + token_of(p, tile_rows - 1) + 1;
        const bool takes_part = g < active(w);
        const bool live = row < tile_rows;
        const int tok = token_of(p, min(row, tile_rows - 1));
        const int limit = live ? ctx + tok + 1 : 0x7fffffff;  // a row that is not there: no masks, never written
        const int64_t channel0 = (static_cast<int64_t>(w.h) * p.G + (row - tok * p.G)) * kD;
        if (takes_part) {
          // ---- the row: scaled to e4m3's range by a power of two, split in two parts
          float rs;
          {
            uint4 u[16];
            float amax = 0.f;
            bool finite = true;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + (w.q0 + tok) * p.q_stride + channel0);
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = live ? src[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t x[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float a = fabsf(__uint_as_float(x[k] << 16)), b = fabsf(__uint_as_float(x[k] & 0xffff0000u));
                finite &= a <= FLT_MAX && b <= FLT_MAX;
                amax = fmaxf(amax, fmaxf(a, b));
              }
            }
            // 2^e with amax 2^-e in (224, 448]
            const uint32_t bits = __float_as_uint(amax);
            int e = static_cast<int>(bits >> 23) - 126 - 9 + ((bits & 0x7fffffu) > 0x600000u);
            e = min(max(e, -100), 119);
            const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            rs = finite ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) * p.scale : __uint_as_float(0x7fc00000u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint4 v = u[2 * i + (j >> 1)];
                const uint32_t x = j & 1 ? v.z : v.x, y = j & 1 ? v.w : v.y;
                uint32_t h0, l0, h1, l1;
                split2(__uint_as_float(x << 16) * inv, __uint_as_float(x & 0xffff0000u) * inv, h0, l0);
                split2(__uint_as_float(y << 16) * inv, __uint_as_float(y & 0xffff0000u) * inv, h1, l1);
                hi[j] = h0 | (h1 << 16);
                lo[j] = l0 | (l1 << 16);
              }
              const int at = (i ^ (t & 7)) * 16;
              *reinterpret_cast<uint4*>(q_row + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4*>(q_row + 128 * kD + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
          }
          if (g == 0) {
            S.nan_at[t] = 0x7fffffff;
            if (t == 0) S.nan_seen = 0;
            group_sync<128>(0);
          }
          fence_async();
          bar_arrive(&S.q_full[g]);
          const int warp_least = __reduce_min_sync(0xffffffffu, limit);
          uint64_t o[kD / 2];
#pragma unroll
          for (int c = 0; c < kD / 2; ++c) o[c] = 0;
          float run = -INFINITY, l = 0.f;       // running maximum and sum of weights
          float alpha = 0.f, beta = 0.f;        // of the tile whose products are not yet added
          auto add_tile = [&](uint32_t j) {     // they join the sums
            bar_wait(&S.o_full[g], j & 1, &S.failed);
            tc_after();
            const uint64_t a2 = pair_of(alpha, alpha), b2 = pair_of(beta, beta);
            const bool grown = __any_sync(0xffffffffu, alpha != 1.f);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float x[32];
              tm_row(o_at + 32 * c, x);
              if (grown) {
#pragma unroll
                for (int i = 0; i < 16; ++i) o[16 * c + i] = mul2(o[16 * c + i], a2);
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) o[16 * c + i] = fma2(pair_of(x[2 * i], x[2 * i + 1]), b2, o[16 * c + i]);
            }
          };
          for (int k = 0;; ++k) {
            const uint32_t j = tiles + k, vs = (it + k) % C::kV;
            const int tile0 = (t0 + k) * kTile;
            const bool masked = tile0 + kTile > warp_least;
            float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            if (k < take) {
              bar_wait(&S.sc_full[vs], ((it + k) / C::kV) & 1, &S.failed);
              bar_wait(&S.s_full[g], j & 1, &S.failed);
              tc_after();
              // ---- the tile's maximum.  (Loops over the chunks of 32 tokens, not unrolled: the
              // loop's code has to stay in the instruction caches.)
              auto maxima = [&](auto masks) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                  float x[32];
                  tm_row(s_at + 32 * c, x);
                  const int sees = limit - tile0 - 32 * c;  // of the chunk's tokens
#pragma unroll
                  for (int part = 0; part < SCALES; ++part) {
                    const float4 sc = S.sc[vs][(32 * c + 16 * part) >> p.bs_log2];
                    const uint64_t f = pair_of(sc.x * rs, sc.x * rs), d = pair_of(sc.y, sc.y);
#pragma unroll
                    for (int i = 0; i < 16 / SCALES; ++i) {
                      const int n = 16 * part + 2 * i;
                      float2 z = both(fma2(pair_of(x[n], x[n + 1]), f, d));
                      if (masks) {
                        if (n >= sees) z.x = -INFINITY;
                        if (n + 1 >= sees) z.y = -INFINITY;
                      }
                      m[i & 3] = fmaxf(m[i & 3], fmaxf(z.x, z.y));
                    }
                  }
                }
              };
              if (masked) maxima(std::true_type{});
              else maxima(std::false_type{});
            }
            const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
            if (k > 0) add_tile(j - 1);  // (also: the weights' place is free)
            if (k == take) break;
            const float next = fmaxf(run, top), ref = next == -INFINITY ? 0.f : next;
            alpha = ex2(run - ref);
            beta = ex2(top - ref);
            run = next;
            const float mt = (top == -INFINITY ? 0.f : top) - 8.f;  // weights up to 2^8
            // ---- weights, their sum, their two e4m3 parts
            float sum = 0.f;
            auto weights = [&](auto masks) {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                float x[32];
                tm_row(s_at + 32 * c, x);
                const int sees = limit - tile0 - 32 * c;
#pragma unroll
                for (int part = 0; part < SCALES; ++part) {
                  const float4 sc = S.sc[vs][(32 * c + 16 * part) >> p.bs_log2];
                  const uint64_t f = pair_of(sc.x * rs, sc.x * rs), d = pair_of(sc.y - mt, sc.y - mt);
                  uint64_t some = 0;
#pragma unroll
                  for (int half = part; half < 3 - SCALES + part; ++half) {  // 16 tokens
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      uint32_t h[2], r[2];
#pragma unroll
                      for (int e = 0; e < 2; ++e) {
                        const int n = 16 * half + 4 * i + 2 * e;
                        float2 z = both(fma2(pair_of(x[n], x[n + 1]), f, d));
                        if (masks) {
                          if (n >= sees) z.x = -INFINITY;
                          if (n + 1 >= sees) z.y = -INFINITY;
                        }
                        const float w0 = ex2(z.x), w1 = ex2(z.y);
                        some = add2(some, pair_of(w0, w1));
                        split2(w0, w1, h[e], r[e]);
                      }
                      hi[i] = h[0] | (h[1] << 16);
                      lo[i] = r[0] | (r[1] << 16);
                    }
                    const int at = ((2 * c + half) ^ (t & 7)) * 16;
                    *reinterpret_cast<uint4*>(p_row + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(p_row + 128 * kTile + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                  }
                  const float2 two = both(some);
                  sum = fmaf(two.x + two.y, sc.z, sum);
                }
              }
            };
            if (masked) weights(std::true_type{});
            else weights(std::false_type{});
            l = l * alpha + sum * beta;
            // ---- values that some row does not see (as in the kernel above)
            if (g == 0 && tile0 + kTile > least) {
              const int pos = tile0 + t;
              bar_wait(&S.v_full[vs], ((it + k) / C::kV) & 1, &S.failed);
              __syncwarp();
              uint4* v = reinterpret_cast<uint4*>(S.v[vs] + t * kD);
              uint32_t nan = 0;
              if (pos >= most) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i ^ (t & 7)] = make_uint4(0, 0, 0, 0);
              } else if (pos >= least) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const uint4 u = v[i ^ (t & 7)];
                  nan |= nan_bytes(u.x) | nan_bytes(u.y) | nan_bytes(u.z) | nan_bytes(u.w);
                }
              }
              if (__any_sync(0xffffffffu, nan != 0)) {
                if (nan) S.nan_seen = 1;
                take_out_nan(S.v[vs] + t * kD, nan != 0, t, pos, S.nan_at);
              }
            }
            __syncwarp();
            fence_async();
            tc_before();
            bar_arrive(&S.p_full[g]);
          }
          tiles += take;
          if (S.nan_seen) {
#pragma unroll
            for (int c = 0; c < kD / 2; ++c) {
              float2 x = both(o[c]);
              if (S.nan_at[2 * c] < limit) x.x = __uint_as_float(0x7fc00000u);
              if (S.nan_at[2 * c + 1] < limit) x.y = __uint_as_float(0x7fc00000u);
              o[c] = pair_of(x.x, x.y);
            }
          }
          auto write_out = [&](float sum) {
            const float f = sum == 0.f ? 0.f : 1.f / sum;
            uint4* dst = reinterpret_cast<uint4*>(p.out + (w.q0 + tok) * p.out_stride + channel0);
            if (live) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                uint32_t r[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float2 x = both(o[4 * i + k]);
                  const __nv_bfloat162 h = __floats2bfloat162_rn(x.x * f, x.y * f);
                  r[k] = *reinterpret_cast<const uint32_t*>(&h);
                }
                dst[i] = make_uint4(r[0], r[1], r[2], r[3]);
              }
            }
          };
          if (take == w.nt) {
            write_out(l);
          } else {
            // a part of the unit: a record for the warp that arrives last, as in the kernel
            // above, but a thread's row is its own in every part
            const int64_t first = sh.us + kUnitCost, cost = S.total;
            const int64_t parties = min(static_cast<int64_t>(gridDim.x), cost);
            const int c0 = static_cast<int>(((first + 1) * parties - 1) / cost);
            const int c1 = static_cast<int>(((first + w.nt) * parties - 1) / cost);
            auto record = [&](int c) {
              return p.partial + ((static_cast<int64_t>(c) * 2 + (c == c0 ? 1 : 0)) * 4 * C::kGroups + 4 * g + wq) * C::kPartial;
            };
            auto write_record = [&](float* rec) {
              rec[lane] = run, rec[32 + lane] = l;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float2 x = both(o[2 * i]), y = both(o[2 * i + 1]);
                reinterpret_cast<float4*>(rec + 64)[32 * i + lane] = make_float4(x.x, x.y, y.x, y.y);
              }
            };
            write_record(record(static_cast<int>(blockIdx.x)));
            auto join = [&](int from, int step, int to) {
              run = -INFINITY, l = 0.f;
#pragma unroll
              for (int c = 0; c < kD / 2; ++c) o[c] = 0;
#pragma unroll 1
              for (int c = from; c <= to; c += step) {
                const float* rec = record(c);
                const float pm = __ldcg(rec + lane), pl = __ldcg(rec + 32 + lane);
                const float next = fmaxf(run, pm), ref = next == -INFINITY ? 0.f : next;
                const float a = ex2(run - ref), b = ex2(pm - ref);
                run = next;
                l = l * a + pl * b;
                const uint64_t a2 = pair_of(a, a), b2 = pair_of(b, b);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float4 x = __ldcg(reinterpret_cast<const float4*>(rec + 64) + 32 * i + lane);
                  o[2 * i] = fma2(pair_of(x.x, x.y), b2, mul2(o[2 * i], a2));
                  o[2 * i + 1] = fma2(pair_of(x.z, x.w), b2, mul2(o[2 * i + 1], a2));
                }
              }
            };
            auto arrive = [&](int32_t* counter, int parts) {
              __syncwarp();
              int before = 0;
              if (lane == 0) {
                asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
                if (before == parts - 1) *counter = 0;
              }
              __syncwarp();  // what lane 0 acquired, the others may read (as above)
              return __shfl_sync(0xffffffffu, before, 0) == parts - 1;
            };
            const int fan = (static_cast<int>(blockIdx.x) - c0) / C::kJoinFan, fans = (c1 - c0) / C::kJoinFan + 1;
            int from = c0 + fan * C::kJoinFan, step = 1, to = min(from + C::kJoinFan - 1, c1);
            int32_t* counter = p.counters + (fan ? kCounters : 0) + (from * C::kGroups + g) * 4 + wq;
#pragma unroll 1
            for (int n = to - from + 1; arrive(counter, n); n = fans) {
              const bool all_parts = fans == 1 || step > 1;
              join(from, step, to);
              if (all_parts) {
                write_out(l);
                break;
              }
              __syncwarp();
              write_record(record(from));
              from = c0, step = C::kJoinFan, to = c1;
              counter = p.counters + 2 * kCounters + (c0 * C::kGroups + g) * 4 + wq;
            }
          }
        }
        it += take;
        // both groups are behind the unit: what they share of it may be written anew
        asm volatile("barrier.cta.sync 3, 256;" ::: "memory");
      }
    }
    if (warp == 0 && !bar_wait(&S.done, 0, &S.failed)) bar_drain(&S.done, 0);
  }
  tc_before();
  __syncthreads();
  if (tid == 0 && S.failed && p.err) atomicOr(p.err, KDA_DEVERR_TIMEOUT);
  __syncwarp();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ------------------------------------------------------------------ host side
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::mutex g_mutex;
int g_sms[64];
EncodeFn g_encode;

using Rows8 = Cfg<8, 1>;
using Rows16 = Cfg<16, 1>;
using Rows24 = Cfg<24, 1>;
using Rows32 = Cfg<16, 2>;
using Rows64 = Cfg<16, 4>;
using Rows96 = Cfg<16, 6>;

template <class C>
constexpr size_t smem_bytes() {
  constexpr size_t n = sizeof(Smem<C>) + 4 * C::kGroups * sizeof(Bcast<C>);
  // an SM has 228 KB, of which each CTA's system part takes 1 KB
  static_assert((n + 1024) * C::kCtasPerSm <= 228 * 1024 && n <= 227 * 1024, "shared memory");
  return n;
}

template <>
constexpr size_t smem_bytes<Wide>() {
  static_assert(sizeof(WideSmem) <= 227 * 1024, "shared memory");
  return sizeof(WideSmem);
}

using Kernel = void (*)(const Params, const CUtensorMap, const CUtensorMap);
template <class C>
constexpr Kernel kernel_of(bool two_scales) {
  if constexpr (std::is_same<C, Wide>::value) return two_scales ? prompt_attention_kernel<2> : prompt_attention_kernel<1>;
  else return cache_attention_kernel<C>;
}
template <class C>
cudaError_t allow_smem() {
  for (bool two : {false, true}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel_of<C>(two), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem_bytes<C>()));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t setup(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!g_sms[dev]) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    g_encode = reinterpret_cast<EncodeFn>(fn);
    if ((e = allow_smem<Rows8>()) != cudaSuccess || (e = allow_smem<Rows16>()) != cudaSuccess ||
        (e = allow_smem<Rows24>()) != cudaSuccess || (e = allow_smem<Rows32>()) != cudaSuccess ||
        (e = allow_smem<Rows64>()) != cudaSuccess || (e = allow_smem<Rows96>()) != cudaSuccess ||
        (e = allow_smem<Wide>()) != cudaSuccess)
      return e;
    int n = 0;
    if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    g_sms[dev] = n < kMaxCtas / 2 ? n : kMaxCtas / 2;
  }
  *sms = g_sms[dev];
  return cudaSuccess;
}

bool misaligned(const void* ptr, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(ptr) & mask) != 0; }

// Calls `f` with the variant for `rows` query rows per kv head and sequence: all
// the queries of a single-token or multi-token step, so that the cache is read
// once and few columns are idle; the kernel for prompts from 97 on.  (64
// sequences x 12 tokens x 64 heads, 96 rows: 215 us, 274 with the kernel for
// prompts; 8 sequences x 16 tokens, 128 rows: 48 us in two tiles of 96, 44 with it.)
template <class F>
auto with_variant(int64_t rows, F f) {
  if (rows <= 8) return f(Rows8{});
  if (rows <= 16) return f(Rows16{});
  if (rows <= 24) return f(Rows24{});
  if (rows <= 32) return f(Rows32{});
  if (rows <= 64) return f(Rows64{});
  if (rows <= 96) return f(Rows96{});
  return f(Wide{});
}

template <class C>
constexpr int64_t partial_bytes() {
  return 2LL * (kMaxCtas / 2) * C::kCtasPerSm * 4 * C::kGroups * C::kPartial * static_cast<int64_t>(sizeof(float));
}

}  // namespace

extern "C" int64_t kda_cache_attention_workspace_bytes(int32_t num_q_heads, int32_t num_kv_heads, int32_t max_new) {
  if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads || max_new < 1) return -1;
  return KDA_CACHE_ATTENTION_COUNTER_BYTES + with_variant(static_cast<int64_t>(max_new) * (num_q_heads / num_kv_heads),
                                                          [](auto c) { return partial_bytes<decltype(c)>(); });
}

extern "C" int kda_cache_attention(const KdaCacheAttentionArgs* a, void* stream) {
  kda_internal_clear_error();
  if (!a) return kda_internal_fail(KDA_ERR_NULLPTR, "args is NULL");
  if (a->struct_size != sizeof(KdaCacheAttentionArgs))
    return kda_internal_fail(KDA_ERR_ABI, "struct_size %u, library expects %zu", a->struct_size,
                             sizeof(KdaCacheAttentionArgs));
  if (a->head_dim != kD) return kda_internal_fail(KDA_ERR_SHAPE, "head_dim %d (need 128)", a->head_dim);
  const int Hq = a->num_q_heads, Hkv = a->num_kv_heads, bs = a->block_size;
  if (a->B < 0 || a->T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq > 65536 || a->num_blocks < 1 || a->max_blocks < 1 ||
      a->max_new < 1)
    return kda_internal_fail(KDA_ERR_SHAPE, "B=%d T=%d num_q_heads=%d num_kv_heads=%d num_blocks=%d max_blocks=%d max_new=%d",
                             a->B, a->T, Hq, Hkv, a->num_blocks, a->max_blocks, a->max_new);
  if (static_cast<int64_t>(a->T) * (Hq / Hkv) > 0x7fffff00LL)
    return kda_internal_fail(KDA_ERR_SHAPE, "T=%d is too large", a->T);
  if (bs != 16 && bs != 32 && bs != 64 && bs != 128 && bs != 256)
    return kda_internal_fail(KDA_ERR_SHAPE, "block_size %d (need 16, 32, 64, 128 or 256)", bs);
  if (a->B == 0 || a->T == 0) return KDA_OK;
  if (!a->q || !a->out || !a->cu_seqlens || !a->seq_lens || !a->block_table || !a->k_cache || !a->v_cache ||
      !a->k_scale || !a->v_scale || !a->workspace)
    return kda_internal_fail(KDA_ERR_NULLPTR, "a required pointer is NULL");
  const int64_t width = static_cast<int64_t>(Hq) * kD;
  if (a->q_row_stride < width || a->out_row_stride < width || a->block_table_stride < a->max_blocks ||
      a->token_stride < kD || a->head_stride < kD || a->block_stride < kD)
    return kda_internal_fail(KDA_ERR_SHAPE, "a stride is smaller than the row");
  if (a->q == a->out) return kda_internal_fail(KDA_ERR_SHAPE, "out may not be q");
  const int64_t need = kda_cache_attention_workspace_bytes(Hq, Hkv, a->max_new);
  if (a->workspace_bytes < need)
    return kda_internal_fail(KDA_ERR_SHAPE, "workspace of %lld bytes, %lld needed",
                             static_cast<long long>(a->workspace_bytes), static_cast<long long>(need));
  if (misaligned(a->q, 15) || (a->q_row_stride & 7) || misaligned(a->out, 15) || (a->out_row_stride & 7) ||
      misaligned(a->cu_seqlens, 3) || misaligned(a->seq_lens, 3) || misaligned(a->block_table, 3) ||
      misaligned(a->k_cache, 15) || misaligned(a->v_cache, 15) || misaligned(a->k_scale, 3) ||
      misaligned(a->v_scale, 3) || misaligned(a->workspace, 15) || misaligned(a->err_flag, 3) ||
      ((a->block_stride | a->head_stride | a->token_stride) & 15))
    return kda_internal_fail(KDA_ERR_ALIGN, "a pointer or stride is not aligned as required");
  int sms = 0;
  cudaError_t e = setup(&sms);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "setup: %s", cudaGetErrorString(e));
  // one copy: up to 128 rows of one block and head
  const cuuint64_t dims[4] = {kD, static_cast<cuuint64_t>(bs), static_cast<cuuint64_t>(Hkv),
                              static_cast<cuuint64_t>(a->num_blocks)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(a->token_stride), static_cast<cuuint64_t>(a->head_stride),
                                 static_cast<cuuint64_t>(a->block_stride)};
  const cuuint32_t box[4] = {kD, static_cast<cuuint32_t>(bs < kTile ? bs : kTile), 1, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  CUtensorMap maps[2];
  const uint8_t* base[2] = {a->k_cache, a->v_cache};
  for (int i = 0; i < 2; ++i) {
    const CUresult r = g_encode(&maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(base[i]), dims, strides,
                                box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return kda_internal_fail(KDA_ERR_LAUNCH, "tensor map: error %d", static_cast<int>(r));
  }
  Params p{};
  p.B = a->B, p.T = a->T, p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv;
  while ((1 << p.bs_log2) < bs) ++p.bs_log2;
  // exact below 2^32 / G, and a row is below T * G
  p.g_mul = p.G > 1 && static_cast<int64_t>(a->T) * p.G * p.G < (1LL << 32) ? static_cast<uint32_t>(((1ULL << 32) + p.G - 1) / p.G) : 0;
  p.num_blocks = a->num_blocks, p.max_blocks = a->max_blocks;
  p.scale = (a->sm_scale == 0.f ? 0.08838834764831845f : a->sm_scale) * kLog2e;
  p.q = a->q, p.q_stride = a->q_row_stride, p.out = a->out, p.out_stride = a->out_row_stride;
  p.cu = a->cu_seqlens, p.lens = a->seq_lens, p.table = a->block_table, p.table_stride = a->block_table_stride;
  p.k_scale = a->k_scale, p.v_scale = a->v_scale, p.err = a->err_flag;
  p.counters = static_cast<int32_t*>(a->workspace);
  p.partial = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + KDA_CACHE_ATTENTION_COUNTER_BYTES);
  e = with_variant(static_cast<int64_t>(a->max_new) * p.G, [&](auto c) {
    using C = decltype(c);
    return kda_internal_launch(kernel_of<C>(bs == 16), dim3(static_cast<unsigned>(sms * C::kCtasPerSm)),
                               dim3(C::kThreads), smem_bytes<C>(), stream, p, maps[0], maps[1]);
  });
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
  return KDA_OK;
}
