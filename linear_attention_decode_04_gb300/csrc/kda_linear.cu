// kda_linear.cu -- matrix products with scales, bias, activation and residual
// in the epilogue (definition in include/kda_linear.h).
//
// Products are formed transposed, Y^T [channel][row] = W [channel][k] X^T: 128
// channels are the wide side of a tile and the rows of x, of which a decode
// step has few, the narrow one (16 to 256 columns).  Tiles of W and X go to
// shared memory by TMA (128 bytes of k, 128-byte swizzle), tcgen05 multiplies
// them as they are, and each of the tile's two accumulators is written out while
// the next tile's products run in the other.  With many rows two CTAs form one
// product of 256 channels, each with its half of the channels and of the rows in
// its own shared memory, so that a pair reads a tile's operands once.
//
// A gated tile has two operands of 128 channels, one of each half, and an
// accumulator for each, so that a thread has both factors of its results.
//
// Few tiles: the CTAs (or pairs) of a cluster share one tile, each with a range
// of k, and add their parts up over distributed shared memory in a fixed order.
//
// What bounds it: with few rows the weights' bytes (64 x 18,432 x 6,144 in e4m3
// 21.7 us, 5.3 TB/s; 64 x 16,384 x 6,144 gated in bf16 37.3 us, 5.4 TB/s), behind
// a start of some 4.5 us and the results of the last tile (4 x 4,608 x 2,048
// 5.9 to 6.2 us); with many the tensor cores, at the card's power limit (16,384 x 18,432 x
// 6,144 in e4m3 1.1 ms, 3.3 PFLOP/s, 0.98 ms from a cool start; 8,192 x 8,192 x
// 8,192 in bf16 0.63 ms, 1.7 PFLOP/s); with short k the results' arithmetic and
// stores (8,192 x 8,192 x 128 43 us, 3.1 TB/s written).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "kda_internal.h"
#include "kda_linear.h"
#include "kda_linear_plan.h"
#include "kda_tc.cuh"

namespace {

// Blocks of k that the tensor cores add up in one sum.  They cut every addition towards zero, which shortens the sum by
// about 2^-26 of itself per 16 products of bf16 (an eighth of that per 32 of e4m3), always in the same direction: by 2e-5
// at 16,384 of k.  So fp32 results are made from sums of 896 of k (e4m3 10,752), which are then added up in fp32 with
// rounding, in the second accumulator: they are off by 1e-6 of themselves, as sums with rounding are, at any k.  bf16
// results, whose rounding is 2^-9, are made from sums of 65,536 (786,432).  A part's end costs 0.8 us, as the products
// wait for the accumulator: 4,096 x 8,192 x 4,096 take 153 us in bf16, 163 in fp32 from sums of 2,048 (off by 2e-6) and 190 from 896.
constexpr int kSegmentF32 = 14, kSegmentBf16 = 1024, kLongerE4m3 = 6;

// Quotients of 0 .. 2^31 - 1 by a divisor of a launch (Granlund and Montgomery 1994, section 4).
struct Divisor {
  uint32_t by, factor, shift;
  Divisor() = default;
  explicit Divisor(uint32_t n) : by(n), shift(31) {
    while ((1ull << (shift - 31)) < n) ++shift;
    factor = static_cast<uint32_t>((1ull << shift) / n + 1);
  }
  __device__ __forceinline__ int of(int n) const { return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(n)) * factor >> shift); }
};

struct Params {
  int M, width;                // rows; channels of out
  int m_tiles, n_tiles, blocks;  // row tiles, channel tiles (of a CTA or pair), blocks of k
  int tile_rows;               // rows of a row tile, at most the variant's
  Divisor group, rows, last;   // tiles of a group of row tiles; row tiles of one, and of the last one
  int split, stages;           // CTAs (or pairs) per tile, ring depth
  int segment;                 // blocks of k that the tensor cores sum up at a time
  int act;
  bool out_f32, early, vec_out, vec_res;  // vec: rows in 16-byte pieces
  const float *x_scale, *w_scale, *bias;
  const uint16_t* residual;
  int64_t res_stride;
  void* out;
  int64_t out_stride;
  int32_t* err;
};

__device__ __forceinline__ uint64_t twice(float x) { return pair_of(x, x); }
__device__ __forceinline__ uint64_t sigmoid_times(uint64_t y) {
  const float2 t = both(mul2(y, twice(-1.44269504088896340736f)));
  const float2 d = both(add2(pair_of(ex2(t.x), ex2(t.y)), twice(1.f)));
  return mul2(y, pair_of(reciprocal(d.x), reciprocal(d.y)));
}
__device__ __forceinline__ float positive(float x) {  // or 0; NaN stays NaN
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
  return r;
}
// y (1 + erf(y / sqrt 2)) / 2 with erfc(x) = t e^(-x^2 + P(t)), t = 1 / (1 + x / 2),
// P of degree 9: Numerical Recipes' erfcc (Press et al., section 6.2), off by 1.2e-7
// of itself at any x >= 0, so that the lower tail keeps its digits; -x^2 = -y^2 / 2
// rounded adds x^2 2^-23.  max(y, 0) - |y| erfc(|y| / sqrt 2) / 2 is that of either
// sign; past 40, where the second part is 0, it stays so for infinity too.  (The two values belong to different rows: of
// NaN the second part is that of 40, and NaN comes from the first, so that no row reaches the other one.)
__device__ __forceinline__ uint64_t gelu(uint64_t y2) {
  const float2 y = both(y2);
  const uint64_t a = pair_of(fminf(fabsf(y.x), 40.f), fminf(fabsf(y.y), 40.f)), h = mul2(a, twice(-.5f));
  const float2 d = both(fma2(a, twice(0.35355339059327376f), twice(1.f)));  // 1 to 16
  const uint64_t t = mul2(twice(reciprocal(d.x * d.y)), pair_of(d.y, d.x));  // (one operation of the slow unit for both)
  uint64_t q = twice(0.17087277f);
  q = fma2(q, t, twice(-0.82215223f));
  q = fma2(q, t, twice(1.48851587f));
  q = fma2(q, t, twice(-1.13520398f));
  q = fma2(q, t, twice(0.27886807f));
  q = fma2(q, t, twice(-0.18628806f));
  q = fma2(q, t, twice(0.09678418f));
  q = fma2(q, t, twice(0.37409196f));
  q = fma2(q, t, twice(1.00002368f));
  q = fma2(q, t, twice(-1.26551223f));
  const float2 e = both(mul2(fma2(h, a, q), twice(1.44269504088896340736f)));
  return fma2(h, mul2(t, pair_of(ex2(e.x), ex2(e.y))), pair_of(positive(y.x), positive(y.y)));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---- A warp's part of a tile: 32 accumulator lanes, which are 32 channels or,
// interleaved, both halves of 16, BLOCKS times eight rows at a time, as fragments:
// a thread has lanes r8 + 8 j and two neighbouring rows of each block.  bf16
// results go through shared memory as four 8 x 8 matrices (eight rows of 32
// channels, or 16 of 16), their 16-byte pieces permuted so that a matrix's lie in
// different banks, and from there to memory a piece per thread: at once, or as the
// words between its ends where rows start on other boundaries.  Residuals come the
// same way, a trip ahead.
template <int GATE, int BLOCKS>
struct Epilogue {
  static constexpr int kAcc = GATE == kTwoSums ? 2 : 1;
  static constexpr int kWidth = GATE == kInterleaved ? 16 : 32;      // channels of out
  static constexpr int kRows = 256 / kWidth, kSets = 8 * BLOCKS / kRows;  // rows of four matrices; sets of them
  static constexpr int kParts = kWidth / 8;                          // pieces of a row
  static constexpr int kBytes = 16 * kParts * 8 * BLOCKS;            // of shared memory, a warp's beside the next one's of its group
  // Where a tile's rows do not end and begin on 16 bytes, the four warps of a group write them together (or a warp by itself).
  static constexpr bool kAlone = BLOCKS == 1;
  // Eight channels of a row as loaded: 16 bytes, or from an address between words the words inside, then the last two
  // bytes, and the first two.
  struct Piece {
    uint4 v;
    uint32_t head;
  };
  // What the next trip and the next tile take: loads only, so that nothing waits for them before they are used.
  struct Ahead {
    Piece res[kSets];
    float x_scale;                  // of row `lane` of the trip
    float scale[kAcc], bias[kAcc];  // of channel `lane` of the warp's, or of lane % 16 in half lane / 16
  };
  const Params& p;
  uint8_t* stage;                                                    // 8 BLOCKS rows of the warp's own
  int warp, lane, n0;
  float scale[kAcc][4], bias[kAcc][4];

  __device__ __forceinline__ Epilogue(const Params& q, uint8_t* st, int w, int ln) : p(q), stage(st), warp(w), lane(ln) {}
  __device__ __forceinline__ void group_sync() const { asm volatile("barrier.cta.sync %0, 128;" ::"r"(2 + (warp >> 2)) : "memory"); }
  __device__ __forceinline__ void tile_ahead(int first, Ahead& a) const {
    const int c = first + lane % kWidth;
#pragma unroll
    for (int h = 0; h < kAcc; ++h) {
      const int n = c + (GATE == kInterleaved ? lane / kWidth : h) * p.width;
      a.scale[h] = p.w_scale && c < p.width ? p.w_scale[n] : 1.f;
      a.bias[h] = p.bias && c < p.width ? p.bias[n] : 0.f;
    }
  }
  __device__ __forceinline__ void tile(int first, const Ahead& a) {
    n0 = first;
#pragma unroll
    for (int h = 0; h < kAcc; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        scale[h][j] = __shfl_sync(0xffffffffu, a.scale[h], (lane >> 2) + 8 * j);
        bias[h][j] = __shfl_sync(0xffffffffu, a.bias[h], (lane >> 2) + 8 * j);
      }
  }
  // block and fragment of matrix k of set s
  __device__ __forceinline__ static constexpr int block_of(int s, int k) { return GATE == kInterleaved ? 2 * s + (k >> 1) : s; }
  __device__ __forceinline__ static constexpr int lane_of(int k) { return GATE == kInterleaved ? k & 1 : k; }
  // piece k of row r in shared memory: eight rows' pieces k lie in different banks, and so do the pieces of two rows (four)
  __device__ __forceinline__ uint8_t* slot(int r, int k) const { return stage + (r * kParts + (k ^ (r / (8 / kParts) & (kParts - 1)))) * 16; }
  // this thread's row of matrix lane / 8 of set s
  __device__ __forceinline__ uint32_t matrix(int s) const {
    const int k = lane >> 3;
    return s32(slot(s * kRows + (GATE == kInterleaved ? 8 * (k >> 1) : 0) + (lane & 7), GATE == kInterleaved ? k & 1 : k));
  }
  // this thread's piece of set s: its row, its first channel, and how many of its channels there are
  __device__ __forceinline__ int row(int s) const { return s * kRows + lane / kParts; }
  __device__ __forceinline__ static int channel(int first, int ln) { return first + ln % kParts * 8; }
  __device__ __forceinline__ int there(int m, int c) const { return m < p.M ? p.width - c : 0; }
  __device__ __forceinline__ static uint32_t word(uint32_t lo, uint32_t hi) { return __funnelshift_l(lo, hi, 16); }  // across a boundary
  __device__ __forceinline__ static bool odd(const uint16_t* at) { return (reinterpret_cast<uintptr_t>(at) & 2) != 0; }
  // The rows from m on at the channels from `first` on.
  __device__ __forceinline__ void fetch(int first, int m, Ahead& a) const {
    a.x_scale = p.x_scale && lane < 8 * BLOCKS && m + lane < p.M ? p.x_scale[m + lane] : 1.f;
    if (!p.residual) return;
    Piece(&res)[kSets] = a.res;
    const int c = channel(first, lane);
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      const int n = there(m + row(s), c);
      const uint16_t* at = p.residual + (m + row(s)) * p.res_stride + c;
      if (n >= 8 && p.vec_res) {
        res[s].v = *reinterpret_cast<const uint4*>(at);
      } else if (n >= 8) {
        const bool o = odd(at);
        const uint32_t* w = reinterpret_cast<const uint32_t*>(at + o);
        if (o) res[s].head = *at;
        res[s].v.x = w[0], res[s].v.y = w[1], res[s].v.z = w[2];
        if (o) res[s].v.w = at[7];
        else res[s].v.w = w[3];
      } else {
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? at[i] : 0;
        res[s].v = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
      }
    }
  }
  // Residuals go to shared memory, in which the results follow them.
  __device__ __forceinline__ void put(int m, const Ahead& a) const {
    if (!p.residual) return;
    const Piece(&res)[kSets] = a.res;
    const int c = channel(n0, lane);
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      uint4 v = res[s].v;
      if (!p.vec_res && there(m + row(s), c) >= 8 && odd(p.residual + (m + row(s)) * p.res_stride + c))
        v = make_uint4(res[s].head | v.x << 16, word(v.x, v.y), word(v.y, v.z), v.z >> 16 | v.w << 16);
      *reinterpret_cast<uint4*>(slot(row(s), lane % kParts)) = v;
    }
  }
  // Rows m .. m + 8 BLOCKS - 1 from their sums (kTwoSums: those of the second half in `u`) and scales.
  __device__ __forceinline__ void rows(int m, float x_scale, const float (&z)[BLOCKS][4][2], const float (&u)[BLOCKS][4][2]) const {
    if (n0 >= p.width && (kAlone || p.out_f32)) return;
    constexpr int kOut = GATE == kInterleaved ? 2 : 4;
    uint64_t v[BLOCKS][kOut];
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
      const int first = 8 * b + 2 * (lane & 3);
      const uint64_t s = pair_of(__shfl_sync(0xffffffffu, x_scale, first), __shfl_sync(0xffffffffu, x_scale, first + 1));
      auto sum = [&](const float (&x)[2], int h, int j) { return fma2(mul2(pair_of(x[0], x[1]), s), twice(scale[h][j]), twice(bias[h][j])); };
#pragma unroll
      for (int j = 0; j < kOut; ++j) {
        v[b][j] = sum(z[b][j], 0, j);
        if constexpr (GATE == kTwoSums) v[b][j] = mul2(sigmoid_times(v[b][j]), sum(u[b][j], 1, j));
        if constexpr (GATE == kInterleaved) v[b][j] = mul2(sigmoid_times(v[b][j]), sum(z[b][j + 2], 0, j + 2));
      }
    }
    if constexpr (GATE == kNoGate) {
      if (p.act == KDA_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 4 * BLOCKS; ++i) v[i >> 2][i & 3] = sigmoid_times(v[i >> 2][i & 3]);
      } else if (p.act == KDA_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 4 * BLOCKS; ++i) v[i >> 2][i & 3] = gelu(v[i >> 2][i & 3]);
      }
    }
    if (p.residual) {
      __syncwarp();
#pragma unroll
      for (int s = 0; s < kSets; ++s) {
        uint32_t r[4];
        load_transposed(matrix(s), r);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint64_t& x = v[block_of(s, k)][lane_of(k)];
          x = add2(x, pair_of(__uint_as_float(r[k] << 16), __uint_as_float(r[k] & 0xffff0000u)));
        }
      }
      __syncwarp();
    }
    if (p.out_f32) {  // eight neighbouring channels of four rows at a time: whole sectors
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b) {
        const int m0 = m + 8 * b + 2 * (lane & 3);
        float* out = static_cast<float*>(p.out) + m0 * p.out_stride + n0 + (lane >> 2);
#pragma unroll
        for (int e = 0; e < 2; ++e, out += p.out_stride)
#pragma unroll
          for (int j = 0; j < kParts; ++j)
            if (m0 + e < p.M && n0 + (lane >> 2) + 8 * j < p.width) out[8 * j] = e ? both(v[b][j]).y : both(v[b][j]).x;
      }
      return;
    }
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      uint32_t r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = both(v[block_of(s, k)][lane_of(k)]);
        r[k] = pack_bf16(x.x, x.y);
      }
      store_transposed(matrix(s), r);
    }
    __syncwarp();
    const int tile0 = kAlone ? n0 : n0 - (warp & 3) * kWidth;  // the first channel written together
    if (p.vec_out && tile0 + (kAlone ? 1 : 4) * kWidth <= p.width) {
      const int c = channel(n0, lane);
#pragma unroll
      for (int s = 0; s < kSets; ++s)
        if (m + row(s) < p.M)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (m + row(s)) * p.out_stride + c) =
              *reinterpret_cast<const uint4*>(slot(row(s), lane % kParts));
    } else {
      // Of a row its 16-byte vectors, a thread each, from two pieces each, and what is left at its ends.
      constexpr int kLanes = (kAlone ? 1 : 4) * kParts, kAtOnce = 32 / kLanes, kMine = 8 * BLOCKS / (kAlone ? 1 : 4);
      const int l = lane % kLanes, width = min(p.width - tile0, (kAlone ? 1 : 4) * kWidth);
      if constexpr (!kAlone) group_sync();
#pragma unroll 2
      for (int k = lane / kLanes; k < kMine; k += kAtOnce) {
        const int r = (kAlone ? 0 : (warp & 3) * kMine) + k;
        if (m + r >= p.M) continue;
        uint16_t* const out = static_cast<uint16_t*>(p.out) + (m + r) * p.out_stride + tile0;
        // piece q of the row, in all warps' memory
        auto piece = [&](int q) { return slot(r, q % kParts) + (q / kParts - (kAlone ? 0 : warp & 3)) * kBytes; };
        const int head = min(-static_cast<int>(reinterpret_cast<uintptr_t>(out) >> 1) & 7, width), vectors = (width - head) / 8;
        if (l < vectors) {
          const uint4 a = *reinterpret_cast<const uint4*>(piece(l)), b = *reinterpret_cast<const uint4*>(piece(min(l + 1, kLanes - 1)));
          uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 6; ++i) x[i] = head & 4 ? x[i + 2] : x[i];
#pragma unroll
          for (int i = 0; i < 5; ++i) x[i] = head & 2 ? x[i + 1] : x[i];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = head & 1 ? word(x[i], x[i + 1]) : x[i];
          *reinterpret_cast<uint4*>(out + head + 8 * l) = make_uint4(x[0], x[1], x[2], x[3]);
        }
        for (int e = l; e < 8; e += kLanes) {
          const int c = head + 8 * vectors + e;
          if (e < head) out[e] = *reinterpret_cast<const uint16_t*>(piece(0) + 2 * e);
          if (c < width) out[c] = *reinterpret_cast<const uint16_t*>(piece(c / 8) + c % 8 * 2);
        }
      }
      if constexpr (!kAlone) group_sync();
    }
    __syncwarp();
  }
};

// Tiles go through the channels for a group of row tiles at a time, so that what
// runs at once shares both operands in L2.
constexpr int kGroup = 10;
struct TileAt {
  int nt, mt;
  __device__ __forceinline__ TileAt(const Params& p, int tile) {
    const int g = p.group.of(tile), first = g * static_cast<int>(p.rows.by), r = tile - first * p.n_tiles;
    const bool ends = first + static_cast<int>(p.rows.by) >= p.m_tiles;
    nt = ends ? p.last.of(r) : p.rows.of(r);
    mt = first + r - nt * static_cast<int>(ends ? p.last.by : p.rows.by);
  }
};

// ---- A tile shared by the CTAs (or pairs) of a cluster.  Each finishes a share of
// the channels: it gets the others' sums of them, and adds them up in the order of
// the CTAs.  Sums are kept as [half][pair of rows][channel], a pair of rows 64
// bytes longer than its channels so that four of them lie in different banks.
template <class C>
struct Parts {
  int channels, pitch, bytes;  // of a share: channels; bytes of a pair of rows, and of all
  __device__ __forceinline__ explicit Parts(int split) : channels(kTileN / split), pitch(channels * 8 + 64), bytes(C::kCols / 2 * pitch) {}
  // of lane channel c (of the share) and pair of rows q
  __device__ __forceinline__ uint8_t* at(uint8_t* part, int h, int q, int c) const { return part + (h * (C::kCols / C::kAcc / 2) + q) * pitch + c * 8; }
};

// The sums of a part of k in the first accumulator, of a warp's rows, added to those in the second.  (Few columns
// at a time: 16 cost registers in the calls without parts too.)
template <class C, int ROWS>
__device__ __forceinline__ void add_part(uint32_t lanes, int group, int rows, bool first) {
  constexpr int kStep = 8 * C::kUnroll;
#pragma unroll 1
  for (int col = kStep * group; col < rows; col += kStep * C::kGroups)
#pragma unroll 1
    for (int c = col; c < col + kStep * C::kAcc; c += 8) {  // (two sums: those of the second half behind the first's)
      const uint32_t from = lanes + (C::kAcc == 2 && c >= col + kStep ? c - kStep + ROWS : c);
      tm_add(from, from + C::kCols, first);
    }
  tm_put_wait();
}

// Clusters of split CTAs, or split pairs.  A pair's even CTA issues the products
// of both and counts the copies of both; its odd one copies its half and writes its
// own channels' results.
template <int ROWS, bool E4M3, int GATE, bool PAIR, bool FEW>
__global__ void __launch_bounds__(Cfg<ROWS, GATE, PAIR, FEW>::kThreads, Cfg<ROWS, GATE, PAIR, FEW>::kCtasPerSm)
    linear_kernel(const Params p, const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map) {
  using C = Cfg<ROWS, GATE, PAIR, FEW>;
  constexpr int kPair = PAIR ? 2 : 1, kCopies = 4 * C::kGroups, kIssuer = kCopies + 2;
  extern __shared__ __align__(1024) uint8_t raw[];
  Head<C>& S = *reinterpret_cast<Head<C>*>(raw + p.stages * C::kStageBytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform, to the compiler too)
  const int log2 = (PAIR ? 1 : 0) + p.split / 2;  // CTAs of a cluster (split is 1, 2 or 4)
  const int in_cluster = blockIdx.x & ((1 << log2) - 1), half = in_cluster % kPair, share = in_cluster / kPair;
  const int first = blockIdx.x >> log2, step = gridDim.x >> log2;
  const uint32_t even = in_cluster - half;  // the CTA whose barriers count
  if (warp == kCopies) {  // (so that its first copies need wait for nothing else)
    if (lane == 0) {
      for (int i = 0; i < p.stages; ++i) bar_init(&S.full[i], 2), bar_init(&S.empty[i], 1);  // (full: both kinds of copies)
      for (int i = 0; i < 2; ++i) bar_init(&S.acc_full[i], 1), bar_init(&S.acc_empty[i], kPair * 4 * C::kGroups);  // warps
      bar_init(&S.joined, 1), bar_init(&S.done, 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      S.failed = 0;
      if (p.split > 1) bar_expect(&S.joined, (p.split - 1) * Parts<C>(p.split).bytes);
      asm volatile("prefetch.tensormap [%0];" ::"l"(&w_map) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(&x_map) : "memory");
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s32(&S.tmem)), "n"(C::kTmemCols));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s32(&S.tmem)), "n"(C::kTmemCols));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
      asm volatile("barrier.cta.arrive 6, 64;" ::: "memory");
    }
    tc_before();
  }
  if (PAIR) {  // the other CTA's barriers are there
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  if (warp == kCopies) asm volatile("barrier.cta.arrive 1, %0;" ::"n"(C::kThreads) : "memory");
  else asm volatile("barrier.cta.sync 1, %0;" ::"n"(C::kThreads) : "memory");
  tc_after();
  const uint32_t tmem = warp == kCopies ? 0 : S.tmem;
  const int k0 = static_cast<int>(static_cast<int64_t>(p.blocks) * share / p.split);
  const int k1 = static_cast<int>(static_cast<int64_t>(p.blocks) * (share + 1) / p.split);
  const int tiles = p.m_tiles * p.n_tiles, mine = first < tiles ? (tiles - first + step - 1) / step : 0;  // tiles of this cluster
  // columns of the products of a row tile: fewer in one that ends early
  auto columns = [&](int mt) { return min(p.tile_rows, (p.M - mt * p.tile_rows + 16 * kPair - 1) / (16 * kPair) * (16 * kPair)); };
  if (warp == kCopies || warp == kCopies + 1) {
    // ================================================== copies: weights, rows of x
    // (Two warps: one issuing both took longer for them than a short tile's products.)
    const int span = k1 - k0;
    const int64_t total = static_cast<int64_t>(mine) * span;
    auto produce = [&](uint32_t bytes, bool early, auto copy) {
      auto expect = [&](int st) {
        if (half == 0) bar_expect(&S.full[st], kPair * bytes);
      };
      // the first round of the ring, a stage per lane: places are worked out side by side
      const bool fills = lane < p.stages && lane < total;
      const TileAt start(p, fills ? first + lane / span * step : 0);
      const int start_k = k0 + lane % span;
      if (fills) expect(lane);
      __syncwarp();
      if (early && fills) copy(lane, start, start_k);  // before the kernel ahead has ended
      asm volatile("griddepcontrol.wait;" ::: "memory");
      // Dependents start only now, when all that is ahead of this call has ended: what they read early need not be
      // written by this call alone.  (By the warp that copies rows, which knows that tensor memory has been asked for.)
      if (warp != kCopies) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      if (!early && fills) copy(lane, start, start_k);
      __syncwarp();
      // Waits have limits, and a limit counts from when only this call's own work is waited for: behind the kernel ahead,
      // and, for the warp that began without it, when tensor memory that other calls hold has been given (in a pair it
      // has been by now).
      if (!PAIR && warp == kCopies) asm volatile("barrier.cta.sync 6, 64;" ::: "memory");
      int64_t it = total < p.stages ? total : p.stages;
      int i = static_cast<int>(it) / span, k = k0 + static_cast<int>(it) % span, st = 0;
      uint32_t parity = 0;
      bool ok = true;
      for (; i < mine && ok; ++i, k = k0) {
        const TileAt at(p, first + i * step);
        for (; k < k1; ++k, ++it) {
          ok = warp_wait(&S.empty[st], parity, &S.failed);
          if (!ok) break;
          if (elect()) {
            expect(st);
            copy(st, at, k);
          }
          __syncwarp();
          if (++st == p.stages) st = 0, parity ^= 1;
        }
      }
      // nothing may land in either CTA's memory after it is gone, whoever gave up
      if (half == 0 && lane == 0)
        for (int64_t j = it > p.stages ? it - p.stages : 0; j < it; ++j)
          bar_drain(&S.full[j % p.stages], static_cast<uint32_t>(j / p.stages) & 1);
      __syncwarp();
    };
    if (warp == kCopies) {
      produce(C::kWeightBytes, p.early, [&](int st, const TileAt& at, int k) {
        const uint32_t dst = s32(raw) + st * C::kStageBytes;
        const int x = k * kBlock, y = (kPair * at.nt + half) * C::kChannels;
        if constexpr (GATE == kInterleaved) {
          static_assert(PAIR, "the map has the halves as a dimension");
#pragma unroll
          for (int i = 0; i < 4; ++i) tma_3d_pair(dst + i * 32 * kBlock, &w_map, x, y + 16 * i, 0, in_cta(&S.full[st], even));
        } else {
#pragma unroll
          for (int h = 0; h < C::kAcc; ++h) {
            if constexpr (PAIR) tma_2d_pair(dst + h * kTileN * kBlock, &w_map, x, y + h * p.width, in_cta(&S.full[st], even));
            else tma_2d(dst + h * kTileN * kBlock, &w_map, x, y + h * p.width, &S.full[st]);
          }
        }
      });
    } else {
      produce(p.tile_rows / kPair * kBlock, false, [&](int st, const TileAt& at, int k) {
        const uint32_t dst = s32(raw) + st * C::kStageBytes + C::kWeightBytes;
        const int x = k * kBlock, y = at.mt * p.tile_rows + (PAIR ? half * columns(at.mt) / 2 : 0);
        if constexpr (PAIR) tma_2d_pair(dst, &x_map, x, y, in_cta(&S.full[st], even));
        else tma_2d(dst, &x_map, x, y, &S.full[st]);
      });
    }
  } else if (warp == kIssuer) {
    // ========================================================== product issuer
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (the limits of its waits count from here)
    if (half == 0) {
      bool ok = true;
      int st = 0;
      uint32_t round = 0;
      const uint64_t desc = sdesc128(s32(raw));
      auto signal = [&](uint64_t* b) {
        if constexpr (PAIR) commit_both(b, even);
        else commit(b);
      };
      const bool parts = k1 - k0 > p.segment;
      uint32_t turn = 0;  // sums so far: in both accumulators in turn, or of parts of k in the first
      for (int i = 0; i < mine && ok; ++i) {
        const uint32_t id = idesc_k(E4M3, kPair * kTileN, columns(TileAt(p, first + i * step).mt));
        for (int from = k0; from < k1 && ok; ++turn) {
          const int to = parts ? min(from + p.segment, k1) : k1;
          const uint32_t buf = parts ? 0 : turn & 1, before = parts ? turn : turn >> 1;  // uses of this accumulator
          if (before > 0) ok = warp_wait(&S.acc_empty[buf], (before - 1) & 1, &S.failed);
          tc_after();
          for (int k = from; k < to && ok; ++k) {
            ok = warp_wait(&S.full[st], round & 1, &S.failed);
            if (!ok) break;
            tc_after();
            if (elect()) {
              // (descriptors count in 16 bytes, and no address carries out of their field)
              const uint64_t w = desc + static_cast<uint32_t>(st * (C::kStageBytes / 16)), x = w + C::kWeightBytes / 16;
#pragma unroll
              for (int j = 0; j < kBlock / 32; ++j)
#pragma unroll
                for (int h = 0; h < C::kAcc; ++h) {
                  const uint64_t a = w + h * kTileN * kBlock / 16 + 2 * j, b = x + 2 * j;
                  const uint32_t d = tmem + buf * C::kCols + h * ROWS;
                  if constexpr (PAIR) mma_2cta<E4M3>(d, a, b, id, k > from || j > 0);
                  else mma_1cta<E4M3>(d, a, b, id, k > from || j > 0);
                }
              signal(&S.empty[st]);
              if (k == to - 1) signal(&S.acc_full[buf]);
            }
            __syncwarp();
            if (++st == p.stages) st = 0, ++round;
          }
          from = to;
        }
      }
      if (elect()) signal(&S.done);
    }
    __syncwarp();
  } else {
    // ================================================================= results
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int wq = warp & 3, group = warp >> 2;  // the warp's quarter of the lanes; its group, which takes every kGroups-th block of rows
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * wq) << 16);
    const Parts<C> part(p.split);
    uint8_t* const sent = raw + p.split * part.bytes;  // what the others send
    using E = Epilogue<GATE, C::kUnroll>;
    constexpr int kStep = 8 * C::kUnroll;
    auto channel_of = [&](const TileAt& at) { return (kPair * at.nt + half) * C::kChannels; };
    TileAt at(p, first);
    E e(p, S.rows[warp], warp, lane);
    static_assert(E::kBytes == C::kRowBytes, "a warp's results");
    typename E::Ahead ahead = {};
    const bool parts = k1 - k0 > p.segment;
    uint32_t turn = 0;  // parts of k so far
    if (mine > 0 && p.split == 1) {
      e.tile_ahead(channel_of(at) + wq * E::kWidth, ahead);
      e.fetch(channel_of(at) + wq * E::kWidth, at.mt * p.tile_rows + kStep * group, ahead);
    }
    for (int i = 0; i < mine; ++i) {
      const uint32_t buf = parts ? 1 : i & 1;
      const int m0 = at.mt * p.tile_rows, rows = min(p.tile_rows, p.M - m0), channel0 = channel_of(at);
      e.tile(channel0 + wq * E::kWidth, ahead);
      if (i + 1 < mine) {
        at = TileAt(p, first + (i + 1) * step);
        e.tile_ahead(channel_of(at) + wq * E::kWidth, ahead);
      }
      if (!parts) {
        if (lane == 0) bar_wait(&S.acc_full[buf], (i >> 1) & 1, &S.failed);  // (one lane: polls are not free for the issuer)
        __syncwarp();
        tc_after();
      } else {
        // the first accumulator's sums of parts of k, added up in the second
        for (int k = k0; k < k1; k += p.segment, ++turn) {
          if (lane == 0) bar_wait(&S.acc_full[0], turn & 1, &S.failed);
          __syncwarp();
          tc_after();
          add_part<C, ROWS>(lanes, group, rows, k == k0);
          tc_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (PAIR) bar_signal_at(in_cta(&S.acc_empty[0], even));
            else bar_signal(&S.acc_empty[0]);
          }
        }
      }
      if (p.split == 1) {
        bool last;
        int col = kStep * group;
        do {  // (a group without rows only fetches for the next tile)
          const bool here = col < rows;
          if (here) e.put(m0 + col, ahead);
          const float x_scale = ahead.x_scale;
          last = col + kStep * C::kGroups >= rows;
          if (!last || i + 1 < mine)
            e.fetch(last ? channel_of(at) + wq * E::kWidth : e.n0, last ? at.mt * p.tile_rows + kStep * group : m0 + col + kStep * C::kGroups, ahead);
          if (here) {
            float z[C::kUnroll][4][2], u[C::kUnroll][4][2];
            tm_fragments(lanes + buf * C::kCols + col, z);
            if constexpr (GATE == kTwoSums) tm_fragments(lanes + buf * C::kCols + ROWS + col, u);
            e.rows(m0 + col, x_scale, z, u);
          }
          col += kStep * C::kGroups;
        } while (!last);
      } else {  // this CTA's sums, where the stages were
        uint8_t* const to = raw + (32 * wq / part.channels) * part.bytes;
#pragma unroll 1
        for (int col = kStep * group; col < rows; col += (col + 8) % kStep ? 8 : kStep * (C::kGroups - 1) + 8)
#pragma unroll
          for (int h = 0; h < C::kAcc; ++h) {
            float z[1][4][2];
            tm_fragments(lanes + buf * C::kCols + h * ROWS + col, z);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<float2*>(part.at(to, h, col / 2 + (lane & 3), 32 * wq % part.channels + (lane >> 2) + 8 * j)) = make_float2(z[0][j][0], z[0][j][1]);
          }
      }
      tc_before();
      __syncwarp();
      if (lane == 0 && !parts) {
        if constexpr (PAIR) bar_signal_at(in_cta(&S.acc_empty[buf], even));
        else bar_signal(&S.acc_empty[buf]);
      }
      if constexpr (GATE == kInterleaved) continue;  // (never split)
      else if (p.split > 1) {  // (this cluster's only tile)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        cluster_arrive();  // its stages are free
        cluster_wait();    // and so are the others', and all of its own sums are in place
        if (tid < p.split && tid != share) {
          const uint32_t cta = tid * kPair + half;
          send(in_cta(sent + share * part.bytes, cta), raw + tid * part.bytes, part.bytes, in_cta(&S.joined, cta));
        }
        __syncwarp();
        // blocks of 32 channels and a few rows, a warp each
        const int wide = part.channels / 32, cb = warp % wide * 32;
        using Own = Epilogue<GATE, 1>;
        Own own(p, S.rows[warp], warp, lane);
        typename Own::Ahead own_ahead = {};
        own.tile_ahead(channel0 + share * part.channels + cb, own_ahead);
        own.tile(channel0 + share * part.channels + cb, own_ahead);
        if (lane == 0) bar_wait(&S.joined, 0, &S.failed);
        __syncwarp();
#pragma unroll 1
        for (int block = warp; block < wide * (ROWS / 8); block += 4 * C::kGroups) {
          const int col = block / wide * 8;
          if (col >= rows) break;
          own.fetch(own.n0, m0 + col, own_ahead);
          float s[2][1][4][2] = {};
#pragma unroll 1
          for (int r = 0; r < p.split; ++r)
#pragma unroll
            for (int h = 0; h < C::kAcc; ++h)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 v = *reinterpret_cast<const float2*>(
                    part.at((r == share ? raw : sent) + r * part.bytes, h, col / 2 + (lane & 3), cb + (lane >> 2) + 8 * j));
                s[h][0][j][0] += v.x, s[h][0][j][1] += v.y;
              }
          own.put(m0 + col, own_ahead);
          own.rows(m0 + col, own_ahead.x_scale, s[0], s[1]);
        }
      }
    }
  }
  if (p.split > 1 && warp >= 4 * C::kGroups) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  // (A pair's odd CTA has no products to issue, which may take the pair longer than a wait may: it waits for the last of
  // them when its results are written.)
  if (PAIR && half != 0) __syncthreads();
  // every product has ended before the accumulators are given back, and in a pair before either CTA leaves, given up or not
  if (warp == kIssuer && lane == 0 && !bar_wait(&S.done, 0, &S.failed)) bar_drain(&S.done, 0);
  __syncwarp();
  tc_before();
  __syncthreads();
  if (tid == 0 && S.failed && p.err) atomicOr(p.err, KDA_DEVERR_TIMEOUT);
  __syncwarp();
  // (what a CTA sent is read from its memory until the others have it)
  if (PAIR || p.split > 1) {
    cluster_arrive();
    cluster_wait();
    // where sums were given up on, they may still be on their way here
    if (p.split > 1 && S.failed && tid < 32) bar_drain(&S.joined, 0);
  }
  if (warp == kIssuer) {
    if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kTmemCols));
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kTmemCols));
  }
}

// ------------------------------------------------------------------ host side
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::mutex g_mutex;
int g_sms[64];
EncodeFn g_encode;

using Kernel = void (*)(const Params, const CUtensorMap, const CUtensorMap);
#define KDA_LINEAR_KERNELS(ROWS, GATE, PAIR, FEW, ...) {linear_kernel<ROWS, false, GATE, PAIR, FEW>, linear_kernel<ROWS, true, GATE, PAIR, FEW>},
const Kernel kKernels[][2] = {KDA_LINEAR_VARIANTS(KDA_LINEAR_KERNELS)};  // of kVariants, for bf16 and e4m3
#undef KDA_LINEAR_KERNELS

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
    for (const auto& of_types : kKernels)
      for (const Kernel k : of_types)
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit)) != cudaSuccess) return e;
    int n = 0;
    if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    g_sms[dev] = n;
  }
  *sms = g_sms[dev];
  return cudaSuccess;
}

bool misaligned(const void* ptr, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(ptr) & mask) != 0; }

}  // namespace

extern "C" int kda_linear(const KdaLinearArgs* a, void* stream) {
  kda_internal_clear_error();
  if (!a) return kda_internal_fail(KDA_ERR_NULLPTR, "args is NULL");
  if (a->struct_size != sizeof(KdaLinearArgs))
    return kda_internal_fail(KDA_ERR_ABI, "struct_size %u, library expects %zu", a->struct_size, sizeof(KdaLinearArgs));
  if (a->flags & ~(KDA_LINEAR_E4M3 | KDA_LINEAR_OUT_F32 | KDA_LINEAR_EARLY_WEIGHT))
    return kda_internal_fail(KDA_ERR_FLAGS, "unknown flags 0x%x", a->flags);
  const bool e4m3 = a->flags & KDA_LINEAR_E4M3, f32 = a->flags & KDA_LINEAR_OUT_F32;
  const bool gated = a->activation == KDA_ACT_SILU_GATED;
  constexpr int kMost = 1 << 24;
  constexpr int kMostRows = 0x7fffffff - 511;  // rows are counted in 32 bits, to the end of the last tile and what is read ahead
  if (a->M < 0 || a->M > kMostRows || a->N < 1 || a->N > kMost || a->K < 1 || a->K > kMost || a->activation < 0 ||
      a->activation > KDA_ACT_SILU_GATED || (gated && a->N % 2))
    return kda_internal_fail(KDA_ERR_SHAPE, "M=%d N=%d K=%d activation=%d", a->M, a->N, a->K, a->activation);
  if (a->M == 0) return KDA_OK;
  if (!a->x || !a->weight || !a->out || (a->x_scale != nullptr) != e4m3 || (a->weight_scale != nullptr) != e4m3)
    return kda_internal_fail(KDA_ERR_NULLPTR, "a required pointer is NULL (x_scale and weight_scale go with e4m3, and only with it)");
  const int width = gated ? a->N / 2 : a->N;
  if (a->x_row_stride < a->K || a->weight_row_stride < a->K || a->out_row_stride < width ||
      (a->residual && a->residual_row_stride < width) || a->x_row_stride >= 1LL << 32 || a->weight_row_stride >= 1LL << 32)
    return kda_internal_fail(KDA_ERR_SHAPE, "a row stride is smaller than the row, or 2^32 elements and more");
  const int64_t each = e4m3 ? 15 : 7;
  if (misaligned(a->x, 15) || misaligned(a->weight, 15) || (a->x_row_stride & each) || (a->weight_row_stride & each) ||
      misaligned(a->x_scale, 3) || misaligned(a->weight_scale, 3) || misaligned(a->bias, 3) || misaligned(a->residual, 1) ||
      misaligned(a->out, f32 ? 3 : 1) || misaligned(a->err_flag, 3))
    return kda_internal_fail(KDA_ERR_ALIGN, "a pointer or stride is not aligned as required");
  if (a->out == a->x || a->out == a->weight ||
      (a->out == a->residual && (f32 || a->out_row_stride != a->residual_row_stride)))
    return kda_internal_fail(KDA_ERR_SHAPE, "out may take the place of a bf16 residual of the same stride, and of nothing else");
  int sms = 0;
  cudaError_t e = setup(&sms);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "setup: %s", cudaGetErrorString(e));
  const cuuint64_t size = e4m3 ? 1 : 2;
  const cuuint64_t k_bytes = static_cast<cuuint64_t>(a->K) * size;
  const cuuint64_t w_pitch = static_cast<cuuint64_t>(a->weight_row_stride) * size, x_pitch = static_cast<cuuint64_t>(a->x_row_stride) * size;
  const cuuint32_t ones[3] = {1, 1, 1};
  const int blocks = static_cast<int>((k_bytes + kBlock - 1) / kBlock);
  const bool vec_out = !f32 && !misaligned(a->out, 15) && a->out_row_stride % 8 == 0;
  const Plan plan = plan_of(a->M, width, blocks, gated, static_cast<double>(k_bytes) * a->N, sms, f32 || vec_out);
  const Variant& v = kVariants[plan.variant];
  CUtensorMap w_map, x_map;
  CUresult r;
  if (v.interleaved) {  // a copy takes 16 channels of each half
    const cuuint64_t dims[3] = {k_bytes, static_cast<cuuint64_t>(width), 2};
    const cuuint64_t strides[2] = {w_pitch, w_pitch * static_cast<cuuint64_t>(width)};
    const cuuint32_t box[3] = {kBlock, 16, 2};
    r = g_encode(&w_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(a->weight), dims, strides, box, ones,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else {
    const cuuint64_t dims[2] = {k_bytes, static_cast<cuuint64_t>(a->N)};
    const cuuint64_t strides[1] = {w_pitch};
    const cuuint32_t box[2] = {kBlock, kTileN};
    r = g_encode(&w_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(a->weight), dims, strides, box, ones,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (r == CUDA_SUCCESS) {
    const cuuint64_t dims[2] = {k_bytes, static_cast<cuuint64_t>(a->M)};
    const cuuint64_t strides[1] = {x_pitch};
    const cuuint32_t box[2] = {kBlock, static_cast<cuuint32_t>(plan.tile_rows / (v.pair ? 2 : 1))};
    r = g_encode(&x_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(a->x), dims, strides, box, ones,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (r != CUDA_SUCCESS) return kda_internal_fail(KDA_ERR_LAUNCH, "tensor map: error %d", static_cast<int>(r));
  Params p{};
  p.M = a->M, p.width = width;
  const int64_t m_tiles = tiles_of(a->M, plan.tile_rows), n_tiles = tiles_of(width, v.channels);
  if (m_tiles * n_tiles > 0x7fffffff / 16) return kda_internal_fail(KDA_ERR_SHAPE, "M=%d N=%d: too many tiles", a->M, a->N);
  p.m_tiles = static_cast<int>(m_tiles), p.n_tiles = static_cast<int>(n_tiles), p.blocks = blocks;
  const int groups = static_cast<int>((m_tiles + kGroup - 1) / kGroup), of_group = static_cast<int>((m_tiles + groups - 1) / groups);
  p.group = Divisor(static_cast<uint32_t>(of_group * n_tiles)), p.rows = Divisor(static_cast<uint32_t>(of_group));
  p.last = Divisor(static_cast<uint32_t>(m_tiles - (m_tiles - 1) / of_group * of_group));
  p.segment = (f32 ? kSegmentF32 : kSegmentBf16) * (e4m3 ? kLongerE4m3 : 1);
  p.split = plan.split, p.stages = plan.stages, p.tile_rows = plan.tile_rows;
  p.act = a->activation, p.out_f32 = f32, p.early = a->flags & KDA_LINEAR_EARLY_WEIGHT;
  p.x_scale = a->x_scale, p.w_scale = a->weight_scale, p.bias = a->bias;
  p.residual = a->residual, p.res_stride = a->residual_row_stride, p.out = a->out, p.out_stride = a->out_row_stride;
  p.err = a->err_flag;
  p.vec_out = vec_out;
  p.vec_res = !misaligned(a->residual, 15) && a->residual_row_stride % 8 == 0;
  const int cluster = plan.split * (v.pair ? 2 : 1);
  const int64_t clusters = plan.split > 1 ? m_tiles * n_tiles : std::min<int64_t>(m_tiles * n_tiles, sms / cluster);
  e = kda_internal_launch_cluster(kKernels[plan.variant][e4m3], dim3(static_cast<unsigned>(clusters * cluster)), dim3(static_cast<unsigned>(v.threads)),
                                  static_cast<size_t>(v.head_bytes + plan.stages * v.stage_bytes), stream,
                                  static_cast<unsigned>(cluster), p, w_map, x_map);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
  return KDA_OK;
}
