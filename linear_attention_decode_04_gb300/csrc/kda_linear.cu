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
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "kda_internal.h"
#include "kda_linear.h"
#include "kda_tc.cuh"

namespace {

constexpr int kTileN = 128;                // channels of a CTA's tile
constexpr int kBlock = 128;                // bytes of k per stage
constexpr int kMaxSplit = 4;
constexpr int kMaxStages = 12;
constexpr int kPitch = 80;                 // bytes between rows of results in shared memory

struct Params {
  int M, N, K, width;          // width: channels of out
  int m_tiles, n_tiles, blocks;  // row tiles, channel tiles (of a CTA or pair), blocks of k
  int split, stages;           // CTAs (or pairs) per tile, ring depth
  int act;
  bool out_f32, early, vec_out, vec_res;  // vec: rows in 16-byte pieces
  const float *x_scale, *w_scale, *bias;
  const uint16_t* residual;
  int64_t res_stride;
  void* out;
  int64_t out_stride;
  int32_t* err;
};

// A gate's two halves: in two accumulators, or 16 and 16 channels in turn in one.
constexpr int kNoGate = 0, kTwoSums = 1, kInterleaved = 2;

// ROWS of x per tile.
template <int ROWS, int GATE, bool PAIR>
struct Cfg {
  static constexpr int kAcc = GATE == kTwoSums ? 2 : 1;
  static constexpr int kChannels = GATE == kInterleaved ? kTileN / 2 : kTileN;  // of out, of a CTA
  static constexpr int kUnroll = PAIR || ROWS > 64 ? 4 : 2;  // blocks of eight rows that a warp writes at a time
  static constexpr int kWeightBytes = kAcc * kTileN * kBlock, kXRows = PAIR ? ROWS / 2 : ROWS;
  static constexpr int kStageBytes = kWeightBytes + kXRows * kBlock;
  static constexpr int kCols = kAcc * ROWS;      // accumulator columns of a tile, of which there are two sets
  static constexpr int kTmemCols = 2 * kCols;    // a power of two from 32 on
  // One CTA takes an SM's shared memory; where a short range of k leaves room, the next call's CTAs start beside it.
  static constexpr int kCtasPerSm = PAIR || ROWS > 64 ? 1 : 2;
  // warpgroups that write results; then a warp that copies weights, one that copies rows, and the issuer
  static constexpr int kGroups = kCtasPerSm == 1 ? 2 : 1, kThreads = 128 * kGroups + 96;
  // sums of a tile that several CTAs share: in the stages, when its products have ended, lie a CTA's own and those sent to it
  static constexpr int kPartBytes = kCols / 2 * (kTileN * 8 + 64 * kMaxSplit);
  static_assert(kTmemCols * kCtasPerSm <= 512, "tensor memory");
};

// Shared memory: the stages, then this.
template <class C>
struct Head {
  alignas(16) uint8_t rows[4 * C::kGroups][8 * C::kUnroll * kPitch];  // of the warps that write results
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], joined, done;
  uint32_t tmem;
  int failed;
};

__device__ __forceinline__ float sigmoid_times(float y) { return __fdividef(y, 1.f + __expf(-y)); }
// y (1 + erf(y / sqrt 2)) / 2 with erfc(x) = t e^(-x^2 + P(t)), t = 1 / (1 + x / 2),
// P of degree 9: Numerical Recipes' erfcc (Press et al., section 6.2), off by 1.2e-7
// of itself at any x >= 0, so that the lower tail keeps its digits; -x^2 rounded
// adds x^2 2^-23.
__device__ __forceinline__ float gelu(float y) {
  const float x = fabsf(y) * 0.70710678118654752f, t = __fdividef(1.f, fmaf(0.5f, x, 1.f));
  float q = 0.17087277f;
  q = fmaf(q, t, -0.82215223f);
  q = fmaf(q, t, 1.48851587f);
  q = fmaf(q, t, -1.13520398f);
  q = fmaf(q, t, 0.27886807f);
  q = fmaf(q, t, -0.18628806f);
  q = fmaf(q, t, 0.09678418f);
  q = fmaf(q, t, 0.37409196f);
  q = fmaf(q, t, 1.00002368f);
  q = fmaf(q, t, -1.26551223f);
  const float half = 0.5f * t * __expf(fmaf(-x, x, q));  // the normal distribution's lower tail
  return y * (y > 0.f ? 1.f - half : half);
}
__device__ __forceinline__ float of_bf16(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---- A warp's part of a tile: 32 accumulator lanes, which are 32 channels or,
// interleaved, both halves of 16, BLOCKS times eight rows at a time, as fragments:
// a thread has lanes r8 + 8 j and two neighbouring rows of each block.  bf16
// results go through shared memory as four 8 x 8 matrices (eight rows of 32
// channels, or 16 of 16), rows 80 bytes apart so that they lie in different banks,
// and from there to memory 16 bytes a thread; residuals come the same way, a trip
// ahead.  (A loop of few instructions: in a short launch all of them are fetched
// for the first time, which with 32 rows unrolled took longer than the products of
// a small matrix.)
template <int GATE, int BLOCKS>
struct Epilogue {
  static constexpr int kAcc = GATE == kTwoSums ? 2 : 1;
  static constexpr int kWidth = GATE == kInterleaved ? 16 : 32;      // channels of out
  static constexpr int kRows = 256 / kWidth, kSets = 8 * BLOCKS / kRows;  // rows of four matrices; sets of them
  static constexpr int kParts = kWidth / 8;                          // 16-byte pieces of a row
  const Params& p;
  uint8_t* stage;                                                    // 8 BLOCKS rows of the warp's own
  int lane, n0;
  float scale[kAcc][4], bias[kAcc][4];

  __device__ __forceinline__ Epilogue(const Params& q, uint8_t* st, int channel0, int ln) : p(q), stage(st), lane(ln), n0(channel0) {
#pragma unroll
    for (int h = 0; h < kAcc; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = n0 + (lane >> 2) + 8 * (GATE == kInterleaved ? j & 1 : j), n = c + (GATE == kInterleaved ? j >> 1 : h) * p.width;
        const bool live = c < p.width;
        scale[h][j] = live && p.w_scale ? p.w_scale[n] : 1.f;
        bias[h][j] = live && p.bias ? p.bias[n] : 0.f;
      }
  }
  __device__ __forceinline__ bool whole() const { return n0 + kWidth <= p.width; }
  // block and fragment of matrix k of set s
  __device__ __forceinline__ static constexpr int block_of(int s, int k) { return GATE == kInterleaved ? 2 * s + (k >> 1) : s; }
  __device__ __forceinline__ static constexpr int lane_of(int k) { return GATE == kInterleaved ? k & 1 : k; }
  // this thread's row of set s
  __device__ __forceinline__ uint32_t matrix(int s) const {
    const int k = lane >> 3, row = GATE == kInterleaved ? 8 * (k >> 1) + (lane & 7) : lane & 7;
    return s32(stage) + (s * kRows + row) * kPitch + (GATE == kInterleaved ? k & 1 : k) * 16;
  }
  // The residuals of the sets from row m on: 16 bytes of a row, or eight rows of a channel.
  __device__ __forceinline__ void fetch(int m, uint4 (&res)[kSets]) const {
    if (!p.residual || n0 >= p.width) return;
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      if (p.vec_res && whole()) {
        const int at = m + s * kRows + lane / kParts;
        res[s] = at < p.M ? *reinterpret_cast<const uint4*>(p.residual + at * p.res_stride + n0 + lane % kParts * 8) : make_uint4(0, 0, 0, 0);
      } else {
        uint32_t v[8];
        const int row = m + s * kRows + lane / kWidth, c = n0 + lane % kWidth;
        const uint16_t* at = p.residual + row * p.res_stride + c;
#pragma unroll
        for (int i = 0; i < 8; ++i, at += p.res_stride * (32 / kWidth)) v[i] = row + i * (32 / kWidth) < p.M && c < p.width ? *at : 0;
        res[s] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
      }
    }
  }
  // Rows m .. m + 8 BLOCKS - 1 from their sums (kTwoSums: those of the second half in `u`).
  __device__ __forceinline__ void rows(int m, float (&z)[BLOCKS][4][2], float (&u)[BLOCKS][4][2], const uint4 (&res)[kSets]) const {
    if (n0 >= p.width) return;
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
      const int m0 = m + 8 * b + 2 * (lane & 3);
      const float s[2] = {p.x_scale && m0 < p.M ? p.x_scale[m0] : 1.f, p.x_scale && m0 + 1 < p.M ? p.x_scale[m0 + 1] : 1.f};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          z[b][j][e] = fmaf(z[b][j][e] * s[e], scale[0][j], bias[0][j]);
          if constexpr (GATE == kTwoSums) z[b][j][e] = sigmoid_times(z[b][j][e]) * fmaf(u[b][j][e] * s[e], scale[1][j], bias[1][j]);
        }
        if constexpr (GATE == kInterleaved)
#pragma unroll
          for (int j = 0; j < 2; ++j) z[b][j][e] = sigmoid_times(z[b][j][e]) * z[b][j + 2][e];
      }
    }
    if constexpr (GATE == kNoGate) {
      if (p.act == KDA_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 8 * BLOCKS; ++i) z[i >> 3][(i >> 1) & 3][i & 1] = sigmoid_times(z[i >> 3][(i >> 1) & 3][i & 1]);
      } else if (p.act == KDA_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 8 * BLOCKS; ++i) z[i >> 3][(i >> 1) & 3][i & 1] = gelu(z[i >> 3][(i >> 1) & 3][i & 1]);
      }
    }
    if (p.residual) {
#pragma unroll
      for (int s = 0; s < kSets; ++s) {
        if (p.vec_res && whole()) {
          *reinterpret_cast<uint4*>(stage + (s * kRows + lane / kParts) * kPitch + lane % kParts * 16) = res[s];
        } else {
          const uint32_t w[4] = {res[s].x, res[s].y, res[s].z, res[s].w};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint16_t*>(stage + (s * kRows + lane / kWidth + i * (32 / kWidth)) * kPitch + lane % kWidth * 2) =
                static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        }
      }
      __syncwarp();
#pragma unroll
      for (int s = 0; s < kSets; ++s) {
        uint32_t r[4];
        load_transposed(matrix(s), r);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float(&v)[2] = z[block_of(s, k)][lane_of(k)];
          v[0] += of_bf16(r[k] & 0xffffu), v[1] += of_bf16(r[k] >> 16);
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
            if (m0 + e < p.M && n0 + (lane >> 2) + 8 * j < p.width) out[8 * j] = z[b][j][e];
      }
      return;
    }
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      uint32_t r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = pack_bf16(z[block_of(s, k)][lane_of(k)][0], z[block_of(s, k)][lane_of(k)][1]);
      store_transposed(matrix(s), r);
    }
    __syncwarp();
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      if (p.vec_out && whole()) {
        const int at = m + s * kRows + lane / kParts;
        const uint4 v = *reinterpret_cast<const uint4*>(stage + (s * kRows + lane / kParts) * kPitch + lane % kParts * 16);
        if (at < p.M) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * p.out_stride + n0 + lane % kParts * 8) = v;
      } else {
        const int row = s * kRows + lane / kWidth, c = n0 + lane % kWidth;
        uint16_t* out = static_cast<uint16_t*>(p.out) + (m + row) * p.out_stride + c;
#pragma unroll
        for (int i = 0; i < 8; ++i, out += p.out_stride * (32 / kWidth)) {
          const uint16_t v = *reinterpret_cast<const uint16_t*>(stage + (row + i * (32 / kWidth)) * kPitch + lane % kWidth * 2);
          if (m + row + i * (32 / kWidth) < p.M && c < p.width) *out = v;
        }
      }
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
    const int groups = (p.m_tiles + kGroup - 1) / kGroup, size = (p.m_tiles + groups - 1) / groups;
    const int g = tile / (size * p.n_tiles), first = g * size;
    const int here = min(size, p.m_tiles - first), r = tile - first * p.n_tiles;
    nt = r / here;
    mt = first + r - nt * here;
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

// Clusters of split CTAs, or split pairs.  A pair's even CTA issues the products
// of both and counts the copies of both; its odd one copies its half and writes its
// own channels' results.
template <int ROWS, bool E4M3, int GATE, bool PAIR>
__global__ void __launch_bounds__(Cfg<ROWS, GATE, PAIR>::kThreads, Cfg<ROWS, GATE, PAIR>::kCtasPerSm)
    linear_kernel(const Params p, const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map) {
  using C = Cfg<ROWS, GATE, PAIR>;
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = warp == kCopies ? 0 : S.tmem;
  const int k0 = static_cast<int>(static_cast<int64_t>(p.blocks) * share / p.split);
  const int k1 = static_cast<int>(static_cast<int64_t>(p.blocks) * (share + 1) / p.split);
  const int tiles = p.m_tiles * p.n_tiles, mine = first < tiles ? (tiles - first + step - 1) / step : 0;  // tiles of this cluster
  // columns of the products of a row tile: fewer in one that ends early
  auto columns = [&](int mt) { return min(ROWS, (p.M - mt * ROWS + 16 * kPair - 1) / (16 * kPair) * (16 * kPair)); };
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
      if (!early && fills) copy(lane, start, start_k);
      __syncwarp();
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
      produce(C::kXRows * kBlock, false, [&](int st, const TileAt& at, int k) {
        const uint32_t dst = s32(raw) + st * C::kStageBytes + C::kWeightBytes;
        const int x = k * kBlock, y = at.mt * ROWS + (PAIR ? half * columns(at.mt) / 2 : 0);
        if constexpr (PAIR) tma_2d_pair(dst, &x_map, x, y, in_cta(&S.full[st], even));
        else tma_2d(dst, &x_map, x, y, &S.full[st]);
      });
    }
  } else if (warp == kIssuer) {
    // ========================================================== product issuer
    if (half == 0) {
      bool ok = true;
      int st = 0;
      uint32_t round = 0;
      const uint64_t desc = sdesc128(s32(raw));
      auto signal = [&](uint64_t* b) {
        if constexpr (PAIR) commit_both(b, even);
        else commit(b);
      };
      for (int i = 0; i < mine && ok; ++i) {
        const uint32_t buf = i & 1, id = idesc_k(E4M3, kPair * kTileN, columns(TileAt(p, first + i * step).mt));
        if (i >= 2) ok = warp_wait(&S.acc_empty[buf], ((i >> 1) - 1) & 1, &S.failed);
        tc_after();
        for (int k = k0; k < k1 && ok; ++k) {
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
                if constexpr (PAIR) mma_2cta<E4M3>(d, a, b, id, k > k0 || j > 0);
                else mma_1cta<E4M3>(d, a, b, id, k > k0 || j > 0);
              }
            signal(&S.empty[st]);
            if (k == k1 - 1) signal(&S.acc_full[buf]);
          }
          __syncwarp();
          if (++st == p.stages) st = 0, ++round;
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
    for (int i = 0; i < mine; ++i) {
      const uint32_t buf = i & 1;
      const TileAt at(p, first + i * step);
      const int m0 = at.mt * ROWS;
      using E = Epilogue<GATE, C::kUnroll>;
      const int channel0 = (kPair * at.nt + half) * C::kChannels;
      E e(p, S.rows[warp], channel0 + wq * E::kWidth, lane);
      constexpr int kStep = 8 * C::kUnroll;
      uint4 ahead[E::kSets] = {};
      if (p.split == 1) e.fetch(m0 + kStep * group, ahead);
      if (p.x_scale && lane < ROWS / 32 + 1 && m0 + 32 * lane < p.M) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.x_scale + m0 + 32 * lane));
      if (lane == 0) bar_wait(&S.acc_full[buf], (i >> 1) & 1, &S.failed);  // (one lane: polls are not free for the issuer)
      __syncwarp();
      tc_after();
      if (p.split == 1) {
#pragma unroll 1
        for (int col = kStep * group; col < ROWS && m0 + col < p.M; col += kStep * C::kGroups) {
          float z[C::kUnroll][4][2], u[C::kUnroll][4][2];
          tm_fragments(lanes + buf * C::kCols + col, z);
          if constexpr (GATE == kTwoSums) tm_fragments(lanes + buf * C::kCols + ROWS + col, u);
          uint4 res[E::kSets];
#pragma unroll
          for (int i = 0; i < E::kSets; ++i) res[i] = ahead[i];
          if (col + kStep * C::kGroups < ROWS) e.fetch(m0 + col + kStep * C::kGroups, ahead);
          e.rows(m0 + col, z, u, res);
        }
      } else {  // this CTA's sums, where the stages were
        uint8_t* const to = raw + (32 * wq / part.channels) * part.bytes;
#pragma unroll 1
        for (int col = 8 * group; col < ROWS && m0 + col < p.M; col += 8 * C::kGroups)
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
      if (lane == 0) {
        if constexpr (PAIR) bar_arrive_at(in_cta(&S.acc_empty[buf], even));
        else bar_arrive(&S.acc_empty[buf]);
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
        const Own own(p, S.rows[warp], channel0 + share * part.channels + cb, lane);
        if (lane == 0) bar_wait(&S.joined, 0, &S.failed);
        __syncwarp();
#pragma unroll 1
        for (int block = warp; block < wide * (ROWS / 8); block += 4 * C::kGroups) {
          const int col = block / wide * 8;
          if (m0 + col >= p.M) break;
          uint4 res[1] = {};
          own.fetch(m0 + col, res);
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
          own.rows(m0 + col, s[0], s[1], res);
        }
      }
    }
  }
  if (p.split > 1 && warp >= 4 * C::kGroups) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
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
// What a kernel takes, with and without the gate, for bf16 and e4m3.
struct Variant {
  int rows, x_rows, channels;  // rows of a tile; of x per copy; channels of out per tile
  bool pair, interleaved;
  Kernel kernel[2];  // bf16, e4m3
  int threads;
  int stage_bytes, part_bytes, head_bytes;
  float start, block, join;  // us, see plan_of
};
template <int ROWS, int GATE, bool PAIR>
Variant variant(float start, float block, float join) {
  using C = Cfg<ROWS, GATE, PAIR>;
  return {ROWS, C::kXRows, C::kChannels * (PAIR ? 2 : 1), PAIR, GATE == kInterleaved, {linear_kernel<ROWS, false, GATE, PAIR>, linear_kernel<ROWS, true, GATE, PAIR>},
          C::kThreads, C::kStageBytes, C::kPartBytes, static_cast<int>(sizeof(Head<C>)), start, block, join};
}
constexpr int kPlain = 6, kGatedVariants = 5;
const Variant kVariants[kPlain + kGatedVariants] = {
    variant<16, kNoGate, false>(4.5f, .146f, .6f), variant<32, kNoGate, false>(4.7f, .17f, 1.f),
    variant<64, kNoGate, false>(5.3f, .22f, 1.6f), variant<128, kNoGate, false>(6.f, .246f, 4.f),
    variant<128, kNoGate, true>(6.3f, .195f, 3.f), variant<256, kNoGate, true>(7.2f, .26f, 0.f),
    variant<16, kTwoSums, false>(4.8f, .26f, 1.f), variant<32, kTwoSums, false>(5.f, .28f, 1.5f),
    variant<64, kTwoSums, false>(5.8f, .33f, 2.5f), variant<128, kTwoSums, false>(7.f, .4f, 0.f),
    variant<256, kInterleaved, true>(8.f, .3f, 0.f)};
constexpr int kSmemLimit = 227 * 1024;  // of a CTA

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
    for (const Variant& v : kVariants)
      for (const Kernel k : v.kernel)
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit)) != cudaSuccess) return e;
    int n = 0;
    if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    g_sms[dev] = n;
  }
  *sms = g_sms[dev];
  return cudaSuccess;
}

// What a call runs with: the variant, CTAs (or pairs) that share a tile, ring depth.
struct Plan {
  const Variant* variant;
  int split, stages;
};
int64_t tiles_of(int n, int size) { return (static_cast<int64_t>(n) + size - 1) / size; }
// The variant and split with the least expected time, in us: what a launch takes
// from its start to its first product and from its last to its results, waves of
// tiles at a time per block of k each, the weights from HBM meanwhile, and what joining takes each time a tile is shared by twice as many.  Measured on
// these shapes, with e4m3 (the other choice in brackets): 4 x 4,608 x 2,048 6.2 us in
// two parts (6.8 whole), 64 x 4,096 x 4,096 10.5 in two and 10.2 in four (12.3 whole),
// 64 x 18,432 x 6,144 22.4 whole (31.7 in two); 256 x 2,048 x 2,048 8.4 with pairs and
// tiles of 128 rows (11.5 with 256, 9.0 with 64 rows and one CTA); bf16, 512 x 4,096 x
// 4,096, 18.9 with pairs and 128 rows (23.6 with 256, 21.8 with 128 and one CTA).
Plan plan_of(int M, int width, int blocks, bool gated, double bytes, int sms) {
  Plan best{nullptr, 1, 0};
  double least = 0;
  for (int i = gated ? kPlain : 0; i < (gated ? kPlain + kGatedVariants : kPlain); ++i) {
    const Variant& v = kVariants[i];
    const int most = std::min((kSmemLimit - v.head_bytes) / v.stage_bytes, kMaxStages);
    const int64_t tiles = tiles_of(width, v.channels) * tiles_of(M, v.rows), at_once = v.pair ? sms / 2 : sms;
    for (int split = 1, log2 = 0; split <= kMaxSplit; split *= 2, ++log2) {
      if (split > 1 && (v.interleaved || tiles * split > at_once || split > blocks || 2 * v.part_bytes > most * v.stage_bytes)) break;
      const int64_t waves = (tiles * split + at_once - 1) / at_once;
      // (of the waves' time and the weights' the shorter hides behind the longer but for some three tenths)
      const double compute = static_cast<double>(waves) * tiles_of(blocks, split) * v.block, memory = bytes / 6.5e6;
      const double us = v.start + std::max(compute, memory) + .3 * std::min(compute, memory) + log2 * v.join;
      if (best.variant && us >= least) continue;
      // no more stages than there is to copy, but room for the sums of a tile in parts
      const int64_t copies = waves * tiles_of(blocks, split), sums = split > 1 ? tiles_of(2 * v.part_bytes, v.stage_bytes) : 1;
      best = {&v, split, static_cast<int>(std::min<int64_t>(most, std::max(copies, sums)))};
      least = us;
    }
  }
  return best;
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
  if (a->M < 0 || a->N < 1 || a->N > kMost || a->K < 1 || a->K > kMost || a->activation < 0 ||
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
  const Plan plan = plan_of(a->M, width, blocks, gated, static_cast<double>(k_bytes) * a->N, sms);
  const Variant& v = *plan.variant;
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
    const cuuint32_t box[2] = {kBlock, static_cast<cuuint32_t>(v.x_rows)};
    r = g_encode(&x_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(a->x), dims, strides, box, ones,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (r != CUDA_SUCCESS) return kda_internal_fail(KDA_ERR_LAUNCH, "tensor map: error %d", static_cast<int>(r));
  Params p{};
  p.M = a->M, p.N = a->N, p.K = a->K, p.width = width;
  const int64_t m_tiles = tiles_of(a->M, v.rows), n_tiles = tiles_of(width, v.channels);
  if (m_tiles * n_tiles > 0x7fffffff / 16) return kda_internal_fail(KDA_ERR_SHAPE, "M=%d N=%d: too many tiles", a->M, a->N);
  p.m_tiles = static_cast<int>(m_tiles), p.n_tiles = static_cast<int>(n_tiles), p.blocks = blocks;
  p.split = plan.split, p.stages = plan.stages;
  p.act = a->activation, p.out_f32 = f32, p.early = a->flags & KDA_LINEAR_EARLY_WEIGHT;
  p.x_scale = a->x_scale, p.w_scale = a->weight_scale, p.bias = a->bias;
  p.residual = a->residual, p.res_stride = a->residual_row_stride, p.out = a->out, p.out_stride = a->out_row_stride;
  p.err = a->err_flag;
  p.vec_out = !f32 && !misaligned(a->out, 15) && a->out_row_stride % 8 == 0;
  p.vec_res = !misaligned(a->residual, 15) && a->residual_row_stride % 8 == 0;
  const int cluster = plan.split * (v.pair ? 2 : 1);
  const int64_t clusters = plan.split > 1 ? m_tiles * n_tiles : std::min<int64_t>(m_tiles * n_tiles, sms / cluster);
  e = kda_internal_launch_cluster(v.kernel[e4m3], dim3(static_cast<unsigned>(clusters * cluster)), dim3(static_cast<unsigned>(v.threads)),
                                  static_cast<size_t>(v.head_bytes + plan.stages * v.stage_bytes), stream,
                                  static_cast<unsigned>(cluster), p, w_map, x_map);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
  return KDA_OK;
}
