// kda_linear.cu -- matrix products with scales, bias, activation and residual
// in the epilogue (definition in include/kda_linear.h).
//
// Products are formed transposed, Y^T [channel][row] = W [channel][k] X^T: 128
// channels are the wide side of a tile and the rows of x, of which a decode
// step has few, the narrow one (16 to 256 columns).  Tiles of W and X go to
// shared memory by TMA (128 bytes of k, 128-byte swizzle), tcgen05 multiplies
// them as they are, and a thread of the epilogue has a channel of its own, with
// its scale and bias in registers.
//
// A gated tile holds 64 channels of each half, 16 and 16 in turn, so that a
// warp's 32 lanes have both halves of 16 results.
//
// Few tiles: the CTAs of a cluster share one tile, each with a range of k, and
// add their parts up over distributed shared memory in a fixed order.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "kda_internal.h"
#include "kda_linear.h"
#include "kda_tc.cuh"

namespace {

constexpr int kTileN = 128;                // channels of a tile
constexpr int kBlock = 128;                // bytes of k per stage
constexpr int kMaxSplit = 8;
constexpr int kPitch = 80;                 // bytes between rows of results in shared memory

struct Params {
  int M, N, K, width;          // width: channels of out
  int m_tiles, tiles, blocks;  // row tiles, tiles, blocks of k
  int act;
  bool out_f32, early, vec_out, vec_res;  // vec: rows in 16-byte pieces
  const float *x_scale, *w_scale, *bias;
  const uint16_t* residual;
  int64_t res_stride;
  void* out;
  int64_t out_stride;
  int32_t* err;
};

// ROWS of x per tile.
template <int ROWS>
struct Cfg {
  static constexpr int kStageBytes = (kTileN + ROWS) * kBlock;
  static constexpr int kStages = 200 * 1024 / kStageBytes;
  static constexpr int kTmemCols = 2 * ROWS;  // two accumulators; a power of two from 32 on
  // A warpgroup of the epilogue per 32 rows, up to two; then producer and issuer.
  static constexpr int kGroups = ROWS > 32 ? 2 : 1, kThreads = 128 * kGroups + 64;
};

template <class C>
struct alignas(1024) Smem {
  uint8_t stage[C::kStages][C::kStageBytes];
  alignas(16) uint8_t rows[4 * C::kGroups][32 * kPitch];  // of the warps of the epilogue
  uint64_t full[C::kStages], empty[C::kStages], acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int failed;
};

__device__ __forceinline__ float sigmoid_times(float y) { return y / (1.f + __expf(-y)); }
// (1 + erf loses gelu's lower tail)
__device__ __forceinline__ float gelu(float y) { return 0.5f * y * erfcf(y * -0.70710678118654752f); }
__device__ __forceinline__ float activate(float y, int act) {
  return act == KDA_ACT_SILU ? sigmoid_times(y) : act == KDA_ACT_GELU ? gelu(y) : y;
}
__device__ __forceinline__ float of_bf16(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---- A warp's part of a tile: 32 accumulator lanes, which are 32 channels of
// out, or gated 16 of them (their two halves 16 lanes apart), as fragments: a
// thread has lanes r8 + 8 j and pairs of neighbouring rows.  Rows of 32 channels
// of bf16 results go through shared memory, 80 bytes apart so that the eight
// rows of a matrix lie in different banks, and from there to memory 16 bytes a
// thread; residuals come the same way.
template <bool GATED>
struct Epilogue {
  static constexpr int kWidth = GATED ? 16 : 32;  // channels of out
  static constexpr int kParts = kWidth / 8;       // 16-byte pieces of a row
  const Params& p;
  uint8_t* stage;                                 // 32 rows of the warp's own
  int lane, n0;
  float scale[4], bias[4];

  __device__ __forceinline__ Epilogue(const Params& q, uint8_t* st, int n_tile, int wq, int ln)
      : p(q), stage(st), lane(ln), n0(n_tile * (GATED ? kTileN / 2 : kTileN) + wq * kWidth) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = n0 + (lane >> 2) + 8 * (GATED ? j & 1 : j), n = GATED ? c + (j >> 1) * p.width : c;
      const bool live = c < p.width;
      scale[j] = live && p.w_scale ? p.w_scale[n] : 1.f;
      bias[j] = live && p.bias ? p.bias[n] : 0.f;
    }
  }
  // this thread's row of the matrices of 8-row block b (gated: of b and b + 1)
  __device__ __forceinline__ uint32_t matrix(int b) const {
    const int m = lane >> 3;
    return s32(stage) + (8 * (GATED ? b + (m >> 1) : b) + (lane & 7)) * kPitch + (GATED ? m & 1 : m) * 16;
  }
  // Rows m0 .. m0 + 8 BLOCKS - 1 between memory and the stage.
  template <int BLOCKS>
  __device__ __forceinline__ void fetch(int m0) {
    const bool vec = p.vec_res && n0 + kWidth <= p.width;
    if (vec) {
      constexpr int kRows = 32 / kParts, kTrips = 8 * BLOCKS / kRows;  // rows per trip
      uint4 v[kTrips];
#pragma unroll
      for (int i = 0; i < kTrips; ++i) {
        const int m = m0 + i * kRows + lane / kParts;
        v[i] = m < p.M ? *reinterpret_cast<const uint4*>(p.residual + m * p.res_stride + n0 + lane % kParts * 8) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kTrips; ++i)
        *reinterpret_cast<uint4*>(stage + (i * kRows + lane / kParts) * kPitch + lane % kParts * 16) = v[i];
    } else {
      constexpr int kRows = 32 / kWidth, kTrips = 8 * BLOCKS / kRows;
      const int c = n0 + lane % kWidth;
      uint16_t v[kTrips];
#pragma unroll
      for (int i = 0; i < kTrips; ++i) {
        const int m = m0 + i * kRows + lane / kWidth;
        v[i] = m < p.M && c < p.width ? p.residual[m * p.res_stride + c] : 0;
      }
#pragma unroll
      for (int i = 0; i < kTrips; ++i)
        *reinterpret_cast<uint16_t*>(stage + (i * kRows + lane / kWidth) * kPitch + lane % kWidth * 2) = v[i];
    }
    __syncwarp();
  }
  template <int BLOCKS>
  __device__ __forceinline__ void put(int m0) {
    __syncwarp();
    uint16_t* out = static_cast<uint16_t*>(p.out);
    if (p.vec_out && n0 + kWidth <= p.width) {
      constexpr int kRows = 32 / kParts, kTrips = 8 * BLOCKS / kRows;
#pragma unroll
      for (int i = 0; i < kTrips; ++i) {
        const int m = m0 + i * kRows + lane / kParts;
        const uint4 v = *reinterpret_cast<const uint4*>(stage + (i * kRows + lane / kParts) * kPitch + lane % kParts * 16);
        if (m < p.M) *reinterpret_cast<uint4*>(out + m * p.out_stride + n0 + lane % kParts * 8) = v;
      }
    } else {
      constexpr int kRows = 32 / kWidth, kTrips = 8 * BLOCKS / kRows;
      const int c = n0 + lane % kWidth;
#pragma unroll
      for (int i = 0; i < kTrips; ++i) {
        const int m = m0 + i * kRows + lane / kWidth;
        const uint16_t v = *reinterpret_cast<const uint16_t*>(stage + (i * kRows + lane / kWidth) * kPitch + lane % kWidth * 2);
        if (m < p.M && c < p.width) out[m * p.out_stride + c] = v;
      }
    }
    __syncwarp();
  }
  // Rows m0 .. m0 + 8 BLOCKS - 1 from their sums.
  template <int BLOCKS>
  __device__ __forceinline__ void rows(int m0, float (&z)[4][2 * BLOCKS]) {
    if (n0 >= p.width) return;
    if (p.residual) fetch<BLOCKS>(m0);
    const int a = 2 * (lane & 3);
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
      const int m = m0 + 8 * b + a;
      const float s0 = p.x_scale && m < p.M ? p.x_scale[m] : 1.f, s1 = p.x_scale && m + 1 < p.M ? p.x_scale[m + 1] : 1.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z[j][2 * b] = fmaf(z[j][2 * b] * s0, scale[j], bias[j]);
        z[j][2 * b + 1] = fmaf(z[j][2 * b + 1] * s1, scale[j], bias[j]);
      }
    }
    if (GATED) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2 * BLOCKS; ++i) z[j][i] = sigmoid_times(z[j][i]) * z[j + 2][i];
    } else if (p.act == KDA_ACT_SILU) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2 * BLOCKS; ++i) z[j][i] = sigmoid_times(z[j][i]);
    } else if (p.act == KDA_ACT_GELU) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2 * BLOCKS; ++i) z[j][i] = gelu(z[j][i]);
    }
    if (p.residual) {
#pragma unroll
      for (int b = 0; b < BLOCKS; b += GATED ? 2 : 1) {
        uint32_t r[4];
        load_transposed(matrix(b), r);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = GATED ? k & 1 : k, i = 2 * (GATED ? b + (k >> 1) : b);
          z[j][i] += of_bf16(r[k] & 0xffffu);
          z[j][i + 1] += of_bf16(r[k] >> 16);
        }
      }
      __syncwarp();
    }
    if (p.out_f32) {  // eight neighbouring channels of four rows at a time: whole sectors
      float* out = static_cast<float*>(p.out);
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int m = m0 + 8 * b + a + e;
#pragma unroll
          for (int j = 0; j < (GATED ? 2 : 4); ++j) {
            const int c = n0 + (lane >> 2) + 8 * j;
            if (m < p.M && c < p.width) out[m * p.out_stride + c] = z[j][2 * b + e];
          }
        }
    } else {
#pragma unroll
      for (int b = 0; b < BLOCKS; b += GATED ? 2 : 1) {
        uint32_t r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = GATED ? k & 1 : k, i = 2 * (GATED ? b + (k >> 1) : b);
          r[k] = pack_bf16(z[j][i], z[j][i + 1]);
        }
        store_transposed(matrix(b), r);
      }
      put<BLOCKS>(m0);
    }
  }
};

// A tile shared by the CTAs of a cluster: this CTA's share of the rows, from all
// their sums.  A thread has one accumulator lane and pairs of rows.
template <int ROWS, bool GATED>
__device__ __forceinline__ void join_parts(const Params& p, uint8_t* raw, int tile, int rank, int split) {
  const int tid = threadIdx.x & 127, group = threadIdx.x >> 7, lane = tid & 31, warp = tid >> 5;
  const int nt = tile / p.m_tiles, m0 = (tile - nt * p.m_tiles) * ROWS;
  const int c = GATED ? nt * (kTileN / 2) + 16 * warp + (lane & 15) : nt * kTileN + tid;  // of out
  const int n = GATED ? c + (lane >> 4) * p.width : c;
  const bool live = c < p.width;
  const float scale = live && p.w_scale ? p.w_scale[n] : 1.f, bias = live && p.bias ? p.bias[n] : 0.f;
  constexpr int kAhead = 4;  // pairs of rows whose parts are on their way together
  const int pairs = ROWS / 2 / split, end = min((rank + 1) * pairs, (p.M - m0 + 1) / 2);
  for (int q0 = rank * pairs + kAhead * group; q0 < end; q0 += kAhead * Cfg<ROWS>::kGroups) {
    float2 a[kAhead];
    float res[kAhead][2], xs[kAhead][2];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      a[k] = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int m = m0 + 2 * (q0 + k) + e;
        const bool there = q0 + k < end && m < p.M;
        xs[k][e] = p.x_scale && there ? p.x_scale[m] : 1.f;
        // (gated: lanes 0 .. 15 finish the even row, 16 .. 31 the odd one)
        res[k][e] = p.residual && there && live && (!GATED || e == lane >> 4) ? of_bf16(p.residual[m * p.res_stride + c]) : 0.f;
      }
    }
#pragma unroll
    for (int r = 0; r < kMaxSplit; ++r) {
      if (r < split) {
        uint32_t from;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(s32(raw) + 8 * tid), "r"(r));
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          float2 v;
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(from + min(q0 + k, end - 1) * (8 * kTileN)) : "memory");
          a[k].x += v.x, a[k].y += v.y;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (q0 + k >= end) break;
      float y[2] = {fmaf(a[k].x * xs[k][0], scale, bias), fmaf(a[k].y * xs[k][1], scale, bias)};
      const bool up = GATED && lane >> 4;
      if (GATED) {
        const float got = __shfl_xor_sync(0xffffffffu, up ? y[0] : y[1], 16);
        if (up) y[1] = sigmoid_times(got) * y[1];
        else y[0] = sigmoid_times(y[0]) * got;
      } else {
        y[0] = activate(y[0], p.act), y[1] = activate(y[1], p.act);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t m = m0 + 2 * (q0 + k) + e;
        if (m >= p.M || !live || (GATED && up != (e == 1))) continue;
        const float v = y[e] + res[k][e];
        if (p.out_f32) static_cast<float*>(p.out)[m * p.out_stride + c] = v;
        else static_cast<__nv_bfloat16*>(p.out)[m * p.out_stride + c] = __float2bfloat16_rn(v);
      }
    }
  }
}

template <int ROWS, bool E4M3, bool GATED>
__global__ void __launch_bounds__(Cfg<ROWS>::kThreads, 1)
    linear_kernel(const Params p, const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map, int split) {
  using C = Cfg<ROWS>;
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem<C>& S = *reinterpret_cast<Smem<C>*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int first = blockIdx.x / split, rank = blockIdx.x - first * split, step = gridDim.x / split;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) bar_init(&S.full[i], 1), bar_init(&S.empty[i], 1);
    for (int i = 0; i < 2; ++i) bar_init(&S.acc_full[i], 1), bar_init(&S.acc_empty[i], 128 * C::kGroups);
    bar_init(&S.done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    S.failed = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&w_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&x_map) : "memory");
  }
  __syncwarp();
  if (warp == 4 * C::kGroups + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s32(&S.tmem)), "n"(C::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_before();
  __syncthreads();
  tc_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = S.tmem;
  const int k0 = static_cast<int>(static_cast<int64_t>(p.blocks) * rank / split);
  const int k1 = static_cast<int>(static_cast<int64_t>(p.blocks) * (rank + 1) / split), span = k1 - k0;
  const int mine = first < p.tiles ? (p.tiles - first + step - 1) / step : 0;  // tiles of this CTA
  if (warp == 4 * C::kGroups) {
    // ================================================================ producer
    if (lane == 0) {
      const int64_t total = static_cast<int64_t>(mine) * span;
      auto weights = [&](uint32_t st, int tile, int k) {
        const int nt = tile / p.m_tiles;
        const uint32_t dst = s32(S.stage[st]);
        if (GATED) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            tma_3d(dst + i * 32 * kBlock, &w_map, k * kBlock, nt * (kTileN / 2) + 16 * i, 0, &S.full[st]);
        } else {
          tma_2d(dst, &w_map, k * kBlock, nt * kTileN, &S.full[st]);
        }
      };
      auto rows = [&](uint32_t st, int tile, int k) {
        tma_2d(s32(S.stage[st]) + kTileN * kBlock, &x_map, k * kBlock, (tile % p.m_tiles) * ROWS, &S.full[st]);
      };
      int64_t ahead = 0;  // stages whose weights were asked for before the kernel ahead ended
      if (p.early) {
        int tile = first, k = k0;
        for (; ahead < total && ahead < C::kStages; ++ahead) {
          bar_expect(&S.full[ahead], C::kStageBytes);
          weights(static_cast<uint32_t>(ahead), tile, k);
          if (++k == k1) k = k0, tile += step;
        }
      }
      asm volatile("griddepcontrol.wait;" ::: "memory");
      int tile = first, k = k0;
      int64_t it = 0;
      for (; it < total; ++it) {
        const uint32_t st = static_cast<uint32_t>(it % C::kStages), round = static_cast<uint32_t>(it / C::kStages);
        if (it >= ahead) {
          if (round > 0 && !bar_wait(&S.empty[st], (round - 1) & 1, &S.failed)) break;
          bar_expect(&S.full[st], C::kStageBytes);
          weights(st, tile, k);
        }
        rows(st, tile, k);
        if (++k == k1) k = k0, tile += step;
      }
      // nothing may land in shared memory after the CTA is gone, whoever gave up
      for (int64_t j = it > C::kStages ? it - C::kStages : 0; j < it; ++j)
        bar_drain(&S.full[j % C::kStages], static_cast<uint32_t>(j / C::kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 4 * C::kGroups + 1) {
    // ========================================================== product issuer
    if (lane == 0) {
      constexpr uint32_t id = idesc_k(E4M3, kTileN, ROWS);
      bool ok = true;
      int64_t it = 0;
      for (int i = 0; i < mine && ok; ++i) {
        const uint32_t buf = i & 1;
        if (i >= 2) ok = bar_wait(&S.acc_empty[buf], ((i >> 1) - 1) & 1, &S.failed);
        tc_after();
        for (int k = 0; k < span && ok; ++k, ++it) {
          const uint32_t st = static_cast<uint32_t>(it % C::kStages);
          ok = bar_wait(&S.full[st], static_cast<uint32_t>(it / C::kStages) & 1, &S.failed);
          if (!ok) break;
          tc_after();
          const uint32_t w = s32(S.stage[st]), x = w + kTileN * kBlock;
#pragma unroll
          for (int j = 0; j < kBlock / 32; ++j)
            mma_1cta<E4M3>(tmem + buf * ROWS, sdesc128(w + 32 * j), sdesc128(x + 32 * j), id, k + j > 0);
          commit(&S.empty[st]);
        }
        if (ok) commit(&S.acc_full[buf]);
      }
      commit(&S.done);
    }
    __syncwarp();
  } else {
    // ================================================================ epilogue
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int wq = warp & 3, group = warp >> 2;  // the warp's quarter of the lanes; its group, which takes every kGroups-th 32 rows
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * wq) << 16);
    for (int i = 0; i < mine; ++i) {
      const uint32_t buf = i & 1;
      const int tile = first + i * step, nt = tile / p.m_tiles, m0 = (tile - nt * p.m_tiles) * ROWS;
      constexpr int kBlocks = ROWS < 32 ? 2 : 4;
      Epilogue<GATED> e(p, S.rows[warp], nt, wq, lane);
      bar_wait(&S.acc_full[buf], (i >> 1) & 1, &S.failed);
      tc_after();
#pragma unroll 1
      for (int col = 8 * kBlocks * group; col < ROWS && m0 + col < p.M; col += 8 * kBlocks * C::kGroups) {
        float z[4][2 * kBlocks];
        tm_fragments<kBlocks>(lanes + buf * ROWS + col, z);
        if (split > 1) {  // [column pair][channel], where the stages were
          float2* part = reinterpret_cast<float2*>(raw) + (col / 2 + (lane & 3)) * kTileN + 32 * wq + (lane >> 2);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[4 * b * kTileN + 8 * j] = make_float2(z[j][2 * b], z[j][2 * b + 1]);
        } else {
          e.template rows<kBlocks>(m0 + col, z);
        }
      }
      tc_before();
      bar_arrive(&S.acc_empty[buf]);
    }
  }
  if (split > 1) {
    // ---- the parts of the cluster's CTAs: each adds up its share of the columns
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (warp < 4 * C::kGroups && mine > 0) {
      join_parts<ROWS, GATED>(p, raw, first, rank, split);
    }
    __syncwarp();
    cluster_arrive();  // nobody reads this CTA's memory any more
    cluster_wait();
  }
  // every product has ended before the accumulators are given back, given up or not
  if (warp == 4 * C::kGroups + 1 && !bar_wait(&S.done, 0, &S.failed)) bar_drain(&S.done, 0);
  tc_before();
  __syncthreads();
  if (tid == 0 && S.failed && p.err) atomicOr(p.err, KDA_DEVERR_TIMEOUT);
  __syncwarp();
  if (warp == 4 * C::kGroups + 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kTmemCols));
}

// ------------------------------------------------------- the kernel, many rows
// 256 rows of x and 256 channels: a pair of CTAs forms one product, each with
// 128 channels of the weights and half of the rows in its shared memory, so that
// a tile's operands are read once per pair.  An accumulator's 256 columns are in
// both CTAs' tensor memory, each with its own channels, twice: a tile's results
// are written while the next one's products run.
template <int ROWS>
struct PairCfg {
  static constexpr int kStageBytes = (kTileN + ROWS / 2) * kBlock;
  static constexpr int kStages = 200 * 1024 / kStageBytes;
  static constexpr int kTmemCols = 2 * ROWS;
  static constexpr int kGroups = 2, kThreads = 128 * kGroups + 64;
};
// Tiles go through the channels for a group of row tiles at a time, so that what
// runs at once shares both operands in L2.
constexpr int kGroup = 10;
struct TileAt {
  int nt, mt;
  __device__ __forceinline__ TileAt(const Params& p, int tile) {
    const int groups = (p.m_tiles + kGroup - 1) / kGroup, size = (p.m_tiles + groups - 1) / groups;
    const int n_tiles = p.tiles / p.m_tiles, g = tile / (size * n_tiles), first = g * size;
    const int here = min(size, p.m_tiles - first), r = tile - first * n_tiles;
    nt = r / here;
    mt = first + r - nt * here;
  }
};

template <int ROWS, bool E4M3, bool GATED>
__global__ void __launch_bounds__(PairCfg<ROWS>::kThreads, 1)
    linear_pair_kernel(const Params p, const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map, int) {
  using C = PairCfg<ROWS>;
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem<C>& S = *reinterpret_cast<Smem<C>*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x & 1, first = blockIdx.x >> 1, step = gridDim.x >> 1;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) bar_init(&S.full[i], 1), bar_init(&S.empty[i], 1);
    for (int i = 0; i < 2; ++i) bar_init(&S.acc_full[i], 1), bar_init(&S.acc_empty[i], 8 * C::kGroups);  // the warps of both epilogues
    bar_init(&S.done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    S.failed = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&w_map) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&x_map) : "memory");
  }
  __syncwarp();
  if (warp == 4 * C::kGroups + 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s32(&S.tmem)), "n"(C::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_before();
  __syncthreads();
  cluster_arrive();  // the other CTA's barriers are there
  cluster_wait();
  tc_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = S.tmem;
  const int mine = first < p.tiles ? (p.tiles - first + step - 1) / step : 0;
  if (warp == 4 * C::kGroups) {
    // ================================================================ producer
    if (lane == 0) {
      const int64_t total = static_cast<int64_t>(mine) * p.blocks;
      auto expect = [&](uint32_t st) {  // both CTAs' copies count at the even one
        if (rank == 0) bar_expect(&S.full[st], 2 * C::kStageBytes);
      };
      auto weights = [&](uint32_t st, int nt, int k) {
        const uint32_t dst = s32(S.stage[st]), b = in_cta(&S.full[st], 0);
        if (GATED) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            tma_3d_pair(dst + i * 32 * kBlock, &w_map, k * kBlock, (2 * nt + rank) * (kTileN / 2) + 16 * i, 0, b);
        } else {
          tma_2d_pair(dst, &w_map, k * kBlock, (2 * nt + rank) * kTileN, b);
        }
      };
      auto rows = [&](uint32_t st, int mt, int k) {
        tma_2d_pair(s32(S.stage[st]) + kTileN * kBlock, &x_map, k * kBlock, mt * ROWS + rank * (ROWS / 2), in_cta(&S.full[st], 0));
      };
      int64_t ahead = 0;  // stages whose weights were asked for before the kernel ahead ended
      if (p.early) {
        int tile = first, k = 0;
        for (; ahead < total && ahead < C::kStages; ++ahead) {
          expect(static_cast<uint32_t>(ahead));
          weights(static_cast<uint32_t>(ahead), TileAt(p, tile).nt, k);
          if (++k == p.blocks) k = 0, tile += step;
        }
      }
      asm volatile("griddepcontrol.wait;" ::: "memory");
      int64_t it = 0;
      bool ok = true;
      for (int i = 0; i < mine && ok; ++i) {
        const TileAt at(p, first + i * step);
        for (int k = 0; k < p.blocks; ++k, ++it) {
          const uint32_t st = static_cast<uint32_t>(it % C::kStages), round = static_cast<uint32_t>(it / C::kStages);
          if (it >= ahead) {
            if (round > 0 && !bar_wait(&S.empty[st], (round - 1) & 1, &S.failed)) {
              ok = false;
              break;
            }
            expect(st);
            weights(st, at.nt, k);
          }
          rows(st, at.mt, k);
        }
      }
      // nothing may land in either CTA's memory after it is gone, whoever gave up
      if (rank == 0)
        for (int64_t j = it > C::kStages ? it - C::kStages : 0; j < it; ++j)
          bar_drain(&S.full[j % C::kStages], static_cast<uint32_t>(j / C::kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 4 * C::kGroups + 1) {
    // ========================================================== product issuer
    if (lane == 0 && rank == 0) {
      constexpr uint32_t id = idesc_k(E4M3, 2 * kTileN, ROWS);
      bool ok = true;
      int64_t it = 0;
      for (int i = 0; i < mine && ok; ++i) {
        const uint32_t buf = i & 1;
        if (i >= 2) ok = bar_wait(&S.acc_empty[buf], ((i >> 1) - 1) & 1, &S.failed);
        tc_after();
        for (int k = 0; k < p.blocks && ok; ++k, ++it) {
          const uint32_t st = static_cast<uint32_t>(it % C::kStages);
          ok = bar_wait(&S.full[st], static_cast<uint32_t>(it / C::kStages) & 1, &S.failed);
          if (!ok) break;
          tc_after();
          const uint32_t w = s32(S.stage[st]), x = w + kTileN * kBlock;
#pragma unroll
          for (int j = 0; j < kBlock / 32; ++j)
            mma_2cta<E4M3>(tmem + buf * ROWS, sdesc128(w + 32 * j), sdesc128(x + 32 * j), id, k + j > 0);
          commit_both(&S.empty[st]);
        }
        if (ok) commit_both(&S.acc_full[buf]);
      }
      commit_both(&S.done);
    }
    __syncwarp();
  } else {
    // ================================================================ epilogue
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int wq = warp & 3, group = warp >> 2;  // the warp's quarter of the lanes; its group, which takes every kGroups-th 32 rows
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * wq) << 16);
    for (int i = 0; i < mine; ++i) {
      const uint32_t buf = i & 1;
      const TileAt at(p, first + i * step);
      const int m0 = at.mt * ROWS;
      Epilogue<GATED> e(p, S.rows[warp], 2 * at.nt + rank, wq, lane);
      bar_wait(&S.acc_full[buf], (i >> 1) & 1, &S.failed);
      tc_after();
#pragma unroll 1
      for (int col = 32 * group; col < ROWS && m0 + col < p.M; col += 32 * C::kGroups) {
        float z[4][8];
        tm_fragments<4>(lanes + buf * ROWS + col, z);
        e.template rows<4>(m0 + col, z);
      }
      tc_before();
      __syncwarp();
      if (lane == 0) bar_arrive_at(in_cta(&S.acc_empty[buf], 0));
    }
  }
  // every product has ended, in both CTAs' memory, before either leaves, given up or not
  if (warp == 4 * C::kGroups + 1 && !bar_wait(&S.done, 0, &S.failed)) bar_drain(&S.done, 0);
  tc_before();
  __syncthreads();
  if (tid == 0 && S.failed && p.err) atomicOr(p.err, KDA_DEVERR_TIMEOUT);
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  if (warp == 4 * C::kGroups + 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kTmemCols));
}

// ------------------------------------------------------------------ host side
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::mutex g_mutex;
int g_sms[64];
EncodeFn g_encode;

using Kernel = void (*)(const Params, const CUtensorMap, const CUtensorMap, int);
struct Variant {
  int rows, box;     // rows of a tile; rows of x per copy
  bool pair;
  Kernel kernel[4];  // bf16, e4m3, and both gated
  size_t smem;
  int threads;
};
template <int ROWS>
Variant single() {
  using M = Smem<Cfg<ROWS>>;
  static_assert(sizeof(M) <= 227 * 1024 && ROWS * kTileN * 4 <= sizeof(M::stage), "shared memory");
  return {ROWS, ROWS, false, {linear_kernel<ROWS, false, false>, linear_kernel<ROWS, true, false>, linear_kernel<ROWS, false, true>, linear_kernel<ROWS, true, true>}, sizeof(M), Cfg<ROWS>::kThreads};
}
template <int ROWS>
Variant pair() {
  using M = Smem<PairCfg<ROWS>>;
  static_assert(sizeof(M) <= 227 * 1024, "shared memory");
  return {ROWS, ROWS / 2, true, {linear_pair_kernel<ROWS, false, false>, linear_pair_kernel<ROWS, true, false>, linear_pair_kernel<ROWS, false, true>, linear_pair_kernel<ROWS, true, true>}, sizeof(M), PairCfg<ROWS>::kThreads};
}
const Variant kVariants[] = {single<16>(), single<32>(), single<64>(), single<128>(), pair<256>()};
const Variant& variant_of(int M) { return kVariants[M <= 16 ? 0 : M <= 32 ? 1 : M <= 64 ? 2 : M <= 128 ? 3 : 4]; }

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
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(v.smem))) != cudaSuccess) return e;
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
  const Variant& v = variant_of(a->M);
  CUtensorMap w_map, x_map;
  CUresult r;
  {
    // gated: the two halves are a dimension of their own, a copy takes 16 rows of each
    const cuuint64_t dims[3] = {k_bytes, static_cast<cuuint64_t>(width), 2};
    const cuuint64_t strides[2] = {w_pitch, w_pitch * static_cast<cuuint64_t>(width)};
    const cuuint32_t box[3] = {kBlock, static_cast<cuuint32_t>(gated ? 16 : kTileN), 2};
    r = g_encode(&w_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, gated ? 3 : 2, const_cast<void*>(a->weight), dims, strides, box, ones,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (r == CUDA_SUCCESS) {
    const cuuint64_t dims[2] = {k_bytes, static_cast<cuuint64_t>(a->M)};
    const cuuint64_t strides[1] = {x_pitch};
    const cuuint32_t box[2] = {kBlock, static_cast<cuuint32_t>(v.box)};
    r = g_encode(&x_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(a->x), dims, strides, box, ones,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (r != CUDA_SUCCESS) return kda_internal_fail(KDA_ERR_LAUNCH, "tensor map: error %d", static_cast<int>(r));
  Params p{};
  p.M = a->M, p.N = a->N, p.K = a->K, p.width = width;
  const int tile_width = (gated ? kTileN / 2 : kTileN) * (v.pair ? 2 : 1);
  const int64_t m_tiles = (static_cast<int64_t>(a->M) + v.rows - 1) / v.rows, n_tiles = (static_cast<int64_t>(width) + tile_width - 1) / tile_width;
  if (m_tiles * n_tiles > 0x7fffffff / kMaxSplit) return kda_internal_fail(KDA_ERR_SHAPE, "M=%d N=%d: too many tiles", a->M, a->N);
  p.m_tiles = static_cast<int>(m_tiles), p.tiles = static_cast<int>(m_tiles * n_tiles);
  p.blocks = static_cast<int>((k_bytes + kBlock - 1) / kBlock);
  p.act = a->activation, p.out_f32 = f32, p.early = a->flags & KDA_LINEAR_EARLY_WEIGHT;
  p.x_scale = a->x_scale, p.w_scale = a->weight_scale, p.bias = a->bias;
  p.residual = a->residual, p.res_stride = a->residual_row_stride, p.out = a->out, p.out_stride = a->out_row_stride;
  p.err = a->err_flag;
  p.vec_out = !f32 && !misaligned(a->out, 15) && a->out_row_stride % 8 == 0;
  p.vec_res = !misaligned(a->residual, 15) && a->residual_row_stride % 8 == 0;
  // few tiles: up to eight CTAs share one, while all of them are resident and each has a block of k
  int split = 1;
  if (!v.pair)
    while (split < kMaxSplit && static_cast<int64_t>(p.tiles) * split * 2 <= sms && split * 2 <= p.blocks) split *= 2;
  const int cluster = v.pair ? 2 : split, resident = v.pair ? sms / 2 : sms;
  const unsigned grid = static_cast<unsigned>((split > 1 || p.tiles < resident ? p.tiles : resident) * cluster);
  e = kda_internal_launch_cluster(v.kernel[(gated ? 2 : 0) + (e4m3 ? 1 : 0)], dim3(grid), dim3(static_cast<unsigned>(v.threads)), v.smem, stream,
                                  static_cast<unsigned>(cluster), p, w_map, x_map, split);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
  return KDA_OK;
}
