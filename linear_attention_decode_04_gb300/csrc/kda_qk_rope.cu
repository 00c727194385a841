// kda_qk_rope.cu -- per-head norm and rotation of q and k, and the write of
// k and v into the 8-bit paged cache (definition in include/kda_qk_rope.h).
//
// Bound by HBM on prompts (each row read once, each output written once) and
// by latency on decode steps.  One launch holds two kinds of CTAs:
//   - cache CTAs: a run of token rows that fall in one block, for one kv head
//     and one of K / V.  The block's scale needs the largest value of all its
//     new rows, so the run's rows stay in registers between the norm, the
//     reduction and the rounding to e4m3; nothing is read twice.
//   - query CTAs: one warp per token and group of heads; the token's sines
//     and cosines are computed once for the warp's heads.
// Eight lanes share a row of 128 channels, 16 channels each, as two 16-byte
// loads: lane l holds the pairs 8l .. 8l + 7 of whichever pairing is used.
//
// The angle is pos * freq modulo one turn in 64-bit integers (exact for any
// position), of which the upper 32 bits go to sincospif as a fraction of a
// half turn: the error is that of one fp32 rounding.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_qk_rope.h"

namespace {

constexpr int kD = KDA_HEAD_DIM;
constexpr int kExpMin = -64, kExpMax = 119;  // range of the block scales' exponents

struct Params {
  int T, Hq, Hkv, rot, bs, num_blocks, interleaved;
  int cache_ctas, rows_per_cta;  // cache CTAs come first in the grid; rows each looks through
  int q_heads, chunks, iters;    // heads that query CTAs write (q, and k with k_out); warps per token; row groups each
  float eps;
  const uint16_t* qkv;
  int64_t qkv_stride;
  uint16_t *q_out, *k_out;
  int64_t q_stride, k_stride;
  const int32_t* positions;
  const uint64_t* freqs;
  const float *q_weight, *k_weight;
  uint8_t *k_cache, *v_cache;
  int64_t block_stride, head_stride, token_stride;
  float *k_scale, *v_scale;
  const int64_t* slot_map;
  int32_t* err;
};

// 16 channels of a row as eight pairs.
struct Pairs {
  float a[8], b[8];
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Where lane l's two runs of 8 channels start.  Half-split pairing: run 0 holds the
// a's and run 1 the b's; channels behind rot_dim are split in halves the same
// way, so every lane holds either rotated pairs only or none.  Interleaved:
// 16 consecutive channels.
struct Runs {
  int c0, c1;
};
__device__ __forceinline__ Runs lane_runs(const Params& p, int l) {
  if (p.interleaved) return {16 * l, 16 * l + 8};
  const int half = p.rot >> 1, i = 8 * l;
  if (i < half) return {i, i + half};
  return {p.rot + (i - half), p.rot + (64 - half) + (i - half)};
}
// Runs <-> pairs: the interleaved pairing takes neighbours.
__device__ __forceinline__ Pairs to_pairs(const Params& p, const uint4& r0, const uint4& r1) {
  float x[8], y[8];
  unpack8(r0, x);
  unpack8(r1, y);
  Pairs q;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float ia = i < 4 ? x[2 * i & 7] : y[2 * i & 7], ib = i < 4 ? x[(2 * i + 1) & 7] : y[(2 * i + 1) & 7];
    q.a[i] = p.interleaved ? ia : x[i];
    q.b[i] = p.interleaved ? ib : y[i];
  }
  return q;
}
__device__ __forceinline__ void to_runs(const Params& p, const Pairs& q, float (&x)[8], float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float lo = i & 1 ? q.b[i >> 1] : q.a[i >> 1], hi = i & 1 ? q.b[4 + (i >> 1)] : q.a[4 + (i >> 1)];
    x[i] = p.interleaved ? lo : q.a[i];
    y[i] = p.interleaved ? hi : q.b[i];
  }
}
__device__ __forceinline__ Pairs load_weight(const Params& p, const float* w, const Runs& r) {
  float x[8], y[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 u = reinterpret_cast<const float4*>(w + r.c0)[i], v = reinterpret_cast<const float4*>(w + r.c1)[i];
    x[4 * i] = u.x, x[4 * i + 1] = u.y, x[4 * i + 2] = u.z, x[4 * i + 3] = u.w;
    y[4 * i] = v.x, y[4 * i + 1] = v.y, y[4 * i + 2] = v.z, y[4 * i + 3] = v.w;
  }
  Pairs q;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float ia = i < 4 ? x[2 * i & 7] : y[2 * i & 7], ib = i < 4 ? x[(2 * i + 1) & 7] : y[(2 * i + 1) & 7];
    q.a[i] = p.interleaved ? ia : x[i];
    q.b[i] = p.interleaved ? ib : y[i];
  }
  return q;
}
__device__ __forceinline__ float sum8(float v) {  // over the 8 lanes of a row
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ void norm_row(Pairs& x, const Pairs& w, float eps) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(x.a[i], x.a[i], fmaf(x.b[i], x.b[i], s));
  const float r = rsqrtf(sum8(s) * (1.f / kD) + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) x.a[i] = x.a[i] * r * w.a[i], x.b[i] = x.b[i] * r * w.b[i];
}
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ Turn turn_of(const Params& p, int pos, int l) {
  Turn t;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * p.freqs[8 * l + i];
    // the upper half as a signed fraction of half a turn, in [-1, 1)
    const float x = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
    sincospif(x, &t.s[i], &t.c[i]);
  }
  return t;
}
__device__ __forceinline__ void rotate_row(Pairs& x, const Turn& t) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = x.a[i], b = x.b[i];
    x.a[i] = a * t.c[i] - b * t.s[i];
    x.b[i] = b * t.c[i] + a * t.s[i];
  }
}
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x2, x3), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
// four codes times a power of two, rounded back to codes
__device__ __forceinline__ uint32_t rescale4(uint32_t v, float ratio) {
  float x[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = f.x * ratio, x[2 * i + 1] = f.y * ratio;
  }
  return e4m3x4(x[0], x[1], x[2], x[3]);
}
// 2^e, the smallest in range with amax <= 448 * 2^e.  amax = m 2^x with m in
// [1/2, 1) and 448 = 0.875 * 2^9.
__device__ __forceinline__ float fit_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int e = static_cast<int>(b >> 23) - 126 - 9 + ((b & 0x7fffffu) > 0x600000u);
  e = min(max(e, kExpMin), kExpMax);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The rows t .. t + count - 1 fall in block `blk` from row `first` on.
template <int THREADS, int ROWS>
__device__ __forceinline__ void write_block(const Params& p, int t, int count, int blk, int first, int h, bool is_v,
                                            float* red) {
  constexpr int kGroups = THREADS / 8;
  const int tid = threadIdx.x, l = tid & 7, g = tid >> 3;
  const Runs run = lane_runs(p, l);
  const float* weight = is_v ? nullptr : p.k_weight;
  const bool rotated = !is_v && 8 * l < (p.rot >> 1);
  const uint16_t* src = p.qkv + static_cast<int64_t>(t) * p.qkv_stride +
                        static_cast<int64_t>(p.Hq + (is_v ? p.Hkv : 0) + h) * kD;
  float* scale_at = (is_v ? p.v_scale : p.k_scale) + static_cast<int64_t>(blk) * p.Hkv + h;
  uint8_t* dst = (is_v ? p.v_cache : p.k_cache) + blk * p.block_stride + h * p.head_stride;
  const float old = first > 0 ? *scale_at : 0.f;
  Pairs x[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int j = g + r * kGroups;  // row of the run
    uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
    if (j < count) {
      const uint16_t* row = src + static_cast<int64_t>(j) * p.qkv_stride;
      r0 = *reinterpret_cast<const uint4*>(row + run.c0);
      r1 = *reinterpret_cast<const uint4*>(row + run.c1);
    }
    x[r] = to_pairs(p, r0, r1);
  }
  float amax = 0.f;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int j = g + r * kGroups;
    if (r * kGroups < count) {  // whole warps leave together: count is the CTA's
      if (weight) norm_row(x[r], load_weight(p, weight, run), p.eps);
      if (rotated && j < count) rotate_row(x[r], turn_of(p, p.positions[t + j], l));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = fabsf(x[r].a[i]), v = fabsf(x[r].b[i]);
        amax = fmaxf(amax, fmaxf(u <= FLT_MAX ? u : 0.f, v <= FLT_MAX ? v : 0.f));
      }
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((tid & 31) == 0) red[tid >> 5] = amax;
  __syncthreads();  // also: every thread has read the old scale
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) amax = fmaxf(amax, red[w]);
  const float scale = fmaxf(old, fit_scale(amax));
  const float inv = 1.f / scale;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int j = g + r * kGroups;
    if (j >= count) continue;
    float u[8], v[8];
    to_runs(p, x[r], u, v);
    uint8_t* row = dst + (first + j) * p.token_stride;
    *reinterpret_cast<uint2*>(row + run.c0) =
        make_uint2(e4m3x4(u[0] * inv, u[1] * inv, u[2] * inv, u[3] * inv),
                   e4m3x4(u[4] * inv, u[5] * inv, u[6] * inv, u[7] * inv));
    *reinterpret_cast<uint2*>(row + run.c1) =
        make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                   e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
  }
  if (first > 0 && scale != old) {  // the older rows follow the scale
    const float ratio = old * inv;
    for (int j = g; j < first; j += kGroups) {
      uint4* row = reinterpret_cast<uint4*>(dst + j * p.token_stride) + l;
      const uint4 v = *row;
      *row = make_uint4(rescale4(v.x, ratio), rescale4(v.y, ratio), rescale4(v.z, ratio), rescale4(v.w, ratio));
    }
  }
  if (tid == 0) *scale_at = scale;
  __syncthreads();  // red is free again
}

template <int THREADS, int ROWS>
__global__ void __launch_bounds__(THREADS) qk_rope_kernel(const Params p) {
  __shared__ float red[THREADS / 32];
  __shared__ int lead[THREADS];
  __shared__ int leads, extent;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (static_cast<int>(blockIdx.x) < p.cache_ctas) {
    const int per_head = 2 * p.Hkv, unit = blockIdx.x % per_head, h = unit >> 1;
    const int64_t base = static_cast<int64_t>(blockIdx.x / per_head) * p.rows_per_cta;
    const bool is_v = unit & 1;
    const int64_t limit = static_cast<int64_t>(p.num_blocks) * p.bs;
    if (tid == 0) leads = 0;
    __syncthreads();
    // rows that begin a run: the first of a block, or one whose slot does not follow the row before
    if (tid < p.rows_per_cta && base + tid < p.T) {
      const int t = static_cast<int>(base) + tid;
      const int64_t s = p.slot_map[t];
      if (s >= limit && unit == 0 && p.err) atomicOr(p.err, KDA_DEVERR_SLOT_RANGE);
      if (s >= 0 && s < limit && (s % p.bs == 0 || t == 0 || p.slot_map[t - 1] != s - 1)) lead[atomicAdd(&leads, 1)] = t;
    }
    __syncthreads();
    const int n = leads;
    for (int i = 0; i < n; ++i) {
      const int t = lead[i];
      const int64_t s = p.slot_map[t];
      const int blk = static_cast<int>(s / p.bs), first = static_cast<int>(s % p.bs);
      // the run's length: the rows that go on in the same block (a run is at
      // most a block, which is at most THREADS rows)
      const int most = min(p.bs - first, p.T - t);
      if (tid == 0) extent = most;
      __syncthreads();
      if (tid > 0 && tid < most && p.slot_map[t + tid] != s + tid) atomicMin(&extent, tid);
      __syncthreads();
      const int count = extent;
      write_block<THREADS, ROWS>(p, t, count, blk, first, h, is_v, red);
    }
    return;
  }
  // ---- queries (and k_out): warp = (token, chunk of heads), four heads at a time
  const int warp = (blockIdx.x - p.cache_ctas) * (THREADS / 32) + (tid >> 5);
  const int t = warp / p.chunks, chunk = warp - t * p.chunks;
  if (t >= p.T) return;
  const int l = tid & 7, sub = (tid & 31) >> 3;
  const Runs run = lane_runs(p, l);
  const bool rotated = 8 * l < (p.rot >> 1);
  const uint16_t* src = p.qkv + static_cast<int64_t>(t) * p.qkv_stride;
  Turn turn;
  if (rotated) turn = turn_of(p, p.positions[t], l);
  for (int it = 0; it < p.iters; ++it) {
    const int h = (chunk * p.iters + it) * 4 + sub;
    const bool live = h < p.q_heads;
    uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
    if (live) {
      r0 = *reinterpret_cast<const uint4*>(src + h * kD + run.c0);
      r1 = *reinterpret_cast<const uint4*>(src + h * kD + run.c1);
    }
    Pairs x = to_pairs(p, r0, r1);
    const float* weight = h < p.Hq ? p.q_weight : p.k_weight;
    if (p.q_weight || p.k_weight) {
      Pairs y = x;
      norm_row(y, weight ? load_weight(p, weight, run) : y, p.eps);
      if (weight) x = y;
    }
    if (rotated) rotate_row(x, turn);
    if (!live) continue;
    float u[8], v[8];
    to_runs(p, x, u, v);
    uint16_t* out = h < p.Hq ? p.q_out + t * p.q_stride + h * kD : p.k_out + t * p.k_stride + (h - p.Hq) * kD;
    *reinterpret_cast<uint4*>(out + run.c0) = pack8(u);
    *reinterpret_cast<uint4*>(out + run.c1) = pack8(v);
  }
}

// THREADS is at least the block size, ROWS * THREADS / 8 exactly.
template <int THREADS, int ROWS>
cudaError_t launch(Params& p, void* stream) {
  constexpr int kWarps = THREADS / 32;
  int64_t cache_ctas = 0;
  if (p.k_cache) {
    // rows looked through per CTA: one while the rows alone give enough CTAs
    // to fill the card, up to a block's worth on prompts
    const int64_t units = static_cast<int64_t>(p.T) * p.Hkv * 2;
    int64_t rows = units / 8192;
    rows = rows < 1 ? 1 : rows > p.bs ? p.bs : rows;
    if (rows > THREADS) rows = THREADS;
    p.rows_per_cta = static_cast<int>(rows);
    cache_ctas = (p.T + rows - 1) / rows * p.Hkv * 2;
  }
  // warps per token: as many as there are groups of four heads while the
  // batch is small, one per token on prompts (the sines are then computed once)
  const int groups = (p.q_heads + 3) / 4;
  int64_t chunks = (static_cast<int64_t>(152) * 32 + p.T - 1) / p.T;
  chunks = chunks < 1 ? 1 : chunks > groups ? groups : chunks;
  p.iters = static_cast<int>((groups + chunks - 1) / chunks);
  p.chunks = (groups + p.iters - 1) / p.iters;
  const int64_t ctas = cache_ctas + (static_cast<int64_t>(p.T) * p.chunks + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  p.cache_ctas = static_cast<int>(cache_ctas);
  return kda_internal_launch(qk_rope_kernel<THREADS, ROWS>, dim3(static_cast<unsigned>(ctas)), dim3(THREADS), 0,
                             stream, p);
}

bool misaligned(const void* ptr, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(ptr) & mask) != 0; }

}  // namespace

extern "C" int kda_qk_rope(const KdaQkRopeArgs* a, void* stream) {
  kda_internal_clear_error();
  if (!a) return kda_internal_fail(KDA_ERR_NULLPTR, "args is NULL");
  if (a->struct_size != sizeof(KdaQkRopeArgs))
    return kda_internal_fail(KDA_ERR_ABI, "struct_size %u, library expects %zu", a->struct_size, sizeof(KdaQkRopeArgs));
  if (a->head_dim != kD) return kda_internal_fail(KDA_ERR_SHAPE, "head_dim %d (need 128)", a->head_dim);
  if (a->T < 0 || a->num_q_heads < 1 || a->num_kv_heads < 0 || a->num_q_heads > 65536 || a->num_kv_heads > 65536)
    return kda_internal_fail(KDA_ERR_SHAPE, "T=%d num_q_heads=%d num_kv_heads=%d", a->T, a->num_q_heads, a->num_kv_heads);
  if (a->rot_dim < 0 || a->rot_dim > kD || a->rot_dim % 16)
    return kda_internal_fail(KDA_ERR_SHAPE, "rot_dim %d (need a multiple of 16 up to 128)", a->rot_dim);
  if (a->flags & ~KDA_ROPE_INTERLEAVED) return kda_internal_fail(KDA_ERR_FLAGS, "flags 0x%x", a->flags);
  const bool cache = a->k_cache || a->v_cache || a->k_scale || a->v_scale;
  const int bs = a->block_size;
  if (cache && bs != 16 && bs != 32 && bs != 64 && bs != 128 && bs != 256)
    return kda_internal_fail(KDA_ERR_SHAPE, "block_size %d (need 16, 32, 64, 128 or 256)", bs);
  if (cache && (a->num_blocks < 1 || a->num_kv_heads < 1))
    return kda_internal_fail(KDA_ERR_SHAPE, "num_blocks=%d num_kv_heads=%d", a->num_blocks, a->num_kv_heads);
  if (a->T == 0) return KDA_OK;
  if (!a->qkv || !a->q_out || !a->positions || (a->rot_dim > 0 && !a->freqs) ||
      (cache && (!a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale || !a->slot_map)))
    return kda_internal_fail(KDA_ERR_NULLPTR, "a required pointer is NULL");
  const int64_t width = (static_cast<int64_t>(a->num_q_heads) + 2LL * a->num_kv_heads) * kD;
  if (a->qkv_row_stride < width || a->q_row_stride < static_cast<int64_t>(a->num_q_heads) * kD ||
      (a->k_out && a->k_row_stride < static_cast<int64_t>(a->num_kv_heads) * kD))
    return kda_internal_fail(KDA_ERR_SHAPE, "a row stride is smaller than the row");
  if (cache && (a->token_stride < kD || a->head_stride < kD || a->block_stride < kD))
    return kda_internal_fail(KDA_ERR_SHAPE, "a cache stride is smaller than a row");
  if (cache && a->k_out && a->k_out == a->qkv + static_cast<int64_t>(a->num_q_heads) * kD)
    return kda_internal_fail(KDA_ERR_SHAPE, "k_out may not be the k part of qkv when keys are cached");
  if (misaligned(a->qkv, 15) || (a->qkv_row_stride & 7) || misaligned(a->q_out, 15) || (a->q_row_stride & 7) ||
      misaligned(a->k_out, 15) || (a->k_out && (a->k_row_stride & 7)) || misaligned(a->positions, 3) ||
      misaligned(a->freqs, 7) || misaligned(a->q_weight, 15) || misaligned(a->k_weight, 15) ||
      misaligned(a->k_cache, 15) || misaligned(a->v_cache, 15) || misaligned(a->k_scale, 3) ||
      misaligned(a->v_scale, 3) || misaligned(a->slot_map, 7) || misaligned(a->err_flag, 3) ||
      (cache && ((a->block_stride | a->head_stride | a->token_stride) & 15)))
    return kda_internal_fail(KDA_ERR_ALIGN, "a pointer or stride is not aligned as required");
  Params p{};
  p.T = a->T, p.Hq = a->num_q_heads, p.Hkv = a->num_kv_heads, p.rot = a->rot_dim, p.bs = bs;
  p.num_blocks = a->num_blocks, p.interleaved = (a->flags & KDA_ROPE_INTERLEAVED) != 0;
  p.q_heads = a->num_q_heads + (a->k_out ? a->num_kv_heads : 0);
  p.eps = a->eps;
  p.qkv = a->qkv, p.qkv_stride = a->qkv_row_stride;
  p.q_out = a->q_out, p.q_stride = a->q_row_stride, p.k_out = a->k_out, p.k_stride = a->k_row_stride;
  p.positions = a->positions, p.freqs = a->freqs, p.q_weight = a->q_weight, p.k_weight = a->k_weight;
  p.k_cache = cache ? a->k_cache : nullptr, p.v_cache = a->v_cache;
  p.block_stride = a->block_stride, p.head_stride = a->head_stride, p.token_stride = a->token_stride;
  p.k_scale = a->k_scale, p.v_scale = a->v_scale, p.slot_map = a->slot_map, p.err = a->err_flag;
  // a run of up to block_size rows stays in registers: rows per 8-lane group
  cudaError_t e;
  if (!cache || bs == 16) e = launch<128, 1>(p, stream);
  else if (bs == 32) e = launch<128, 2>(p, stream);
  else if (bs == 64) e = launch<128, 4>(p, stream);
  else if (bs == 128) e = launch<256, 4>(p, stream);
  else e = launch<256, 8>(p, stream);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
  return KDA_OK;
}
