// kda_qk_rope.cu -- per-head norm and rotation of q and k, and the write of
// k and v into the 8-bit paged cache (definition in include/kda_qk_rope.h).
//
// Bound by HBM on prompts (each row read once, each output written once) and
// by latency on decode steps.  One launch holds two kinds of CTAs:
//   - cache CTAs: some token rows for K or V of one or more kv heads.  Rows
//     that go on in one block form a run; the block's scale needs the largest
//     value of the whole run, so its rows stay in registers between the norm,
//     the reduction and the rounding to e4m3, and nothing is read twice.  A
//     short run (a decode or multi-token step) is one warp's work, a long one
//     the CTA's, whose heads share the rows' sines and cosines.
//   - query CTAs: one warp per token and group of heads.  The token's sines and
//     cosines are computed once for the warp's heads and multiplied by the
//     norm's weights, so that a row costs six multiply-adds per pair.
// Eight lanes share a row of 128 channels, 16 channels each, as two 16-byte
// loads: lane l holds the pairs 8l .. 8l + 7 of whichever pairing is used.
//
// Measured on a GB300 (a copy runs at 6795 GB/s): 16,384 token rows, 48 q and 8
// kv heads, blocks of 64, 97 us for 500 MB, 74 at a copy's rate; loads wait on
// registers there (80 a thread, 24 warps an SM, DRAM 67% busy).  64 sequences of 4
// tokens 6.8 us, 4 single tokens 3.7 us.  One CTA per block and head, without
// the sharing of sines, took 155, 13 and 5.4.  Without a cache, queries and keys
// written as bf16: 87 us (69 at a copy's rate), and 4.4 and 2.7 us for 256 and 4 rows.
//
// The angle is pos * freq modulo one turn in 64-bit integers (exact for any
// position), of which the upper 32 bits go to sincospif as a fraction of a
// half turn.  Rounding that to fp32 is off by at most 2^-25 of a half turn, and the
// sines are fp32's: a sine or cosine is off by less than 2^-22, where the outputs are
// rounded to 2^-8 (bf16) or 2^-4 (e4m3) of themselves.
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
constexpr int kMaxBlock = 256;               // largest block size
constexpr int kTableRows = 64;               // largest block whose rows' sines the heads of a CTA share (32 KB)

struct Params {
  int T, Hq, Hkv, rot, bs, num_blocks;
  int cache_ctas, rows_per_cta, heads_per_cta;  // cache CTAs come first in the grid; rows and heads of each
  int q_groups, groups;          // groups of four heads that query CTAs write: of q; of q and, with k_out, k
  int chunks, iters;             // warps per token; head groups each
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
template <bool INTER>
__device__ __forceinline__ Runs lane_runs(int rot, int l) {
  if (INTER) return {16 * l, 16 * l + 8};
  const int half = rot >> 1, i = 8 * l;
  if (i < half) return {i, i + half};
  return {rot + (i - half), rot + (64 - half) + (i - half)};
}
// Runs <-> pairs: the interleaved pairing takes neighbours.
template <bool INTER>
__device__ __forceinline__ Pairs to_pairs(const float (&x)[8], const float (&y)[8]) {
  Pairs q;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (INTER) q.a[i] = i < 4 ? x[2 * i & 7] : y[2 * i & 7], q.b[i] = i < 4 ? x[(2 * i + 1) & 7] : y[(2 * i + 1) & 7];
    else q.a[i] = x[i], q.b[i] = y[i];
  }
  return q;
}
template <bool INTER>
__device__ __forceinline__ Pairs to_pairs(const uint4& r0, const uint4& r1) {
  float x[8], y[8];
  unpack8(r0, x);
  unpack8(r1, y);
  return to_pairs<INTER>(x, y);
}
template <bool INTER>
__device__ __forceinline__ void to_runs(const Pairs& q, float (&x)[8], float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (INTER) x[i] = i & 1 ? q.b[i >> 1] : q.a[i >> 1], y[i] = i & 1 ? q.b[4 + (i >> 1)] : q.a[4 + (i >> 1)];
    else x[i] = q.a[i], y[i] = q.b[i];
  }
}
template <bool INTER>
__device__ __forceinline__ Pairs load_weight(const float* w, const Runs& r) {
  float x[8], y[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 u = reinterpret_cast<const float4*>(w + r.c0)[i], v = reinterpret_cast<const float4*>(w + r.c1)[i];
    x[4 * i] = u.x, x[4 * i + 1] = u.y, x[4 * i + 2] = u.z, x[4 * i + 3] = u.w;
    y[4 * i] = v.x, y[4 * i + 1] = v.y, y[4 * i + 2] = v.z, y[4 * i + 3] = v.w;
  }
  return to_pairs<INTER>(x, y);
}
__device__ __forceinline__ float sum8(float v) {  // over the 8 lanes of a row
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float norm_factor(const Pairs& x, float eps) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(x.a[i], x.a[i], fmaf(x.b[i], x.b[i], s));
  return rsqrtf(sum8(s) * (1.f / kD) + eps);
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

// A run: `count` token rows from t on, in block `blk` from its row `first` on.
struct Run {
  int t, count, blk, first;
};
// Sines and cosines of a run's rows in shared memory: [row][4][lane], two pairs
// of one lane each, so that eight lanes read 128 bytes in a row.
__device__ __forceinline__ Turn turn_from(const float4* table, int row, int l) {
  Turn t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = table[row * 32 + i * 8 + l];
    t.c[2 * i] = v.x, t.s[2 * i] = v.y, t.c[2 * i + 1] = v.z, t.s[2 * i + 1] = v.w;
  }
  return t;
}
__device__ __forceinline__ void fill_table(const Params& p, const Run& u, float4* table, int threads) {
  for (int e = threadIdx.x; e < u.count * 32; e += threads) {
    const int row = e >> 5, pair = 8 * (e & 7) + 2 * ((e >> 3) & 3);
    if (pair >= (p.rot >> 1)) continue;
    const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(p.positions[u.t + row]));
    float4 v;
    sincospif(static_cast<float>(static_cast<int32_t>((pos * p.freqs[pair]) >> 32)) * 0x1p-31f, &v.y, &v.x);
    sincospif(static_cast<float>(static_cast<int32_t>((pos * p.freqs[pair + 1]) >> 32)) * 0x1p-31f, &v.w, &v.z);
    table[e] = v;
  }
}
// Writes a run of at most GROUPS * ROWS rows of one head of K or V; group g of
// the GROUPS that work on it (eight lanes each) takes rows g, g + GROUPS ...
// `all_max` reduces a warp's maximum to that of all groups.  `table`: the rows'
// sines and cosines, or null.
template <int GROUPS, int ROWS, bool INTER, class Reduce>
__device__ __forceinline__ void write_run(const Params& p, const Run& u, int h, bool is_v, int g, const float4* table,
                                          Reduce all_max) {
  const int l = threadIdx.x & 7;
  const Runs run = lane_runs<INTER>(p.rot, l);
  const float* weight = is_v ? nullptr : p.k_weight;
  const bool rotated = !is_v && 8 * l < (p.rot >> 1);
  const uint16_t* src = p.qkv + static_cast<int64_t>(u.t) * p.qkv_stride +
                        static_cast<int64_t>(p.Hq + (is_v ? p.Hkv : 0) + h) * kD;
  float* scale_at = (is_v ? p.v_scale : p.k_scale) + static_cast<int64_t>(u.blk) * p.Hkv + h;
  uint8_t* dst = (is_v ? p.v_cache : p.k_cache) + u.blk * p.block_stride + h * p.head_stride;
  uint4 r0[ROWS], r1[ROWS];
  int pos[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {  // everything that is needed from memory is asked for first
    const int j = g + r * GROUPS;
    r0[r] = r1[r] = make_uint4(0, 0, 0, 0);
    pos[r] = 0;
    if (j < u.count) {
      const uint16_t* row = src + static_cast<int64_t>(j) * p.qkv_stride;
      r0[r] = *reinterpret_cast<const uint4*>(row + run.c0);
      r1[r] = *reinterpret_cast<const uint4*>(row + run.c1);
      if (rotated && !table) pos[r] = p.positions[u.t + j];
    }
  }
  const float old = u.first > 0 ? *scale_at : 0.f;
  Pairs x[ROWS];
  float amax = 0.f;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    x[r] = to_pairs<INTER>(r0[r], r1[r]);
    if (r * GROUPS < u.count) {  // the same for all threads of the run
      if (weight) {
        const Pairs w = load_weight<INTER>(weight, run);
        const float f = norm_factor(x[r], p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[r].a[i] = x[r].a[i] * f * w.a[i], x[r].b[i] = x[r].b[i] * f * w.b[i];
      }
      if (rotated && g + r * GROUPS < u.count) {
        const Turn t = table ? turn_from(table, g + r * GROUPS, l) : turn_of(p, pos[r], l);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = x[r].a[i], b = x[r].b[i];
          x[r].a[i] = a * t.c[i] - b * t.s[i];
          x[r].b[i] = b * t.c[i] + a * t.s[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        amax = fmaxf(amax, fmaxf(fabsf(x[r].a[i]), fabsf(x[r].b[i])));  // passes over NaN
      }
    }
  }
  if (__any_sync(0xffffffffu, amax > FLT_MAX)) {  // an infinity among them: it does not count
    amax = 0.f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = fabsf(x[r].a[i]), b = fabsf(x[r].b[i]);
        amax = fmaxf(amax, fmaxf(a <= FLT_MAX ? a : 0.f, b <= FLT_MAX ? b : 0.f));
      }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  amax = all_max(amax);  // also: every thread of the run has read the old scale
  const float scale = fmaxf(old, fit_scale(amax));
  const float inv = 1.f / scale;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int j = g + r * GROUPS;
    if (j >= u.count) continue;
    float a[8], b[8];
    to_runs<INTER>(x[r], a, b);
    uint8_t* row = dst + (u.first + j) * p.token_stride;
    *reinterpret_cast<uint2*>(row + run.c0) =
        make_uint2(e4m3x4(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv),
                   e4m3x4(a[4] * inv, a[5] * inv, a[6] * inv, a[7] * inv));
    *reinterpret_cast<uint2*>(row + run.c1) =
        make_uint2(e4m3x4(b[0] * inv, b[1] * inv, b[2] * inv, b[3] * inv),
                   e4m3x4(b[4] * inv, b[5] * inv, b[6] * inv, b[7] * inv));
  }
  if (u.first > 0 && scale != old) {  // the older rows follow the scale
    const float ratio = old * inv;
#pragma unroll 4
    for (int j = g; j < u.first; j += GROUPS) {
      uint4* row = reinterpret_cast<uint4*>(dst + j * p.token_stride) + l;
      const uint4 v = *row;
      *row = make_uint4(rescale4(v.x, ratio), rescale4(v.y, ratio), rescale4(v.z, ratio), rescale4(v.w, ratio));
    }
  }
  if (l == 0 && g == 0) *scale_at = scale;
}

// THREADS / 8 * ROWS is at least the block size.
template <int THREADS, int ROWS, bool INTER>
__global__ void __launch_bounds__(THREADS, ROWS > 2 ? 512 / THREADS : 768 / THREADS) qk_rope_kernel(const Params p) {
  constexpr int kWarps = THREADS / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (static_cast<int>(blockIdx.x) < p.cache_ctas) {
    __shared__ float red[kWarps];
    __shared__ int64_t slots[2 * kMaxBlock + 1];  // of the row before the CTA's rows, of them, and a block's worth behind
    __shared__ Run run_of[kMaxBlock];
    __shared__ int runs;
    extern __shared__ float4 table[];
    const int units = 2 * ((p.Hkv + p.heads_per_cta - 1) / p.heads_per_cta), unit = blockIdx.x % units;
    const int h0 = (unit >> 1) * p.heads_per_cta, h1 = min(h0 + p.heads_per_cta, p.Hkv);
    const int base = static_cast<int>(blockIdx.x / units) * p.rows_per_cta;
    const bool is_v = unit & 1;
    const int64_t limit = static_cast<int64_t>(p.num_blocks) * p.bs;
    const int seen = min(p.rows_per_cta + p.bs, p.T - base);
    for (int i = tid; i <= seen; i += THREADS) {
      const int64_t s = base + i > 0 ? p.slot_map[base + i - 1] : -1;
      if (s >= limit && unit == 0 && p.err) atomicOr(p.err, KDA_DEVERR_SLOT_RANGE);
      slots[i] = s >= limit ? -1 : s;
    }
    if (tid == 0) runs = 0;
    __syncthreads();
    // runs that begin here: at the first row of a block, or at a slot that does not follow the row before
    const int rows = min(p.rows_per_cta, p.T - base);
    for (int i = tid; i < rows; i += THREADS) {
      const int64_t s = slots[i + 1];
      if (s >= 0 && (s % p.bs == 0 || slots[i] != s - 1)) {
        Run u;
        u.t = base + i;
        u.blk = static_cast<int>(s / p.bs);
        u.first = static_cast<int>(s % p.bs);
        u.count = 0;
        run_of[atomicAdd(&runs, 1)] = u;
      }
    }
    __syncthreads();
    const int n = runs;
    for (int i = warp; i < n; i += kWarps) {  // how far each goes on in its block
      const Run u = run_of[i];
      const int at = u.t - base + 1, most = min(p.bs - u.first, seen - at + 1);
      const int64_t s = slots[at];
      int count = 0;
      while (count < most) {
        const int j = count + lane;
        const uint32_t on = __ballot_sync(0xffffffffu, j < most && slots[at + j] == s + j);
        count += on == 0xffffffffu ? 32 : __ffs(~on) - 1;
        if (on != 0xffffffffu) break;
      }
      __syncwarp();
      if (lane == 0) run_of[i].count = count;
    }
    __syncthreads();
    for (int i = warp; i < n; i += kWarps)
      if (run_of[i].count <= 4 * ROWS)
        for (int h = h0; h < h1; ++h)
          write_run<4, ROWS, INTER>(p, run_of[i], h, is_v, lane >> 3, nullptr, [](float m) {
            __syncwarp();
            return m;
          });
    const bool shared = !is_v && p.rot > 0 && p.heads_per_cta > 1 && p.bs <= kTableRows;
    for (int i = 0; i < n; ++i) {
      if (run_of[i].count <= 4 * ROWS) continue;
      if (shared) {
        __syncthreads();  // the run before has been read
        fill_table(p, run_of[i], table, THREADS);
        __syncthreads();
      }
      for (int h = h0; h < h1; ++h)
        write_run<THREADS / 8, ROWS, INTER>(p, run_of[i], h, is_v, tid >> 3, shared ? table : nullptr, [&](float m) {
          __syncthreads();  // of the head before: `red` is free
          if (lane == 0) red[warp] = m;
          __syncthreads();
#pragma unroll
          for (int w = 0; w < kWarps; ++w) m = fmaxf(m, red[w]);
          return m;
        });
    }
    return;
  }
  // ---- queries (and k_out): warp = (token, chunk of head groups), four heads at a time
  const int64_t work = static_cast<int64_t>(blockIdx.x - p.cache_ctas) * kWarps + warp;
  const int t = static_cast<int>(work / p.chunks), chunk = static_cast<int>(work - static_cast<int64_t>(t) * p.chunks);
  if (t >= p.T) return;
  const int l = tid & 7, sub = lane >> 3;
  const Runs run = lane_runs<INTER>(p.rot, l);
  const bool rotated = 8 * l < (p.rot >> 1);
  const uint16_t* src = p.qkv + static_cast<int64_t>(t) * p.qkv_stride;
  const int from = chunk * p.iters, to = min(from + p.iters, p.groups);
  // q's groups first, then k's: heads of a group are of one kind
  auto head_of = [&](int i) { return i < p.q_groups ? 4 * i + sub : p.Hq + 4 * (i - p.q_groups) + sub; };
  auto live_of = [&](int i) { return i < p.q_groups ? 4 * i + sub < p.Hq : 4 * (i - p.q_groups) + sub < p.Hkv; };
  uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
  if (live_of(from)) {
    r0 = *reinterpret_cast<const uint4*>(src + head_of(from) * kD + run.c0);
    r1 = *reinterpret_cast<const uint4*>(src + head_of(from) * kD + run.c1);
  }
  const int pos = p.positions[t];
  // weights times cosines and sines: a' = f (a ac - b bs), b' = f (b bc + a as)
  float ac[8], bs[8], bc[8], as[8];
  const float* weight = nullptr;
  for (int i = from; i < to; ++i) {
    if (i == from || i == p.q_groups) {
      weight = i < p.q_groups ? p.q_weight : p.k_weight;
      Pairs w;
#pragma unroll
      for (int k = 0; k < 8; ++k) w.a[k] = w.b[k] = 1.f;
      if (weight) w = load_weight<INTER>(weight, run);
      Turn turn;
#pragma unroll
      for (int k = 0; k < 8; ++k) turn.c[k] = 1.f, turn.s[k] = 0.f;
      if (rotated) turn = turn_of(p, pos, l);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ac[k] = w.a[k] * turn.c[k], as[k] = w.a[k] * turn.s[k];
        bc[k] = w.b[k] * turn.c[k], bs[k] = w.b[k] * turn.s[k];
      }
    }
    const Pairs x = to_pairs<INTER>(r0, r1);
    const int h = head_of(i);
    const bool live = live_of(i);
    if (i + 1 < to) {  // the next group's rows, while this one's are worked on
      r0 = r1 = make_uint4(0, 0, 0, 0);
      if (live_of(i + 1)) {
        r0 = *reinterpret_cast<const uint4*>(src + head_of(i + 1) * kD + run.c0);
        r1 = *reinterpret_cast<const uint4*>(src + head_of(i + 1) * kD + run.c1);
      }
    }
    const float f = weight ? norm_factor(x, p.eps) : 1.f;
    Pairs y;
    if (rotated) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        y.a[k] = f * (x.a[k] * ac[k] - x.b[k] * bs[k]);
        y.b[k] = f * (x.b[k] * bc[k] + x.a[k] * as[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) y.a[k] = f * (x.a[k] * ac[k]), y.b[k] = f * (x.b[k] * bc[k]);
    }
    if (!live) continue;
    float u[8], v[8];
    to_runs<INTER>(y, u, v);
    uint16_t* out = h < p.Hq ? p.q_out + t * p.q_stride + h * kD : p.k_out + t * p.k_stride + (h - p.Hq) * kD;
    *reinterpret_cast<uint4*>(out + run.c0) = pack8(u);
    *reinterpret_cast<uint4*>(out + run.c1) = pack8(v);
  }
}

template <int THREADS, int ROWS>
cudaError_t launch(Params& p, bool interleaved, void* stream) {
  constexpr int kWarps = THREADS / 32;
  int64_t cache_ctas = 0;
  if (p.k_cache) {
    // rows per CTA: as few as fill half the card's room (three CTAs of 256
    // threads an SM; fewer rows cost more CTAs than they help), up to a
    // block's worth on prompts; then all heads that still leave it filled
    const int64_t room = 152 * 768 / THREADS / 2, rows = static_cast<int64_t>(p.T) * p.Hkv * 2 / room;
    p.rows_per_cta = static_cast<int>(rows < 1 ? 1 : rows > p.bs ? p.bs : rows);
    const int64_t chunks = (static_cast<int64_t>(p.T) + p.rows_per_cta - 1) / p.rows_per_cta;
    p.heads_per_cta = p.Hkv;
    while (p.heads_per_cta > 1 && chunks * 2 * (p.Hkv / p.heads_per_cta) < room) p.heads_per_cta = (p.heads_per_cta + 1) / 2;
    cache_ctas = chunks * 2 * ((p.Hkv + p.heads_per_cta - 1) / p.heads_per_cta);
  }
  // warps per token: as many as there are groups of four heads while the
  // batch is small, one per token on prompts (the sines are then computed once)
  int64_t chunks = (static_cast<int64_t>(152) * 24 + p.T - 1) / p.T;
  chunks = chunks < 1 ? 1 : chunks > p.groups ? p.groups : chunks;
  p.iters = static_cast<int>((p.groups + chunks - 1) / chunks);
  p.chunks = (p.groups + p.iters - 1) / p.iters;
  const int64_t ctas = cache_ctas + (static_cast<int64_t>(p.T) * p.chunks + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  p.cache_ctas = static_cast<int>(cache_ctas);
  return kda_internal_launch(interleaved ? qk_rope_kernel<THREADS, ROWS, true> : qk_rope_kernel<THREADS, ROWS, false>,
                             dim3(static_cast<unsigned>(ctas)), dim3(THREADS),
                             p.k_cache && p.heads_per_cta > 1 && p.bs <= kTableRows ? p.bs * 512u : 0u, stream, p);
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
  // in place every warp writes the rows it has read, and only those
  if ((a->q_out == a->qkv && a->q_row_stride != a->qkv_row_stride) ||
      (a->k_out && a->k_out == a->qkv + static_cast<int64_t>(a->num_q_heads) * kD && a->k_row_stride != a->qkv_row_stride))
    return kda_internal_fail(KDA_ERR_SHAPE, "an output in the place of its input needs the input's row stride");
  if (misaligned(a->qkv, 15) || (a->qkv_row_stride & 7) || misaligned(a->q_out, 15) || (a->q_row_stride & 7) ||
      misaligned(a->k_out, 15) || (a->k_out && (a->k_row_stride & 7)) || misaligned(a->positions, 3) ||
      misaligned(a->freqs, 7) || misaligned(a->q_weight, 15) || misaligned(a->k_weight, 15) ||
      misaligned(a->k_cache, 15) || misaligned(a->v_cache, 15) || misaligned(a->k_scale, 3) ||
      misaligned(a->v_scale, 3) || misaligned(a->slot_map, 7) || misaligned(a->err_flag, 3) ||
      (cache && ((a->block_stride | a->head_stride | a->token_stride) & 15)))
    return kda_internal_fail(KDA_ERR_ALIGN, "a pointer or stride is not aligned as required");
  Params p{};
  p.T = a->T, p.Hq = a->num_q_heads, p.Hkv = a->num_kv_heads, p.rot = a->rot_dim, p.bs = bs;
  p.num_blocks = a->num_blocks;
  p.q_groups = (a->num_q_heads + 3) / 4;
  p.groups = p.q_groups + (a->k_out ? (a->num_kv_heads + 3) / 4 : 0);
  p.eps = a->eps;
  p.qkv = a->qkv, p.qkv_stride = a->qkv_row_stride;
  p.q_out = a->q_out, p.q_stride = a->q_row_stride, p.k_out = a->k_out, p.k_stride = a->k_row_stride;
  p.positions = a->positions, p.freqs = a->freqs, p.q_weight = a->q_weight, p.k_weight = a->k_weight;
  p.k_cache = cache ? a->k_cache : nullptr, p.v_cache = a->v_cache;
  p.block_stride = a->block_stride, p.head_stride = a->head_stride, p.token_stride = a->token_stride;
  p.k_scale = a->k_scale, p.v_scale = a->v_scale, p.slot_map = a->slot_map, p.err = a->err_flag;
  // a run of up to block_size rows stays in registers: rows per 8-lane group
  const bool inter = (a->flags & KDA_ROPE_INTERLEAVED) != 0;
  cudaError_t e;
  if (!cache || bs == 64) e = launch<256, 2>(p, inter, stream);
  else if (bs == 16) e = launch<128, 1>(p, inter, stream);
  else if (bs == 32) e = launch<128, 2>(p, inter, stream);
  else if (bs == 128) e = launch<256, 4>(p, inter, stream);
  else e = launch<512, 4>(p, inter, stream);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
  return KDA_OK;
}
