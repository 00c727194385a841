// kda_add_norm.cu -- residual addition, root-mean-square norm and 8-bit
// output (definition in include/kda_add_norm.h).
//
// A CTA (or a warp) per row: the row stays in registers from its load to its
// codes, so that every byte crosses HBM once, which bounds large calls: 16,384
// rows of 6,144 channels with residual and 8-bit output, 705 MB, 103.2 us,
// 6.8 TB/s (some of it from L2; a copy has 6.8).  256 rows take 4.1 us (2.1 at
// that rate), 4 rows of 2,048 2.9: the launch, a load and its two reductions.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_add_norm.h"
#include "kda_internal.h"
#include "kda_tc.cuh"

namespace {

constexpr float kPerCode = 1.f / 448.f;   // 448 is the largest e4m3 value
constexpr float kScaleFloor = 0x1p-100f;
constexpr float kLeastSquare = 0x1p-120f;  // of a mean: one of squares that fp32 holds with all their digits
constexpr uint32_t kInfinity = 0x7f800000u;
constexpr int kShort = 512;               // channels of rows that a warp takes
constexpr int kRows = 4;                  // of these, in a CTA

struct Params {
  int T, D;
  float eps;
  const uint16_t *x, *residual;
  int64_t x_stride, residual_stride;
  const float* weight;
  uint16_t *residual_out, *out;
  int64_t residual_out_stride, out_stride;
  uint8_t* out_q;
  int64_t out_q_stride;
  float* out_scale;
};

__device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The quotients by the scale as it is stored, rounded to fp32 and then to codes.  (Products with 448 / amax as rounded give
// 229 of 9.5 million codes of bf16 rows the other neighbour of a quotient near their middle.)  q = f r with r = 1 / scale
// rounded, and once more with its exact remainder: q + (f - q scale) r is the rounded quotient (Markstein 1990).  A
// division per element instead: 16,384 rows of 6,144 channels 120 us instead of 104, without residual and norm 71 instead
// of 55 (with the product alone 104 and 53).
__device__ __forceinline__ uint2 codes(const float (&f)[8], float scale, float inv) {
  const uint64_t r = pair_of(inv, inv), minus = pair_of(-scale, -scale);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t x = pair_of(f[2 * i], f[2 * i + 1]), q = mul2(x, r);
    w[i] = __nv_cvt_float2_to_fp8x2(both(fma2(fma2(q, minus, x), r, q)), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

__device__ __forceinline__ float warp_total(float x) {  // in all lanes the same
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A CTA per row, or a warp per row (WARP): a thread holds VECS pieces of 8 channels, as many apart as threads have the row.
template <int VECS, bool NORM, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kRows : 1024) add_norm_kernel(const Params p) {
  __shared__ float sums[32];
  __shared__ uint32_t tops[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, n = p.D / 8;
  const int tid = WARP ? lane : threadIdx.x, apart = WARP ? 32 : blockDim.x;  // of the row
  const int64_t t = WARP ? static_cast<int64_t>(blockIdx.x) * kRows + warp : blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (WARP && t >= p.T) return;
  float h[VECS][8], total = 0.f;
  {
    uint4 a[VECS], b[VECS];
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int c = tid + i * apart;
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (c < n) {
        a[i] = reinterpret_cast<const uint4*>(p.x + t * p.x_stride)[c];
        if (p.residual) b[i] = reinterpret_cast<const uint4*>(p.residual + t * p.residual_stride)[c];
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      float r[8];
      unpack(a[i], h[i]);
      unpack(b[i], r);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        h[i][k] += r[k];
        sum = fmaf(h[i][k], h[i][k], sum);
      }
    }
    if (NORM) {
      sum = warp_total(sum);
      if (WARP) total = sum;
      else if (lane == 0) sums[warp] = sum;
    }
  }
  // the row's largest magnitude, as a bit pattern: NaN above infinity above everything else
  auto row_top = [&]() {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(h[i][k]) & 0x7fffffffu);
    top = __reduce_max_sync(0xffffffffu, top);
    if (!WARP) {
      if (lane == 0) tops[warp] = top;
      __syncthreads();
      top = __reduce_max_sync(0xffffffffu, lane < warps ? tops[lane] : 0);
    }
    return top;
  };
  if (!WARP) __syncthreads();
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int c = tid + i * apart;
    if (c < n && p.residual_out) reinterpret_cast<uint4*>(p.residual_out + t * p.residual_out_stride)[c] = pack(h[i]);
  }
  if (NORM) {
    if (!WARP) {
      total = warp_total(lane < warps ? sums[lane] : 0.f);
    }
    const float square = total / static_cast<float>(p.D) + p.eps;
    float f = 1.f / sqrtf(square);
    // Squares that pass fp32's range, or lose digits at its other end: once more, with the row and eps relative to a power
    // of two near the largest of them.  (All threads of the row have the same sum.)
    if (!(total < INFINITY) || square < kLeastSquare) {
      const uint32_t top = row_top();
      const float most = fmaxf(__uint_as_float(top), sqrtf(p.eps));
      if (top < kInfinity && most > 0.f && most < INFINITY) {
        const float by = __uint_as_float(static_cast<uint32_t>(min(max(254 - (__float_as_int(most) >> 23), 1), 254)) << 23);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VECS; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            h[i][k] *= by;
            sum = fmaf(h[i][k], h[i][k], sum);
          }
        sum = warp_total(sum);
        if (!WARP) {
          if (lane == 0) sums[warp] = sum;
          __syncthreads();
          sum = warp_total(lane < warps ? sums[lane] : 0.f);
        }
        const float e = sqrtf(p.eps) * by;
        f = 1.f / sqrtf(sum / static_cast<float>(p.D) + e * e);
      }
    }
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int c = tid + i * apart;
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] *= f;
      if (c < n && p.weight) {
        const float4 u = reinterpret_cast<const float4*>(p.weight)[2 * c], v = reinterpret_cast<const float4*>(p.weight)[2 * c + 1];
        h[i][0] *= u.x, h[i][1] *= u.y, h[i][2] *= u.z, h[i][3] *= u.w;
        h[i][4] *= v.x, h[i][5] *= v.y, h[i][6] *= v.z, h[i][7] *= v.w;
      }
    }
  }
  if (p.out) {
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int c = tid + i * apart;
      if (c < n) reinterpret_cast<uint4*>(p.out + t * p.out_stride)[c] = pack(h[i]);
    }
  }
  if (!p.out_q) return;
  const uint32_t top = row_top();
  const float amax = top < kInfinity ? fmaxf(__uint_as_float(top), kScaleFloor) : __uint_as_float(0x7fc00000u);
  const float scale = amax * kPerCode, inv = 1.f / scale;
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int c = tid + i * apart;
    if (c < n) reinterpret_cast<uint2*>(p.out_q + t * p.out_q_stride)[c] = codes(h[i], scale, inv);
  }
  if (tid == 0) p.out_scale[t] = scale;
}

bool misaligned(const void* ptr, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(ptr) & mask) != 0; }

template <bool NORM>
auto kernel_of(int vecs, bool warp) {
  if (warp)
    return vecs == 1 ? add_norm_kernel<1, NORM, true> : add_norm_kernel<2, NORM, true>;
  return vecs == 1 ? add_norm_kernel<1, NORM, false> : vecs == 2 ? add_norm_kernel<2, NORM, false>
       : vecs == 3 ? add_norm_kernel<3, NORM, false> : add_norm_kernel<4, NORM, false>;
}

}  // namespace

extern "C" int kda_add_norm(const KdaAddNormArgs* a, void* stream) {
  kda_internal_clear_error();
  if (!a) return kda_internal_fail(KDA_ERR_NULLPTR, "args is NULL");
  if (a->struct_size != sizeof(KdaAddNormArgs))
    return kda_internal_fail(KDA_ERR_ABI, "struct_size %u, library expects %zu", a->struct_size, sizeof(KdaAddNormArgs));
  if (a->flags & ~KDA_ADD_NORM_NO_NORM) return kda_internal_fail(KDA_ERR_FLAGS, "unknown flags 0x%x", a->flags);
  const bool norm = !(a->flags & KDA_ADD_NORM_NO_NORM);
  if (!norm && a->weight) return kda_internal_fail(KDA_ERR_FLAGS, "a weight without the norm");
  if (a->T < 0 || a->D < 8 || a->D % 8 || a->D > KDA_ADD_NORM_MAX_D || !(a->eps >= 0.f))
    return kda_internal_fail(KDA_ERR_SHAPE, "T=%d D=%d eps=%g (D a multiple of 8 up to %d)", a->T, a->D,
                             static_cast<double>(a->eps), KDA_ADD_NORM_MAX_D);
  if (a->T == 0) return KDA_OK;
  if (!a->x || (!a->out && !a->out_q && !a->residual_out) || (a->out_q != nullptr) != (a->out_scale != nullptr))
    return kda_internal_fail(KDA_ERR_NULLPTR, "x and a result are required; out_q and out_scale go together");
  if (a->x_row_stride < a->D || (a->residual && a->residual_row_stride < a->D) ||
      (a->residual_out && a->residual_out_row_stride < a->D) || (a->out && a->out_row_stride < a->D) ||
      (a->out_q && a->out_q_row_stride < a->D))
    return kda_internal_fail(KDA_ERR_SHAPE, "a row stride is smaller than the row");
  if (misaligned(a->x, 15) || (a->x_row_stride & 7) || (a->residual && (misaligned(a->residual, 15) || (a->residual_row_stride & 7))) ||
      (a->residual_out && (misaligned(a->residual_out, 15) || (a->residual_out_row_stride & 7))) ||
      (a->out && (misaligned(a->out, 15) || (a->out_row_stride & 7))) ||
      (a->out_q && (misaligned(a->out_q, 7) || (a->out_q_row_stride & 7))) || misaligned(a->weight, 15) ||
      misaligned(a->out_scale, 3))
    return kda_internal_fail(KDA_ERR_ALIGN, "a pointer or stride is not aligned as required");
  // a result in the place of an input has to have its rows in the same places
  const auto races = [](const void* r, int64_t rs, const void* i, int64_t is) { return r && r == i && rs != is; };
  if (races(a->residual_out, a->residual_out_row_stride, a->x, a->x_row_stride) ||
      races(a->residual_out, a->residual_out_row_stride, a->residual, a->residual_row_stride) ||
      races(a->out, a->out_row_stride, a->x, a->x_row_stride) ||
      races(a->out, a->out_row_stride, a->residual, a->residual_row_stride) || (a->out && a->out == a->residual_out) ||
      (a->out_q && (static_cast<const void*>(a->out_q) == a->x || static_cast<const void*>(a->out_q) == a->residual ||
                    static_cast<const void*>(a->out_q) == a->out || static_cast<const void*>(a->out_q) == a->residual_out)))
    return kda_internal_fail(KDA_ERR_SHAPE, "a result stands in the place of another or, with another stride, of an input");
  const Params p{a->T, a->D, a->eps, a->x, a->residual, a->x_row_stride, a->residual_row_stride, a->weight,
                 a->residual_out, a->out, a->residual_out_row_stride, a->out_row_stride, a->out_q, a->out_q_row_stride,
                 a->out_scale};
  // A warp for short rows: 40,000 rows of 256 channels 13.6 us (with CTAs 40.6), of 512 23.3 (40.9), a few rows of 512
  // 1.9 (1.7); of 1,024 43.5 (46.8) and 2.1 (1.75), which is not worth it.  Others have up to 256 threads with one to
  // three pieces each, then more threads.  (By the row's length alone: a row's results do not depend on how many there are.)
  const int n = a->D / 8;
  const bool warp = a->D <= kShort;
  const int vecs = warp ? (n + 31) / 32 : n > 768 ? 4 : (n + 255) / 256;
  const int threads = warp ? 32 * kRows : ((n + vecs - 1) / vecs + 31) / 32 * 32;
  const int64_t ctas = warp ? (static_cast<int64_t>(a->T) + kRows - 1) / kRows : a->T;
  const cudaError_t e = kda_internal_launch(norm ? kernel_of<true>(vecs, warp) : kernel_of<false>(vecs, warp),
                                            dim3(static_cast<unsigned>(ctas)), dim3(threads), 0, stream, p);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
  return KDA_OK;
}
