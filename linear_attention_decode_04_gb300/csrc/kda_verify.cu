// kda_verify.cu -- verification of drafted tokens (definition in
// include/kda_verify.h).
//
// HBM bound on large batches (one row of target probabilities per sequence,
// and one of the draft's where a draft was refused), latency bound on small
// ones.  One cluster of CTAs per sequence: every CTA works out for itself
// which draft is the first refused (a few gathers), sums its part of that one
// row, and the CTAs exchange their sums through distributed shared memory;
// the CTA, then the warp, in whose part the inversion ends reads that part
// once more (out of L2) to find the token.  Rows that no sample needs are
// never read.
//
// The weights are 64-bit integers in units of 2^-60, so sums are exact and
// the token does not depend on how the row was split.  They are made from the
// floats' bits with a 64-bit shift: the conversion instruction is several
// times slower and would bound the kernel.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_verify.h"

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

struct Params {
  int N, T, V;
  const int32_t* draft;
  const float *target, *probs;
  int64_t target_stride, probs_stride;
  const float *accept_u, *sample_u;
  const int32_t *src_slot, *slots;
  int32_t *tokens, *accepted, *next;
  int32_t* err;
};

// floor(min(max(x, 0), 1) 2^60), NaN as 0.  With the mantissa at the top of 64
// bits, x = m 2^(e - 190) for exponent field e, so the value is m >> (130 - e);
// x <= 1 has e <= 127, and below 2^-60 nothing is left.
__device__ __forceinline__ uint64_t fixed60(float x) {
  const uint32_t u = __float_as_uint(fminf(fmaxf(x, 0.f), 1.f));
  const uint32_t e = u >> 23;
  const uint64_t m = static_cast<uint64_t>((u << 8) | 0x80000000u) << 32;
  const uint32_t shift = 130u - e;
  return shift < 64 ? m >> shift : 0;
}

// What a row's weights are made of: w = max(P - Q, 0) with Q from the draft's
// row, or P with the refused token taken out, or P.
struct Row {
  const float *p, *q;
  int out;  // token taken out, or -1
};
template <bool VEC>
__device__ __forceinline__ void load4(const float* row, int i, int V, float (&x)[4]) {
  if (VEC && i + 4 <= V) {
    const float4 v = *reinterpret_cast<const float4*>(row + i);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = i + k < V ? row[i + k] : 0.f;
  }
}
__device__ __forceinline__ uint64_t weight(const Row& r, float p, float q, int i) {
  const uint64_t P = fixed60(p), Q = fixed60(q);
  return i == r.out ? 0 : P > Q ? P - Q : 0;
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads) verify_kernel(const Params p, int cluster, int part) {
  __shared__ uint64_t cta_sum[2][kMaxCluster];  // every CTA's sum, in every CTA; of the rest, of the row itself
  __shared__ uint64_t warp_sums[kWarps], found[kWarps];
  __shared__ int verdict[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = blockIdx.x / cluster, rank = blockIdx.x - n * cluster;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (p.src_slot && p.src_slot[n] <= 0) {  // the whole cluster leaves here
    if (rank == 0) {
      if (tid < p.T) p.tokens[static_cast<int64_t>(n) * p.T + tid] = -1;
      if (tid == 0) {
        p.accepted[n] = 0;
        if (p.next) p.next[n] = 0;
      }
    }
    return;
  }
  // a CTA's memory may be written once that CTA has started: arrive here, wait
  // before the exchange
  if (cluster > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  if (warp == 0) {
    bool stands = false, drafted = false;
    if (lane < p.T - 1) {
      const int64_t at = static_cast<int64_t>(n) * (p.T - 1) + lane;
      const int d = p.draft[at];
      drafted = d >= 0 && d < p.V;
      if (d >= p.V && rank == 0 && p.err) atomicOr(p.err, KDA_DEVERR_TOKEN_RANGE);
      if (drafted) {
        const double u = p.accept_u[at];
        const double q = p.probs ? p.probs[at * p.probs_stride + d] : 1.f;
        stands = u * q < p.target[(static_cast<int64_t>(n) * p.T + lane) * p.target_stride + d];
      }
    }
    const uint32_t s = __ballot_sync(0xffffffffu, stands), v = __ballot_sync(0xffffffffu, drafted);
    if (lane == 0) {
      const int k = __ffs(~s) - 1;  // leading drafts that stand; at most T - 1 < 32
      verdict[0] = k;
      verdict[1] = (v >> k) & 1;    // a draft stood at k and was refused
    }
  }
  __syncthreads();
  const int k = verdict[0];
  const bool refused = verdict[1];
  Row r;
  r.p = p.target + (static_cast<int64_t>(n) * p.T + k) * p.target_stride;
  r.q = refused && p.probs ? p.probs + (static_cast<int64_t>(n) * (p.T - 1) + k) * p.probs_stride : nullptr;
  r.out = refused && !p.probs ? p.draft[static_cast<int64_t>(n) * (p.T - 1) + k] : -1;
  // this warp's part of the row: `part` consecutive tokens
  const int64_t lo64 = static_cast<int64_t>(rank * kWarps + warp) * part;
  const int lo = static_cast<int>(lo64 < p.V ? lo64 : p.V);
  const int hi = static_cast<int>(lo64 + part < p.V ? lo64 + part : p.V);
  const float u = fmaxf(p.sample_u[n], 0.f);
  const uint64_t u31 = u < 1.f ? static_cast<uint64_t>(u * 0x1p31f) : 0x7fffffffu;
  uint64_t total = 0, before = 0;  // of the whole row; ahead of this CTA
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {  // the second round where the rest has no mass: the row itself
    uint64_t sum = 0;
#pragma unroll 4
    for (int i = lo + 4 * lane; i < hi; i += 128) {
      float a[4], b[4] = {0.f, 0.f, 0.f, 0.f};
      load4<VEC>(r.p, i, p.V, a);
      if (r.q) load4<VEC>(r.q, i, p.V, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += weight(r, a[j], b[j], i + j);
    }
    sum = warp_sum(sum);
    if (lane == 0) warp_sums[warp] = sum;
    __syncthreads();
    if (cluster > 1 && round == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (warp == 0) {
      const uint64_t s = warp_sum(lane < kWarps ? warp_sums[lane] : 0);
      if (cluster == 1) {
        if (lane == 0) cta_sum[round][0] = s;
      } else if (lane < cluster) {  // lane c tells CTA c
        asm volatile(
            "{\n\t.reg .b32 x;\n\tmapa.shared::cluster.u32 x, %0, %1;\n\tst.shared::cluster.u64 [x], %2;\n\t}" ::"r"(
                static_cast<uint32_t>(__cvta_generic_to_shared(&cta_sum[round][rank]))),
            "r"(lane), "l"(s)
            : "memory");
      }
    }
    if (cluster > 1) cluster_barrier();  // no CTA reads another's memory behind this
    else __syncthreads();
    total = before = 0;
    for (int c = 0; c < cluster; ++c) {
      total += cta_sum[round][c];
      if (c < rank) before += cta_sum[round][c];
    }
    if (total != 0 || !refused) break;
    r.q = nullptr, r.out = -1;
  }
  const uint64_t goal = __umul64hi(u31 << 33, total);  // floor(u31 total / 2^31)
  if (rank == 0) {
    if (tid < p.T && tid != k) p.tokens[static_cast<int64_t>(n) * p.T + tid] = tid < k ? p.draft[static_cast<int64_t>(n) * (p.T - 1) + tid] : -1;
    if (tid == 0) {
      p.accepted[n] = k;
      if (p.next) p.next[n] = p.slots[static_cast<int64_t>(n) * p.T + k];
      if (total == 0) p.tokens[static_cast<int64_t>(n) * p.T + k] = p.V - 1;
    }
  }
  // the warp in whose part the inversion ends
  int owner = -1;
  for (int w = 0; w < kWarps; ++w) {
    if (owner < 0 && goal >= before) {
      if (goal < before + warp_sums[w]) owner = w;
      else before += warp_sums[w];
    }
  }
  if (total == 0 || owner < 0) return;  // not this CTA's part
  // That part once more, with all threads: each takes `each` tokens in a row.
  const int64_t begin = static_cast<int64_t>(rank * kWarps + owner) * part;
  const int each = (part + 4 * kThreads - 1) / (4 * kThreads) * 4;
  const int last = static_cast<int>(begin + part < p.V ? begin + part : p.V);
  const int64_t from64 = begin + static_cast<int64_t>(tid) * each;
  const int from = static_cast<int>(from64 < last ? from64 : last), to = min(from + each, last);
  uint64_t mine = 0;
#pragma unroll 2
  for (int i = from; i < to; i += 4) {
    float a[4], b[4] = {0.f, 0.f, 0.f, 0.f};
    load4<VEC>(r.p, i, p.V, a);
    if (r.q) load4<VEC>(r.q, i, p.V, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) mine += i + j < to ? weight(r, a[j], b[j], i + j) : 0;
  }
  uint64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) found[warp] = x;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before += found[w];
  before += x - mine;
  if (goal < before || goal >= before + mine) return;
  for (int i = from; i < to; i += 4) {  // one thread is left
    float a[4], b[4] = {0.f, 0.f, 0.f, 0.f};
    load4<VEC>(r.p, i, p.V, a);
    if (r.q) load4<VEC>(r.q, i, p.V, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t w = i + j < to ? weight(r, a[j], b[j], i + j) : 0;
      if (w > 0 && goal >= before && goal < before + w) p.tokens[static_cast<int64_t>(n) * p.T + k] = i + j;
      before += w;
    }
  }
}

bool misaligned(const void* ptr, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(ptr) & mask) != 0; }

}  // namespace

extern "C" int kda_verify_draft(const KdaVerifyArgs* a, void* stream) {
  kda_internal_clear_error();
  if (!a) return kda_internal_fail(KDA_ERR_NULLPTR, "args is NULL");
  if (a->struct_size != sizeof(KdaVerifyArgs))
    return kda_internal_fail(KDA_ERR_ABI, "struct_size %u, library expects %zu", a->struct_size, sizeof(KdaVerifyArgs));
  if (a->N < 0 || a->T < 1 || a->T > KDA_MAX_TOKENS_PER_SEQ || a->V < 1 || a->V > (1 << 30))
    return kda_internal_fail(KDA_ERR_SHAPE, "N=%d T=%d V=%d", a->N, a->T, a->V);
  if (a->N > 0x7fffffff / kMaxCluster) return kda_internal_fail(KDA_ERR_SHAPE, "N=%d is too large", a->N);
  if (a->N == 0) return KDA_OK;
  const bool drafts = a->T > 1;
  if (!a->target_probs || !a->sample_u || !a->tokens || !a->num_accepted || (drafts && (!a->draft_tokens || !a->accept_u)) ||
      (a->slot_idx != nullptr) != (a->next_slot != nullptr))
    return kda_internal_fail(KDA_ERR_NULLPTR, "a required pointer is NULL (slot_idx and next_slot go together)");
  const float* probs = drafts ? a->draft_probs : nullptr;
  if (a->target_row_stride < a->V || (probs && a->draft_row_stride < a->V))
    return kda_internal_fail(KDA_ERR_SHAPE, "a row stride is smaller than the row");
  if (misaligned(a->draft_tokens, 3) || misaligned(a->target_probs, 3) || misaligned(probs, 3) ||
      misaligned(a->accept_u, 3) || misaligned(a->sample_u, 3) || misaligned(a->src_slot, 3) ||
      misaligned(a->slot_idx, 3) || misaligned(a->tokens, 3) || misaligned(a->num_accepted, 3) ||
      misaligned(a->next_slot, 3) || misaligned(a->err_flag, 3))
    return kda_internal_fail(KDA_ERR_ALIGN, "a pointer is not aligned as required");
  const Params p{a->N, a->T, a->V, a->draft_tokens, a->target_probs, probs, a->target_row_stride, a->draft_row_stride,
                 a->accept_u, a->sample_u, a->src_slot, a->slot_idx, a->tokens, a->num_accepted, a->next_slot,
                 a->err_flag};
  // CTAs per sequence: as many as are resident at once (four of 512 threads on
  // each of 152 SMs), one on the largest batches
  int cluster = kMaxCluster;
  while (cluster > 1 && static_cast<int64_t>(a->N) * cluster > 4 * 152) cluster >>= 1;
  const int parts = cluster * kWarps;
  const int part = static_cast<int>((static_cast<int64_t>(a->V) + parts * 128LL - 1) / (parts * 128LL)) * 128;
  const bool vec = !misaligned(a->target_probs, 15) && a->target_row_stride % 4 == 0 &&
                   (!probs || (!misaligned(probs, 15) && a->draft_row_stride % 4 == 0));
  const dim3 grid(static_cast<unsigned>(a->N) * cluster);
  const cudaError_t e = kda_internal_launch_cluster(vec ? verify_kernel<true> : verify_kernel<false>, grid,
                                                    dim3(kThreads), 0, stream, cluster, p, cluster, part);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
  return KDA_OK;
}
