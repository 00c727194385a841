// kda_verify.cu -- verification of drafted tokens (definition in
// include/kda_verify.h).
//
// HBM bound on large batches (one row of target probabilities per sequence,
// and one of the draft's where a draft was refused), latency bound on small
// ones: measured on a GB300, 131,072 tokens, 256 sequences of 4 rows 49 us for
// the 206 MB that are read (4.2 TB/s; sequences whose draft was refused read two
// rows, the others one).  The loads alone took 37 us, a copy would take 30: what is
// missing is most likely bytes in flight, two 16-byte loads per row and thread, in the
// registers that the arithmetic needs too.  That 1,024 CTAs are 1.7 times what is
// resident is not it: CTAs that take rows from a counter were no faster.  One sequence
// takes 6.6 to 7.6 us from card to card, of which the trips decide -> row -> exchange ->
// search take most.  One cluster of CTAs per sequence: every CTA works out for itself which
// draft is the first refused (a few gathers), sums its part of that one row,
// and the CTAs exchange their sums through distributed shared memory; the CTA
// and warp in whose part the inversion ends have that part read once more (out
// of L2) to find the token.  Rows that no sample needs are never read.
//
// The weights are integers in units of 2^-60, so sums are exact and the token
// does not depend on how the row was split.  Making such integers from floats
// with shifts or conversions bounds the kernel (the integer and conversion
// pipes are the slow ones: 52 us where the loads alone took 37); instead every
// weight is cut, with additions of a large constant and without error, into
// multiples of 2^-20, 2^-41 and 2^-60, and each kind is summed in fp32 where
// such sums are exact: the first because a row's mass is below 2^3, the
// others for eight tokens at a time.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_verify.h"

namespace {

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

__device__ __forceinline__ float clamp01(float x) { return __saturatef(x); }  // NaN as 0
// x rounded to a multiple of 2^(E - 23), for |x| < 2^(E - 1): 1.5 * 2^E has its
// last bit there.
template <int E>
__device__ __forceinline__ float multiple(float x) {
  constexpr float c = E == 3 ? 12.f : E == -18 ? 0x1.8p-18f : 0x1.8p-37f;
  static_assert(E == 3 || E == -18 || E == -37, "one of the three units");
  return __fsub_rn(__fadd_rn(x, c), c);
}
// Sums of weights: `a` in multiples of 2^-20, b of 2^-41, c of 2^-60.
struct Parts {
  float a = 0.f, b = 0.f, c = 0.f;
  __device__ __forceinline__ void low(float x) {  // |x| < 2^-19
    const float h = multiple<-18>(x);
    b += h;
    c += multiple<-37>(x - h);
  }
  __device__ __forceinline__ void add(float x) {  // 0 <= x <= 1
    const float h = multiple<3>(x);
    a += h;
    low(x - h);
  }
  // max(x - y, 0) for x, y in [0, 1]: d is the difference, e what its rounding left out
  __device__ __forceinline__ void add_difference(float x, float y) {
    const float z = fmaxf(x, y), d = z - y, e = (z - d) - y;
    add(d);
    low(e);
  }
  __device__ __forceinline__ uint64_t low_sum() const {
    return (static_cast<uint64_t>(static_cast<int64_t>(__float2int_rn(b * 0x1p41f))) << 19) +
           static_cast<uint64_t>(static_cast<int64_t>(__float2int_rn(c * 0x1p60f)));
  }
  __device__ __forceinline__ uint64_t sum() const { return (static_cast<uint64_t>(__float2uint_rn(a * 0x1p20f)) << 40) + low_sum(); }
};

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
  Parts w;
  if (i != r.out) w.add_difference(clamp01(p), clamp01(q));
  return w.sum();
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Sum of this lane's share of the weights of tokens lo .. hi - 1 (lo a
// multiple of 4), which the warp goes through four tokens a lane at a time.  DEPTH
// loads per row are always on their way while the ones before are worked on:
// the arithmetic takes about as long as the row takes to come.  The last
// hi % 4 tokens come separately.
template <bool VEC, int DEPTH>
__device__ __forceinline__ uint64_t sum_weights(const Row& r, int lo, int hi, int first) {
  constexpr int stride = 128;
  const int full = lo + ((hi - lo) & ~3);
  auto four = [&](const float* row, int i) {  // nothing past the end; tokens there weigh 0
    if (i >= full) return make_float4(0.f, 0.f, 0.f, 0.f);
    if (VEC) return *reinterpret_cast<const float4*>(row + i);
    return make_float4(row[i], row[i + 1], row[i + 2], row[i + 3]);
  };
  uint64_t sum = 0;  // of the lower parts
  float high = 0.f;
  int i = lo + 4 * first;
  float4 a[DEPTH], b[DEPTH];
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) a[d] = four(r.p, i + d * stride);
  if (r.q) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) b[d] = four(r.q, i + d * stride);
    for (; i < full; i += DEPTH * stride) {
      Parts w;
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        const float4 x = a[d], y = b[d];
        a[d] = four(r.p, i + (DEPTH + d) * stride);
        b[d] = four(r.q, i + (DEPTH + d) * stride);
        w.add_difference(clamp01(x.x), clamp01(y.x));
        w.add_difference(clamp01(x.y), clamp01(y.y));
        w.add_difference(clamp01(x.z), clamp01(y.z));
        w.add_difference(clamp01(x.w), clamp01(y.w));
        if (d & 1 || d + 1 == DEPTH) sum += w.low_sum(), w.b = w.c = 0.f;  // of eight tokens
      }
      high += w.a;
    }
  } else {
    for (; i < full; i += DEPTH * stride) {
      Parts w;
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        const float4 x = a[d];
        a[d] = four(r.p, i + (DEPTH + d) * stride);
        w.add(clamp01(x.x));
        w.add(clamp01(x.y));
        w.add(clamp01(x.z));
        w.add(clamp01(x.w));
        if (d & 1 || d + 1 == DEPTH) sum += w.low_sum(), w.b = w.c = 0.f;
      }
      high += w.a;
    }
    if (first == 0 && r.out >= lo && r.out < full) {
      Parts w;
      w.add(clamp01(r.p[r.out]));
      sum -= w.sum();
    }
  }
  sum += static_cast<uint64_t>(__float2uint_rn(high * 0x1p20f)) << 40;
  if (first < hi - full) sum += weight(r, r.p[full + first], r.q ? r.q[full + first] : 0.f, full + first);
  return sum;
}
// All threads of the CTA: the token among begin .. end - 1 (`before` is the
// weight ahead of them) at which the running sum passes `goal`, four tokens a
// thread and a block of 4 * THREADS at a time.
template <bool VEC, int THREADS>
__device__ __forceinline__ void search(const Row& r, int begin, int end, uint64_t before, uint64_t goal, int V,
                                       int32_t* token) {
  __shared__ uint64_t found[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int64_t block = begin; block < end; block += 4 * THREADS) {
    const int i = static_cast<int>(min(block + 4 * tid, static_cast<int64_t>(end)));
    float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
    if (i < end) {
      load4<VEC>(r.p, i, V, a);
      if (r.q) load4<VEC>(r.q, i, V, b);
    }
    uint64_t w[4], mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) mine += w[j] = i + j < end ? weight(r, a[j], b[j], i + j) : 0;
    uint64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) found[warp] = x;
    __syncthreads();
    uint64_t here = before;
#pragma unroll
    for (int u = 0; u < THREADS / 32; ++u) {
      if (u < warp) here += found[u];
      before += found[u];
    }
    here += x - mine;
    if (goal >= here && goal < here + mine) {
      int j = 0;
      while (j < 3 && goal >= here + w[j]) here += w[j++];
      *token = min(i + j, end - 1);  // (past the end only where sums ran over)
    }
    if (goal < before) return;
  }
}
// How many drafts of sequence n stand, and whether the next was refused (warp 0).
__device__ __forceinline__ void decide(const Params& p, int n, bool report, int* outcome) {
  const int lane = threadIdx.x & 31;
  bool stands = false, drafted = false;
  if (lane < p.T - 1) {
    const int64_t at = static_cast<int64_t>(n) * (p.T - 1) + lane;
    const int d = p.draft[at];
    drafted = d >= 0 && d < p.V;
    if (d >= p.V && report && p.err) atomicOr(p.err, KDA_DEVERR_TOKEN_RANGE);
    if (drafted) {
      const double u = p.accept_u[at];
      const double q = p.probs ? p.probs[at * p.probs_stride + d] : 1.f;
      stands = u * q < p.target[(static_cast<int64_t>(n) * p.T + lane) * p.target_stride + d];
    }
  }
  const uint32_t s = __ballot_sync(0xffffffffu, stands), v = __ballot_sync(0xffffffffu, drafted);
  if (lane == 0) {
    const int k = __ffs(~s) - 1;  // leading drafts that stand; at most T - 1 < 32
    outcome[0] = k;
    outcome[1] = (v >> k) & 1;    // a draft stood at k and was refused
  }
}
__device__ __forceinline__ Row row_of(const Params& p, int n, int k, bool refused) {
  Row r;
  r.p = p.target + (static_cast<int64_t>(n) * p.T + k) * p.target_stride;
  r.q = refused && p.probs ? p.probs + (static_cast<int64_t>(n) * (p.T - 1) + k) * p.probs_stride : nullptr;
  r.out = refused && !p.probs ? p.draft[static_cast<int64_t>(n) * (p.T - 1) + k] : -1;
  return r;
}
__device__ __forceinline__ void write_padding(const Params& p, int n) {
  const int tid = threadIdx.x;
  if (tid < p.T) p.tokens[static_cast<int64_t>(n) * p.T + tid] = -1;
  if (tid == 0) {
    p.accepted[n] = 0;
    if (p.next) p.next[n] = 0;
  }
}
__device__ __forceinline__ uint64_t goal_of(const Params& p, int n, uint64_t total) {  // floor(u31 total / 2^31)
  const float u = fmaxf(p.sample_u[n], 0.f);
  const uint64_t u31 = u < 1.f ? static_cast<uint64_t>(u * 0x1p31f) : 0x7fffffffu;
  return __umul64hi(u31 << 33, total);
}
__device__ __forceinline__ void write_results(const Params& p, int n, int k) {
  const int tid = threadIdx.x;
  if (tid < p.T && tid != k) p.tokens[static_cast<int64_t>(n) * p.T + tid] = tid < k ? p.draft[static_cast<int64_t>(n) * (p.T - 1) + tid] : -1;
  if (tid == 0) {
    p.accepted[n] = k;
    if (p.next) p.next[n] = p.slots[static_cast<int64_t>(n) * p.T + k];
  }
}

// A warp's part of the row is `part` consecutive tokens.
template <bool VEC, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) verify_kernel(const Params p, int cluster, int part) {
  constexpr int kWarps = THREADS / 32;
  __shared__ uint64_t cta_sum[2][kMaxCluster];  // every CTA's sum, in every CTA; of the rest, of the row itself
  __shared__ uint64_t warp_sums[kWarps];
  __shared__ int outcome[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = blockIdx.x / cluster, rank = blockIdx.x - n * cluster;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (p.src_slot && p.src_slot[n] <= 0) {  // the whole cluster leaves here
    if (rank == 0) write_padding(p, n);
    return;
  }
  // a CTA's memory may be written once that CTA has started: arrive here, wait
  // before the exchange
  if (cluster > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  if (warp == 0) decide(p, n, rank == 0, outcome);
  __syncthreads();
  const int k = outcome[0];
  const bool refused = outcome[1];
  // the token of a row without mass, or of one whose sums run over; the barriers
  // below put it before the one that is found
  if (rank == 0 && tid == 0) p.tokens[static_cast<int64_t>(n) * p.T + k] = p.V - 1;
  Row r = row_of(p, n, k, refused);
  // this warp's part of the row: `part` consecutive tokens
  const int64_t lo64 = static_cast<int64_t>(rank * kWarps + warp) * part;
  const int lo = static_cast<int>(lo64 < p.V ? lo64 : p.V);
  const int hi = static_cast<int>(lo64 + part < p.V ? lo64 + part : p.V);
  uint64_t total = 0, before = 0;  // of the whole row; ahead of this CTA
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {  // the second round where the rest has no mass: the row itself
    uint64_t sum = sum_weights<VEC, 2>(r, lo, hi, lane);
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
  const uint64_t goal = goal_of(p, n, total);
  if (rank == 0) write_results(p, n, k);
  // the warp in whose part the inversion ends
  int owner = -1;
  for (int w = 0; w < kWarps; ++w) {
    if (owner < 0 && goal >= before) {
      if (goal < before + warp_sums[w]) owner = w;
      else before += warp_sums[w];
    }
  }
  if (total == 0 || owner < 0) return;  // not this CTA's part
  const int64_t begin = static_cast<int64_t>(rank * kWarps + owner) * part;
  search<VEC, THREADS>(r, static_cast<int>(begin), static_cast<int>(begin + part < p.V ? begin + part : p.V), before, goal,
                       p.V, p.tokens + static_cast<int64_t>(n) * p.T + k);
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
  if ((drafts && a->tokens == a->draft_tokens) || (a->src_slot && (a->tokens == a->src_slot || a->num_accepted == a->src_slot)) ||
      (a->slot_idx && (a->next_slot == a->slot_idx || a->tokens == a->slot_idx)))
    return kda_internal_fail(KDA_ERR_SHAPE, "a result may not take the place of an input (but next_slot of src_slot)");
  const bool vec = !misaligned(a->target_probs, 15) && a->target_row_stride % 4 == 0 &&
                   (!probs || (!misaligned(probs, 15) && a->draft_row_stride % 4 == 0));
  const Params p{a->N, a->T, a->V, a->draft_tokens, a->target_probs, probs, a->target_row_stride, a->draft_row_stride,
                 a->accept_u, a->sample_u, a->src_slot, a->slot_idx, a->tokens, a->num_accepted, a->next_slot, a->err_flag};
  // CTAs per sequence: as many as are resident at once (1024 threads an SM: two
  // of 512 threads while clusters of 8 of them fit, else four of 256), and on
  // batches past that so many more that a CTA keeps about 16,384 tokens, for
  // then sequences of unequal cost even out (256 x 131,072 tokens: 48 us with
  // four, 52 with two or eight; 256 x 50,000: 19 with two, 22 with four).
  const bool wide = static_cast<int64_t>(a->N) * kMaxCluster <= 2 * 152;
  int cluster = kMaxCluster;
  while (cluster > 1 && static_cast<int64_t>(a->N) * cluster > 4 * 152) cluster >>= 1;
  while (cluster < kMaxCluster && a->V / (2 * cluster) > 16384) cluster <<= 1;
  const int threads = wide ? 512 : 256, slices = cluster * (threads / 32);
  const int part = static_cast<int>((static_cast<int64_t>(a->V) + slices * 128LL - 1) / (slices * 128LL)) * 128;
  auto kernel = wide ? (vec ? verify_kernel<true, 512> : verify_kernel<false, 512>)
                     : (vec ? verify_kernel<true, 256> : verify_kernel<false, 256>);
  const cudaError_t e = kda_internal_launch_cluster(kernel, dim3(static_cast<unsigned>(a->N) * cluster), dim3(threads), 0,
                                                    stream, cluster, p, cluster, part);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
  return KDA_OK;
}
