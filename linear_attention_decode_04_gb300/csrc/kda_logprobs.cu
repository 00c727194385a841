// kda_logprobs.cu -- log probabilities of given tokens, entropy and likeliest
// alternatives (definition in include/kda_logprobs.h).
//
// One pass over the logits: every thread keeps the largest logit m of its
// elements, s = sum e^(x - m) and t = sum (x - m) e^(x - m), from which lse and
// entropy follow (lse = m + log s, entropy = log s - t / s), and counts the
// logits ahead of the given token's.  The top alternatives cost next to nothing
// in that pass: the num_top-th largest of the threads' largest elements bounds
// the num_top-th largest element from below, and only the threads whose largest
// element reaches it can hold one that does.  Those (at most num_top of a CTA)
// have their elements read once more, out of L2.
//
// Orders are those of 64-bit keys, the logit's bits in an order-preserving
// form above the complement of the index: keys differ, so ties go to the lower
// index and results do not depend on how a row was split.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_logprobs.h"

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxTop = KDA_LOGPROBS_MAX_TOP;
constexpr int kList = 1024;                // elements that a CTA lists as candidates
constexpr float kLog2e = 1.44269504088896340736f;

struct Params {
  int R, V, top;
  const void* logits;
  int64_t stride;
  const int32_t* tokens;
  float* logprobs;
  int32_t* ranks;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  int32_t* err;
};

// Sums of elements relative to their largest, m (see above); s and t are 0 where m is -infinity.
struct Sums {
  float m, s, t;
};
struct Shared {
  uint64_t keys[kWarps][32];
  uint64_t list[kList];
  uint64_t best[kMaxCluster][kMaxTop];     // every CTA's alternatives, in the cluster's first CTA
  Sums sums[kMaxCluster];
  int count[kMaxCluster];
  Sums warp_sums[kWarps];
  int warp_count[kWarps];
  int owner[kMaxTop];                      // threads whose elements are read again
  int owners, listed;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ Sums join(Sums a, Sums b) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  const float da = a.m == r.m ? 0.f : a.m - r.m, db = b.m == r.m ? 0.f : b.m - r.m;
  const float fa = ex2(da * kLog2e), fb = ex2(db * kLog2e);  // 0 from -infinity, where s and t are 0
  r.s = a.s * fa + b.s * fb;
  r.t = (a.t + fmaxf(da, -1e30f) * a.s) * fa + (b.t + fmaxf(db, -1e30f) * b.s) * fb;
  return r;
}
__device__ __forceinline__ Sums warp_join(Sums v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums w;
    w.m = __shfl_xor_sync(0xffffffffu, v.m, o);
    w.s = __shfl_xor_sync(0xffffffffu, v.s, o);
    w.t = __shfl_xor_sync(0xffffffffu, v.t, o);
    v = join(v, w);
  }
  return v;
}
__device__ __forceinline__ uint64_t key_of(float x, int i) {
  uint32_t b = __float_as_uint(x + 0.f);   // (-0 and 0 are equal)
  b ^= b >> 31 ? 0xffffffffu : 0x80000000u;
  return static_cast<uint64_t>(b) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float logit_of(uint64_t key) {
  uint32_t b = static_cast<uint32_t>(key >> 32);
  b ^= b >> 31 ? 0x80000000u : 0xffffffffu;
  return __uint_as_float(b);
}
__device__ __forceinline__ int index_of(uint64_t key) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)); }
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }
// One step of a bitonic network over the warp's lanes.
__device__ __forceinline__ uint64_t exchange(uint64_t v, int distance, bool descending, int lane) {
  const uint64_t w = __shfl_xor_sync(0xffffffffu, v, distance);
  return ((lane & distance) == 0) == descending ? max64(v, w) : (v < w ? v : w);
}
__device__ __forceinline__ uint64_t warp_sort(uint64_t v, int lane) {  // descending over the lanes
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int d = size / 2; d > 0; d >>= 1) v = exchange(v, d, (lane & size) == 0 || size == 32, lane);
  return v;
}
__device__ __forceinline__ uint64_t warp_merge(uint64_t a, uint64_t b_reversed, int lane) {  // the 32 largest of both
  uint64_t v = max64(a, b_reversed);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = exchange(v, d, true, lane);
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// The row as vectors of 16 bytes from the boundary at or below its start: vector
// j holds elements j * W - shift and on.
template <bool BF16>
struct Row {
  static constexpr int W = BF16 ? 8 : 4;
  const char* base;
  int shift, V;
  __device__ __forceinline__ Row(const Params& p, int r) {
    const char* at = static_cast<const char*>(p.logits) + static_cast<int64_t>(r) * p.stride * (16 / W);
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at)) & 15u;
    base = at - off;
    shift = static_cast<int>(off) / (16 / W);
    V = p.V;
  }
  __device__ __forceinline__ int vectors() const { return static_cast<int>((static_cast<int64_t>(V) + shift + W - 1) / W); }
  __device__ __forceinline__ float at(int i) const {
    if (BF16) return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(base)[shift + i]) << 16);
    return reinterpret_cast<const float*>(base)[shift + i];
  }
  __device__ __forceinline__ int first(int j) const { return j * W - shift; }
  __device__ __forceinline__ bool whole(int j) const { return first(j) >= 0 && first(j) + W <= V; }
  __device__ __forceinline__ uint4 load(int j) const { return reinterpret_cast<const uint4*>(base)[j]; }
  __device__ __forceinline__ static void values(uint4 u, float (&x)[W]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF16) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      else x[i] = __uint_as_float(w[i]);
    }
  }
};

// What a thread has seen: its sums, the first batch of vectors that held its
// largest element, and how many logits were ahead of the token's.
struct Seen {
  Sums sums{-INFINITY, 0.f, 0.f};
  int batch = -1;
  int ahead = 0;
};
constexpr int kBatch = 4;  // vectors

__device__ __forceinline__ void see_one(Seen& s, float x, int i, int batch, float given, int token) {
  if (x > s.sums.m) {
    s.sums = join(s.sums, Sums{x, 0.f, 0.f});
    s.batch = batch;
  } else if (s.batch < 0) {
    s.batch = batch;  // -infinity (or NaN) so far
  }
  const float d = x - (s.sums.m == -INFINITY ? 0.f : s.sums.m), e = ex2(d * kLog2e);
  s.sums.s += e;
  s.sums.t = fmaf(fmaxf(d, -1e30f), e, s.sums.t);
  s.ahead += x > given || (x == given && i < token);
}
template <int N>
__device__ __forceinline__ void see(Seen& s, const float (&x)[N], int batch) {
  float top = x[0];
#pragma unroll
  for (int k = 1; k < N; ++k) top = fmaxf(top, x[k]);
  if (top > s.sums.m) {
    s.sums = join(s.sums, Sums{top, 0.f, 0.f});
    s.batch = batch;
  } else if (s.batch < 0) {
    s.batch = batch;
  }
  const float ref = s.sums.m == -INFINITY ? 0.f : s.sums.m;
  float sum = 0.f, weighted = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float d = x[k] - ref, e = ex2(d * kLog2e);
    sum += e;
    weighted = fmaf(fmaxf(d, -1e30f), e, weighted);
  }
  s.sums.s += sum;
  s.sums.t += weighted;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const Params p, int cluster) {
  using Row = Row<BF16>;
  constexpr int W = Row::W;
  __shared__ Shared S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / cluster, rank = blockIdx.x - r * cluster;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int token = p.tokens ? p.tokens[r] : 0;
  if (token < 0 || token >= p.V) {  // not asked for; the whole cluster leaves here
    if (rank == 0) {
      if (tid == 0) {
        p.logprobs[r] = 0.f, p.ranks[r] = -1, p.entropy[r] = 0.f;
        if (token >= p.V && p.err) atomicOr(p.err, KDA_DEVERR_TOKEN_RANGE);
      }
      if (tid < p.top) p.top_ids[static_cast<int64_t>(r) * p.top + tid] = -1, p.top_logprobs[static_cast<int64_t>(r) * p.top + tid] = 0.f;
    }
    return;
  }
  const Row row(p, r);
  const float given = p.tokens ? row.at(token) : INFINITY;
  if (tid == 0) S.owners = S.listed = 0;
  // this CTA's vectors: whole batches of all threads, so that a thread's elements are easily found again
  const int vectors = row.vectors(), per_batch = kThreads * kBatch;
  const int batches = static_cast<int>((vectors + static_cast<int64_t>(per_batch) * cluster - 1) / (static_cast<int64_t>(per_batch) * cluster));
  const int64_t begin64 = static_cast<int64_t>(rank) * batches * per_batch;
  const int begin = static_cast<int>(begin64 < vectors ? begin64 : vectors);
  const int end = static_cast<int>(begin64 + static_cast<int64_t>(batches) * per_batch < vectors ? begin64 + static_cast<int64_t>(batches) * per_batch : vectors);
  // vector k of batch b of a thread
  auto vector_of = [&](int thread, int b, int k) { return begin + (b * kBatch + k) * kThreads + thread; };
  Seen seen;
  for (int b = 0; b < batches; ++b) {
    if (vector_of(0, b, 0) >= end) break;
    const int j0 = vector_of(tid, b, 0), j1 = vector_of(tid, b, kBatch - 1);
    if (row.first(j0) >= 0 && j1 < end && row.first(j1) + W <= row.V) {
      uint4 u[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) u[k] = row.load(vector_of(tid, b, k));
      float x[kBatch * W];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        float y[W];
        Row::values(u[k], y);
        const int i0 = row.first(vector_of(tid, b, k));
#pragma unroll
        for (int e = 0; e < W; ++e) {
          x[k * W + e] = y[e];
          seen.ahead += y[e] > given || (y[e] == given && i0 + e < token);
        }
      }
      see(seen, x, b);
    } else {
      for (int k = 0; k < kBatch; ++k) {
        const int j = vector_of(tid, b, k);
        if (j >= end) break;
        for (int e = 0; e < W; ++e) {
          const int i = row.first(j) + e;
          if (i >= 0 && i < row.V) see_one(seen, row.at(i), i, b, given, token);
        }
      }
    }
  }
  // ---- the CTA's sums
  {
    const Sums w = warp_join(seen.sums);
    const int n = __reduce_add_sync(0xffffffffu, seen.ahead);
    if (lane == 0) S.warp_sums[warp] = w, S.warp_count[warp] = n;
  }
  // ---- the bound: the top-th largest of the threads' largest elements
  uint64_t mine = 0;
  if (p.top > 0) {
    if (seen.batch >= 0) {
      const float m = seen.sums.m;
      int at = -1;
      for (int k = 0; k < kBatch && at < 0; ++k) {
        const int j = vector_of(tid, seen.batch, k);
        if (j >= end) break;
        for (int e = 0; e < W; ++e) {
          const int i = row.first(j) + e;
          if (at < 0 && i >= 0 && i < row.V && row.at(i) == m) at = i;
        }
      }
      if (at >= 0) mine = key_of(m, at);  // (none where every element is NaN: such a row has no result)
    }
    uint64_t v = warp_sort(mine, lane);
    S.keys[warp][lane] = v;
    __syncthreads();
#pragma unroll
    for (int half = kWarps / 2; half > 0; half >>= 1) {
      if (warp < half) {
        v = warp_merge(v, S.keys[warp + half][31 - lane], lane);
        S.keys[warp][lane] = v;
      }
      __syncthreads();
    }
    const uint64_t bound = S.keys[0][p.top - 1];
    if (mine != 0 && mine >= bound) S.owner[atomicAdd(&S.owners, 1)] = tid;
    __syncthreads();
    // ---- the elements at or above it, of the threads that can have any
    const int owners = S.owners;
    auto scan = [&](auto f) {  // f(key) for the owners' elements, a warp per owner and lanes over its batches' vectors
      for (int o = warp; o < owners; o += kWarps) {
        const int thread = S.owner[o];
        for (int q = lane; q < batches * kBatch; q += 32) {
          const int j = vector_of(thread, q / kBatch, q % kBatch);
          if (j >= end) continue;
          for (int e = 0; e < W; ++e) {
            const int i = row.first(j) + e;
            if (i >= 0 && i < row.V) {
              const float x = row.at(i);
              if (x == x) f(key_of(x, i));
            }
          }
        }
      }
    };
    scan([&](uint64_t key) {
      if (key >= bound) {
        const int n = atomicAdd(&S.listed, 1);
        if (n < kList) S.list[n] = key;
      }
    });
    __syncthreads();
    uint64_t* best = S.best[rank];
    if (S.listed <= kList) {
      const int n = S.listed;
      if (tid < p.top && tid >= n) best[tid] = 0;
      for (int c = tid; c < n; c += kThreads) {
        const uint64_t key = S.list[c];
        int ahead = 0;
        for (int k = 0; k < n; ++k) ahead += S.list[k] > key;
        if (ahead < p.top) best[ahead] = key;
      }
    } else {
      // many elements of few threads reach the bound (rows in order, say): one alternative after another
      uint64_t last = ~0ull;
      for (int n = 0; n < p.top; ++n) {
        uint64_t top = 0;
        scan([&](uint64_t key) {
          if (key < last) top = max64(top, key);
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = max64(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) S.keys[0][warp] = top;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) top = max64(top, S.keys[0][w]);
        if (tid == 0) best[n] = top;
        last = top;
        __syncthreads();
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    Sums w = lane < kWarps ? S.warp_sums[lane] : Sums{-INFINITY, 0.f, 0.f};
    w = warp_join(w);
    const int n = __reduce_add_sync(0xffffffffu, lane < kWarps ? S.warp_count[lane] : 0);
    if (lane == 0) S.sums[rank] = w, S.count[rank] = n;
  }
  if (cluster > 1) {
    __syncthreads();
    cluster_barrier();  // every CTA has its results
    if (rank == 0) {
      auto remote = [&](const void* at, int cta) {
        uint32_t a;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(at))), "r"(cta));
        return a;
      };
      for (int c = 1 + warp; c < cluster; c += kWarps) {
        if (lane < p.top) {
          uint64_t v;
          asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(&S.best[c][lane], c)) : "memory");
          S.best[c][lane] = v;
        }
        if (lane < 4) {
          const void* at = lane == 0 ? static_cast<const void*>(&S.sums[c].m) : lane == 1 ? &S.sums[c].s : lane == 2 ? &S.sums[c].t : static_cast<const void*>(&S.count[c]);
          uint32_t v;
          asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(at, c)) : "memory");
          *const_cast<uint32_t*>(static_cast<const uint32_t*>(at)) = v;
        }
      }
    }
    cluster_barrier();  // read: the others may leave
    if (rank != 0) return;
  }
  __syncthreads();
  // ---- the row's results
  Sums all{-INFINITY, 0.f, 0.f};
  int ahead = 0;
  for (int c = 0; c < cluster; ++c) all = join(all, S.sums[c]), ahead += S.count[c];
  const bool good = all.s > 0.f && all.s < INFINITY && all.m < INFINITY;
  const float nan = __uint_as_float(0x7fc00000u), logs = logf(all.s);
  if (tid == 0) {
    p.entropy[r] = good ? logs - all.t / all.s : nan;
    if (p.tokens) {
      p.logprobs[r] = good ? given - all.m - logs : nan;
      p.ranks[r] = good ? ahead : -1;
    }
  }
  const int n = cluster * p.top;
  for (int c = tid; c < n; c += kThreads) {
    const uint64_t key = S.best[c / p.top][c % p.top];
    int place = 0;  // keys differ but for the zeros past a CTA's last element
    for (int k = 0; k < n; ++k) {
      const uint64_t other = S.best[k / p.top][k % p.top];
      place += other > key || (other == key && k < c);
    }
    if (place < p.top) {
      const int64_t at = static_cast<int64_t>(r) * p.top + place;
      p.top_ids[at] = good && key ? index_of(key) : -1;
      p.top_logprobs[at] = !good ? nan : key ? logit_of(key) - all.m - logs : -INFINITY;
    }
  }
}

bool misaligned(const void* ptr, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(ptr) & mask) != 0; }

}  // namespace

extern "C" int kda_logprobs(const KdaLogprobsArgs* a, void* stream) {
  kda_internal_clear_error();
  if (!a) return kda_internal_fail(KDA_ERR_NULLPTR, "args is NULL");
  if (a->struct_size != sizeof(KdaLogprobsArgs))
    return kda_internal_fail(KDA_ERR_ABI, "struct_size %u, library expects %zu", a->struct_size, sizeof(KdaLogprobsArgs));
  if (a->flags & ~KDA_LOGPROBS_BF16) return kda_internal_fail(KDA_ERR_FLAGS, "unknown flags 0x%x", a->flags);
  if (a->R < 0 || a->R > 0x7fffffff / kMaxCluster || a->V < 1 || a->V > (1 << 30) || a->num_top < 0 ||
      a->num_top > kMaxTop || (a->R > 0 && a->logits_row_stride < a->V))
    return kda_internal_fail(KDA_ERR_SHAPE, "R=%d V=%d num_top=%d row stride %lld", a->R, a->V, a->num_top,
                             static_cast<long long>(a->logits_row_stride));
  if (a->R == 0) return KDA_OK;
  if (!a->logits || !a->entropy || (a->tokens != nullptr) != (a->logprobs != nullptr) ||
      (a->tokens != nullptr) != (a->ranks != nullptr) || (a->num_top > 0 && (!a->top_ids || !a->top_logprobs)))
    return kda_internal_fail(KDA_ERR_NULLPTR, "a required pointer is NULL (tokens, logprobs and ranks go together)");
  const bool bf16 = a->flags & KDA_LOGPROBS_BF16;
  if (misaligned(a->logits, bf16 ? 1 : 3) || misaligned(a->tokens, 3) || misaligned(a->logprobs, 3) ||
      misaligned(a->ranks, 3) || misaligned(a->entropy, 3) || misaligned(a->top_ids, 3) ||
      misaligned(a->top_logprobs, 3) || misaligned(a->err_flag, 3))
    return kda_internal_fail(KDA_ERR_ALIGN, "a pointer is not aligned as required");
  if (a->tokens && (a->tokens == a->ranks || a->tokens == a->top_ids || static_cast<const void*>(a->tokens) == a->logprobs ||
                    static_cast<const void*>(a->tokens) == a->entropy))
    return kda_internal_fail(KDA_ERR_SHAPE, "a result may not take the place of the tokens");
  const Params p{a->R, a->V, a->num_top, a->logits, a->logits_row_stride, a->tokens, a->logprobs, a->ranks, a->entropy,
                 a->top_ids, a->top_logprobs, a->err_flag};
  // CTAs per row: as many as are resident at once (four an SM)
  int cluster = kMaxCluster;
  while (cluster > 1 && static_cast<int64_t>(a->R) * cluster > 4 * 152) cluster >>= 1;
  const cudaError_t e = kda_internal_launch_cluster(bf16 ? logprobs_kernel<true> : logprobs_kernel<false>,
                                                    dim3(static_cast<unsigned>(a->R) * cluster), dim3(kThreads), 0, stream,
                                                    cluster, p, cluster);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
  return KDA_OK;
}
