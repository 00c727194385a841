// kda_logprobs.cu -- log probabilities of given tokens, entropy and likeliest
// alternatives (definition in include/kda_logprobs.h).
//
// One pass over the logits, which a warp of its own copies to shared memory in a
// ring: every thread keeps s = sum 2^y and t = sum y 2^y with y = x log2 e - c and c =
// m log2 e as rounded for an m near its largest logit (it follows in steps of 16, for
// most batches have a new largest in some lane), from which lse and entropy follow (lse
// = ln 2 (c + log2 s), entropy = ln 2 (log2 s - t / s)).  y is one
// fused operation, so neither c's rounding nor a large logit costs digits.  The top
// alternatives cost little beside that pass: the num_top-th largest of the threads'
// largest logits bounds the num_top-th largest logit from below, and of a thread's
// elements, in two halves, only those can reach it whose half's largest does.  The
// threads know where that one is and what comes next in the half, so that some num_top
// pieces of 32 bytes are read once more; the whole half only where two of its pieces
// reach the bound.
//
// What bounds it: many fp32 rows HBM (1,000 rows of 131,072 94 us, 5.5 TB/s), bf16
// rows the issue of 19 instructions per element, 80% of all slots (4,099 rows of
// 100,003 198 us, 4.1 TB/s), few rows the launch, a CTA's share of the row and the
// join (one row of 131,072 7.4 to 7.9 us).  Rows of one value, whose elements all
// reach the bound, take two to three times as long.
//
// Orders are those of 64-bit keys, the logit's bits in an order-preserving form
// above the complement of the index: keys differ, so ties go to the lower index and
// results do not depend on how a row was split.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "kda_internal.h"
#include "kda_logprobs.h"
#include "kda_tc.cuh"

namespace {

constexpr int kVecs = 4;                   // 16-byte pieces of a stage, per thread
constexpr int kStages = 3;
constexpr int kHalves = 2;                 // of a thread's elements, by their place in a batch
constexpr int kMaxCluster = 8;
constexpr int kMaxTop = KDA_LOGPROBS_MAX_TOP;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kLeast = -200.f;           // of y: 2^y is 0 in fp32 from -150 on, and y 2^y is too where x is -infinity
constexpr float kStep = 16.f;              // a reference follows a logit that is further above it
constexpr float kFar = 1e7f;               // from here on m log2 e is rounded by whole numbers: elements are taken relative to m itself

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

// Sums of elements relative to one of them, m, which no other is more than kStep above; s and t are 0 where m is
// -infinity.
struct Sums {
  float m, s, t;
};
// THREADS that sum, and a warp that copies.
template <int THREADS>
struct Cfg {
  static constexpr int kThreads = THREADS, kWarps = THREADS / 32, kAllThreads = THREADS + 32;
  static constexpr int kStageBytes = kThreads * kVecs * 16;
  static constexpr int kCtasPerSm = THREADS > 128 ? 4 : 12;
  static constexpr int kList = 4 * THREADS;  // elements that a CTA lists as candidates
};
template <class C>
struct Shared {
  static constexpr int kThreads = C::kThreads, kWarps = C::kWarps, kList = C::kList;
  union {
    alignas(128) uint8_t stage[kStages][C::kStageBytes];
    struct {                               // when the row has been seen
      uint64_t list[kList];
      int spot[kThreads * kHalves];        // pieces that are read again: the first vector of each
      int16_t half[kThreads * kHalves];    // halves that are
    };
  };
  uint64_t full[kStages], empty[kStages];
  uint64_t best[kMaxTop];
  uint64_t round[kWarps + 1];
  Sums warp_sums[kWarps];
  int warp_count[kWarps];
  uint32_t warp_bound[kWarps];
  int found[2][kWarps + 1];
  int spots, halves, listed, none, failed;
  // in a cluster's first CTA: what every CTA has of the row
  uint64_t part_top[kMaxCluster][kMaxTop];
  Sums part_sums[kMaxCluster];
  int part_count[kMaxCluster];
};

__device__ __forceinline__ float one_from(float x, float limit) {  // 1 where x >= limit, else 0
  float r;
  asm("set.ge.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(limit));
  return r;
}
__device__ __forceinline__ float float_above(float x) {  // the next higher float; NaN, which nothing reaches, of infinity
  const int b = __float_as_int(x + 0.f);
  return __int_as_float(b >= 0 ? b + 1 : b - 1);
}
__device__ __forceinline__ float at_least(float y) {  // NaN stays NaN
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(y), "f"(kLeast));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Sums of reference m are relative to c = m log2 e as rounded where |m| < kFar, to m log2 e itself further out, to 0
// where there is nothing.  (c is rounded wherever it is used: fused into a difference it would be another one.)
__device__ __forceinline__ bool is_near(float m) { return fabsf(m) < kFar || m == -INFINITY; }
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.f : __fmul_rn(m, kLog2e); }
// log2 of an element relative to that, and of m itself.
__device__ __forceinline__ float relative(float x, float m) { return is_near(m) ? fmaf(x, kLog2e, -reference(m)) : (x - m) * kLog2e; }
__device__ __forceinline__ float residue(float m) { return fabsf(m) < kFar ? fmaf(m, kLog2e, -reference(m)) : 0.f; }
// The exponent that takes sums from reference m to reference `to` >= m.
__device__ __forceinline__ float shift(float m, float to) {
  if (m == to) return 0.f;
  return m > -INFINITY ? fmaxf(fmaf(m - to, kLog2e, residue(to) - residue(m)), kLeast) : kLeast;
}
__device__ __forceinline__ Sums scaled(Sums a, float to) {
  const float y = shift(a.m, to), f = ex2(y);
  return Sums{to, a.s * f, (a.t + y * a.s) * f};
}
// Over the warp's lanes, in all of them.
__device__ __forceinline__ Sums warp_sum(Sums v) {
  float m = v.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  v = scaled(v, m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.s += __shfl_xor_sync(0xffffffffu, v.s, o);
    v.t += __shfl_xor_sync(0xffffffffu, v.t, o);
  }
  return v;
}
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // (-0 and 0 are equal)
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(float x, int i) {
  return static_cast<uint64_t>(order_of(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float logit_of(uint64_t key) {
  uint32_t b = static_cast<uint32_t>(key >> 32);
  b ^= b >> 31 ? 0x80000000u : 0xffffffffu;
  return __uint_as_float(b);
}
__device__ __forceinline__ int index_of(uint64_t key) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)); }
// A row: `head` elements up to the first 16-byte boundary, whole vectors of W, and
// `tail` elements.
template <bool BF16>
struct Row {
  static constexpr int W = BF16 ? 8 : 4;
  const char* base;  // of the row
  int V, head, vectors, tail;
  __device__ __forceinline__ Row(const Params& p, int r) : V(p.V) {
    base = static_cast<const char*>(p.logits) + static_cast<int64_t>(r) * p.stride * (16 / W);
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(base) & 15u);
    head = min(off ? (16 - off) / (16 / W) : 0, V);
    vectors = (V - head) / W;
    tail = V - head - vectors * W;
  }
  __device__ __forceinline__ float at(int i) const {
    if (BF16) return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(base)[i]) << 16);
    return reinterpret_cast<const float*>(base)[i];
  }
  __device__ __forceinline__ int first(int j) const { return head + j * W; }  // element of vector j
  __device__ __forceinline__ const char* vector(int j) const { return base + static_cast<int64_t>(head) * (16 / W) + static_cast<int64_t>(j) * 16; }
  // the element of the row's ends that a thread of the first CTA has, or -1: those of the head, then those of the tail
  __device__ __forceinline__ int edge(int thread) const {
    return thread < head ? thread : thread < head + tail ? V - tail + thread - head : -1;
  }
  __device__ __forceinline__ static void values(uint4 u, float (&x)[W]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF16) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      else x[i] = __uint_as_float(w[i]);
    }
  }
};

// Fewer alternatives than asked for: the first elements equal to the bound, and where fewer are above -infinity the first of
// those that are not, which most are.  For all threads of the CTA.
template <bool BF16, class C>
__device__ __forceinline__ void first_equal(Shared<C>& S, int tid, int warp, int lane, const Row<BF16>& row, int begin, int end,
                                            bool ends, int have, int top, float next) {
  constexpr int W = Row<BF16>::W;
  const int head = ends ? row.head : 0, last = head + (end - begin) * W, count = ends ? last + row.tail : last;
  int turn = 0;
  for (;; next = -INFINITY) {
    for (int q0 = 0; q0 < count && have < top; q0 += C::kAllThreads, turn ^= 1) {  // head, slice, tail
      const int q = q0 + tid, i = q < head ? q : q < last ? row.first(begin) + q - head : q < count ? row.V - row.tail + q - last : -1;
      const bool here = i >= 0 && row.at(i) == next;
      const uint32_t found = __ballot_sync(0xffffffffu, here);
      if (lane == 0) S.found[turn][warp] = __popc(found);
      __syncthreads();
      int place = have + __popc(found & ((1u << lane) - 1));
      for (int w = 0; w <= C::kWarps; ++w) {
        if (w < warp) place += S.found[turn][w];
        have += S.found[turn][w];
      }
      if (here && place < top) S.best[place] = key_of(next, i);
    }
    if (next == -INFINITY) return;
  }
}

// For fp32 rows a call, as it is seldom needed (64 x 4 rows of 131,072 35.7 us, inlined 36.2); in bf16 rows the call costs the
// sums registers (4,099 rows of 100,003 242 us, inlined 238).
template <class C>
__device__ __noinline__ void first_equal_f32(Shared<C>& S, Row<false> row, int begin, int end, bool ends, int have, int top, float next) {
  first_equal<false>(S, threadIdx.x, threadIdx.x >> 5, threadIdx.x & 31, row, begin, end, ends, have, top, next);
}

template <bool BF16, int THREADS>
__global__ void __launch_bounds__(Cfg<THREADS>::kAllThreads, Cfg<THREADS>::kCtasPerSm) logprobs_kernel(const Params p, int cluster) {
  using C = Cfg<THREADS>;
  constexpr int kThreads = C::kThreads, kWarps = C::kWarps, kAllThreads = C::kAllThreads, kList = C::kList;
  using Row = Row<BF16>;
  constexpr int W = Row::W;
  constexpr int kStageVecs = kThreads * kVecs;
  constexpr int kBatch = 16 / W, kHalf = kBatch / kHalves;  // vectors of 16 elements, of half of them
  constexpr int kBatches = kVecs / kBatch;                   // of a stage, per thread
  extern __shared__ __align__(128) uint8_t raw[];
  Shared<C>& S = *reinterpret_cast<Shared<C>*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int r = blockIdx.x / cluster, rank = blockIdx.x - r * cluster;
  if (tid == kThreads) {
    for (int i = 0; i < kStages; ++i) bar_init(&S.full[i], 1), bar_init(&S.empty[i], kWarps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 0) S.spots = S.halves = S.listed = S.none = S.failed = 0;
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
  // this CTA's vectors: whole stages, the last of the row's perhaps short
  const int64_t stages_all = (static_cast<int64_t>(row.vectors) + kStageVecs - 1) / kStageVecs;
  const int64_t stages = (stages_all + cluster - 1) / cluster;
  const int begin = static_cast<int>(min(rank * stages * kStageVecs, static_cast<int64_t>(row.vectors)));
  const int end = static_cast<int>(min((rank + 1) * stages * kStageVecs, static_cast<int64_t>(row.vectors)));
  const int fills = (end - begin + kStageVecs - 1) / kStageVecs;  // stages that hold any
  __syncthreads();
  if (cluster > 1) cluster_arrive();  // a CTA's memory may be written once it has arrived here
  const float given = p.tokens ? row.at(token) : INFINITY;
  Sums mine{-INFINITY, 0.f, 0.f};
  int ahead = 0;
  // of each half: the largest element, the batch that it is in, and the largest of the other batches
  float largest[kHalves] = {-INFINITY, -INFINITY}, second[kHalves] = {-INFINITY, -INFINITY};
  int at[kHalves] = {0, 0};
  const int edge = rank == 0 ? row.edge(tid) : -1;
  const float edge_x = edge >= 0 ? row.at(edge) : -INFINITY;
  if (warp == kWarps) {
    // ================================================================== copies
    bool ok = true;
    int b = 0;
    for (; b < fills; ++b) {
      const int st = b % kStages;
      if (b >= kStages) ok = warp_wait(&S.empty[st], (b / kStages - 1) & 1, &S.failed);
      if (!ok) break;
      if (elect()) {
        const int from = begin + b * kStageVecs, n = min(kStageVecs, end - from) * 16;
        bar_expect(&S.full[st], n);
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(s32(S.stage[st])),
                     "l"(row.vector(from)), "r"(n), "r"(s32(&S.full[st]))
                     : "memory");
      }
      __syncwarp();
    }
    // nothing may land in shared memory after the CTA is gone, whoever gave up
    if (lane == 0)
      for (int j = b > kStages ? b - kStages : 0; j < b; ++j) bar_drain(&S.full[j % kStages], (j / kStages) & 1);
    __syncwarp();
  } else {
    // ==================================================================== sums
    float c = 0.f;  // the reference
    bool near = true;
    const float above = float_above(given);
    // 16 elements: the largest of their halves, then their sums
    auto see = [&](const uint64_t (&x)[8], int batch, auto index) {
      float top[kHalves];
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        top[h] = max3(fmaxf(both(x[4 * h]).x, both(x[4 * h]).y), both(x[4 * h + 1]).x, both(x[4 * h + 1]).y);
        top[h] = max3(max3(top[h], both(x[4 * h + 2]).x, both(x[4 * h + 2]).y), both(x[4 * h + 3]).x, both(x[4 * h + 3]).y);
        second[h] = fmaxf(second[h], fminf(top[h], largest[h]));
        if (top[h] > largest[h]) largest[h] = top[h], at[h] = batch;
      }
      const float most = fmaxf(top[0], top[1]);
      if (most > mine.m + kStep) {
        mine = scaled(mine, most);
        c = reference(most);
        near = is_near(most);
      }
      // logits ahead of the given one: x >= given of tokens of a lower index, x >= the float above it of others.
      // (A token drawn from the row has hundreds ahead of it: many warps have one among a few hundred elements.)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        if (top[h] >= given) {
#pragma unroll
          for (int k = 0; k < kHalf; ++k) {
            const int i = index(h * kHalf + k);  // of the vector's first element
            const float from = i + W <= token ? given : above;
            uint64_t n = 0;
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
              const float2 v = both(x[(h * kHalf + k) * (W / 2) + e]);
              n = add2(n, pair_of(one_from(v.x, from), one_from(v.y, from)));
              if (i < token && token < i + W) {  // (the token's own vector: equal ones ahead of it)
                ahead += v.x == given && i + 2 * e < token;
                ahead += v.y == given && i + 2 * e + 1 < token;
              }
            }
            ahead += static_cast<int>(both(n).x + both(n).y);
          }
        }
      }
      const uint64_t log2e = pair_of(kLog2e, kLog2e), c2 = pair_of(-c, -c);
      uint64_t s[2] = {0, 0}, t[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint64_t y = fma2(x[k], log2e, c2), e = pair_of(ex2(both(y).x), ex2(both(y).y));
        s[k & 1] = add2(s[k & 1], e);
        t[k & 1] = fma2(y, e, t[k & 1]);
      }
      float2 s2 = both(add2(s[0], s[1])), t2 = both(add2(t[0], t[1]));
      // y 2^y is NaN where y is -infinity (ruled out, or that far below), and y is not y where the reference is far out:
      // once more, with care
      if (!(t2.x + t2.y == t2.x + t2.y) || !near) {
        s2 = t2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float y0 = at_least(relative(both(x[k]).x, mine.m)), y1 = at_least(relative(both(x[k]).y, mine.m));
          const float e0 = ex2(y0), e1 = ex2(y1);
          s2.x += e0, s2.y += e1;
          t2.x = fmaf(y0, e0, t2.x), t2.y = fmaf(y1, e1, t2.y);
        }
      }
      mine.s += s2.x + s2.y;
      mine.t += t2.x + t2.y;
    };
    for (int b = 0; b < fills; ++b) {
      const int st = b % kStages, from = begin + b * kStageVecs;
      bar_wait(&S.full[st], (b / kStages) & 1, &S.failed);
      uint4 u[kVecs];
      const uint4* const in = reinterpret_cast<const uint4*>(S.stage[st]) + tid;
#pragma unroll
      for (int k = 0; k < kVecs; ++k) u[k] = in[k * kThreads];
      const int left = end - from - tid;  // vectors of the slice from this thread's first on
      if (left <= (kVecs - 1) * kThreads) {
        const uint32_t out = BF16 ? 0xff80ff80u : 0xff800000u;  // -infinity: not there
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
          if (k * kThreads >= left) u[k] = make_uint4(out, out, out, out);
      }
#pragma unroll
      for (int k0 = 0; k0 < kVecs; k0 += kBatch) {
        uint64_t x[8];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          float v[W];
          Row::values(u[k0 + k], v);
#pragma unroll
          for (int i = 0; i < W / 2; ++i) x[k * (W / 2) + i] = pair_of(v[2 * i], v[2 * i + 1]);
        }
        // (what is not there counts for nothing even where the token itself is ruled out: its index is past the row's)
        see(x, b * kBatches + k0 / kBatch, [&](int k) { const int j = from + (k0 + k) * kThreads + tid; return j < end ? row.first(j) : 0x7fffff00; });
      }
      // (Only now: every lane's pieces have arrived in its registers, as they have been used.  An arrival right behind the
      // loads let copies overtake some of them.)
      __syncwarp();
      if (lane == 0) bar_arrive(&S.empty[st]);
    }
    if (edge >= 0) {
      if (edge_x > mine.m + kStep) mine = scaled(mine, edge_x);
      const float y = at_least(relative(edge_x, mine.m)), e = ex2(y);
      mine.s += e;
      mine.t += y * e;
      ahead += edge_x > given || (edge_x == given && edge < token);
    }
    // ---- the warp's sums, and its share of the bound: each warp has so many threads whose largest elements reach its own
    // bound that there are num_top of all warps, as many of it as it has of the threads with elements (the first, and
    // all of them but in short rows); so num_top elements reach the least of the warps' bounds
    const Sums w = warp_sum(mine);
    const int n = __reduce_add_sync(0xffffffffu, ahead);
    uint32_t left = order_of(fmaxf(fmaxf(largest[0], largest[1]), edge >= 0 ? edge_x : -INFINITY)), bound = 0;
    const int all = min(end - begin, kThreads), own = min(max(all - 32 * warp, 0), 32);
    if (p.top <= all) {  // (else everything passes)
      bound = 0xffffffffu;  // (of no concern where the warp has none)
      for (int k = 0; k < (p.top * own + all - 1) / all; ++k) {
        bound = __reduce_max_sync(0xffffffffu, left);
        if (lane == __ffs(__ballot_sync(0xffffffffu, left == bound)) - 1) left = 0;
      }
    }
    if (lane == 0) S.warp_sums[warp] = w, S.warp_count[warp] = n, S.warp_bound[warp] = bound;
    if (lane == 0 && (!(w.s < INFINITY) || w.m == INFINITY)) S.none = 1;
  }
  __syncthreads();
  if (tid == 0 && S.failed && p.err) atomicOr(p.err, KDA_DEVERR_TIMEOUT);
  if (S.none) {  // a row with NaN or +infinity is no distribution, and has no alternatives (all of it may reach the bound)
    if (tid < kMaxTop) S.best[tid] = 0;
  } else if (p.top > 0) {
    uint32_t bound = S.warp_bound[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) bound = min(bound, S.warp_bound[w]);
    // (-infinity, which threads without elements have too, is left to the end: it would let all ruled-out tokens pass)
    const float least = bound <= order_of(-3.4028235e38f) ? -3.4028235e38f : logit_of(static_cast<uint64_t>(bound) << 32);
    if (warp < kWarps) {
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        if (second[h] >= least) S.half[atomicAdd(&S.halves, 1)] = static_cast<int16_t>(h * kThreads + tid);
        else if (largest[h] >= least) S.spot[atomicAdd(&S.spots, 1)] = begin + (at[h] * kBatch + h * kHalf) * kThreads + tid;
      }
    }
    auto list = [&](uint64_t key) {
      const int n = atomicAdd(&S.listed, 1);
      if (n < kList) S.list[n] = key;
    };
    __syncthreads();
    // ---- the elements at or above it.  Where many threads have two, or they are more than the list takes, most are equal to
    // it (a row of one value, say): then those above it, and the first of the others.
    bool ties = S.halves > kThreads / 2;
    const int spots = S.spots * kHalf, vecs = fills * kBatches * kHalf, all = spots + S.halves * vecs;  // vectors; of a half
    auto scan = [&](float low, auto f) {  // f(key) for those from a value on
      constexpr int kAhead = 4;
      for (int q0 = tid; q0 < all; q0 += kAhead * kAllThreads) {
        uint4 u[kAhead];
        int where[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const int q = q0 + a * kAllThreads;
          where[a] = end;
          if (q < spots) {
            where[a] = S.spot[q / kHalf] + q % kHalf * kThreads;
          } else if (q < all) {
            const int o = (q - spots) / vecs, k = q - spots - o * vecs, who = S.half[o];
            where[a] = begin + (k / kHalf * kBatch + who / kThreads * kHalf + k % kHalf) * kThreads + who % kThreads;
          }
          if (where[a] < end) u[a] = *reinterpret_cast<const uint4*>(row.vector(where[a]));
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          if (where[a] >= end) continue;
          float x[W], top = -INFINITY;
          Row::values(u[a], x);
#pragma unroll
          for (int e = 0; e < W; ++e) top = fmaxf(top, x[e]);
          if (top >= low) {
#pragma unroll
            for (int e = 0; e < W; ++e)
              if (x[e] >= low) f(key_of(x[e], row.first(where[a]) + e));
          }
        }
      }
    };
    int n;
    for (;; ties = true) {
      const float from = ties ? float_above(least) : least;
      if (edge >= 0 && edge_x >= from) list(key_of(edge_x, edge));
      scan(from, list);
      __syncthreads();
      n = S.listed;
      if (n <= kList || ties) break;
      __syncthreads();
      if (tid == 0) S.listed = 0;
      __syncthreads();
    }
    if (n <= kList) {
      if (tid < p.top && tid >= n) S.best[tid] = 0;
      for (int c = tid; c < n; c += kAllThreads) {
        const uint64_t key = S.list[c];
        int before = 0;
#pragma unroll 4
        for (int k = 0; k < n; ++k) before += S.list[k] > key;
        if (before < p.top) S.best[before] = key;
      }
      if constexpr (BF16) first_equal<true>(S, tid, warp, lane, row, begin, end, rank == 0, n, p.top, ties ? least : -INFINITY);
      else if (n < p.top) first_equal_f32(S, row, begin, end, rank == 0, n, p.top, ties ? least : -INFINITY);
    } else {
      // many elements of few threads reach the bound (rows in order, say): one alternative after another
      uint64_t last = ~0ull;
      for (int k = 0; k < p.top; ++k) {
        uint64_t top = 0;
        auto below = [&](uint64_t key) {
          if (key < last && key > top) top = key;
        };
        scan(least, below);
        if (edge >= 0 && edge_x >= least) below(key_of(edge_x, edge));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const uint64_t other = __shfl_xor_sync(0xffffffffu, top, o);
          if (other > top) top = other;
        }
        if (lane == 0) S.round[warp] = top;
        __syncthreads();
        for (int w = 0; w <= kWarps; ++w)
          if (S.round[w] > top) top = S.round[w];
        if (tid == 0) S.best[k] = top;
        last = top;
        __syncthreads();
      }
    }
    __syncthreads();
  }
  if (warp != 0) {  // the rest is one warp's
    if (cluster > 1) {
      cluster_wait();
      cluster_arrive();
      cluster_wait();
    }
    return;
  }
  Sums all = warp_sum(lane < kWarps ? S.warp_sums[lane] : Sums{-INFINITY, 0.f, 0.f});
  int before = __reduce_add_sync(0xffffffffu, lane < kWarps ? S.warp_count[lane] : 0);
  uint64_t key = lane < p.top ? S.best[lane] : 0;
  if (cluster > 1) {  // to the cluster's first CTA
    cluster_wait();
    if (lane < p.top) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_cta(&S.part_top[rank][lane], 0)), "l"(key) : "memory");
    if (lane == 0) {
      const uint32_t to = in_cta(&S.part_sums[rank], 0);
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(all.m) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4), "f"(all.s) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 8), "f"(all.t) : "memory");
      asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(in_cta(&S.part_count[rank], 0)), "r"(before) : "memory");
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    all = warp_sum(lane < cluster ? S.part_sums[lane] : Sums{-INFINITY, 0.f, 0.f});
    before = __reduce_add_sync(0xffffffffu, lane < cluster ? S.part_count[lane] : 0);
    // of all CTAs' alternatives, each list in order: one after another the largest of the lists' heads
    int next = 0;
    for (int k = 0; k < p.top; ++k) {
      const uint64_t head = lane < cluster && next < p.top ? S.part_top[lane][next] : 0;
      uint64_t most = head;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        const uint64_t other = __shfl_xor_sync(0xffffffffu, most, o);
        if (other > most) most = other;
      }
      most = __shfl_sync(0xffffffffu, most, 0);
      if (most != 0 && head == most) ++next;
      if (lane == k) key = most;
    }
  }
  // ---- the row's results
  const bool good = all.s > 0.f && all.s < INFINITY && all.m < INFINITY;
  const float nan = __uint_as_float(0x7fc00000u), logs = log2f(all.s);
  auto share = [&](float x) { return kLn2 * (relative(x, all.m) - logs); };  // the log probability of an element
  const int64_t place = static_cast<int64_t>(r) * p.top + lane;
  if (lane == 0) {
    p.entropy[r] = good ? kLn2 * (logs - all.t / all.s) : nan;
    if (p.tokens) {
      p.logprobs[r] = good ? share(given) : nan;
      p.ranks[r] = good ? before : -1;
    }
  }
  if (lane < p.top) {
    p.top_ids[place] = good && key ? index_of(key) : -1;
    p.top_logprobs[place] = !good ? nan : key ? share(logit_of(key)) : -INFINITY;
  }
}

// ------------------------------------------------------------------ host side
// CTAs of 64 threads, of which three times as many are resident, or of 256.
constexpr int kFew = 64, kMany = 256, kShort = 32768;
std::mutex g_mutex;
int g_sms[64];

cudaError_t setup(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!g_sms[dev]) {
    for (auto kernel : {logprobs_kernel<false, kFew>, logprobs_kernel<true, kFew>, logprobs_kernel<false, kMany>, logprobs_kernel<true, kMany>})
      if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(Shared<Cfg<kMany>>)))) != cudaSuccess) return e;
    int n = 0;
    if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    g_sms[dev] = n;
  }
  *sms = g_sms[dev];
  return cudaSuccess;
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
                    static_cast<const void*>(a->tokens) == a->entropy || static_cast<const void*>(a->tokens) == a->top_logprobs))
    return kda_internal_fail(KDA_ERR_SHAPE, "a result may not take the place of the tokens");
  const Params p{a->R, a->V, a->num_top, a->logits, a->logits_row_stride, a->tokens, a->logprobs, a->ranks, a->entropy,
                 a->top_ids, a->top_logprobs, a->err_flag};
  int sms = 0;
  cudaError_t e = setup(&sms);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "setup: %s", cudaGetErrorString(e));
  // Short rows, where a CTA's start and end count more than its sums, get small CTAs: those of one stage (549 of 424 fp32
  // logits 4.9 us, with 256 threads 6.7), and where all CTAs are not resident at once those up to kShort bytes (1,000 of
  // 4,096 fp32 logits 11.8 and 14.3, of 16,000 25.5 and 23.1) or, in many waves, twice that (4,000 of 5,000 30 and 53, of
  // 16,000 60 and 67, of 32,000 103 and 97).  Others get a cluster of CTAs each while those are resident at once and
  // each has a stage at least.
  const int64_t bytes = static_cast<int64_t>(a->V) * (bf16 ? 2 : 4);
  const int at_once = Cfg<kMany>::kCtasPerSm * sms;
  const bool few = bytes <= Cfg<kFew>::kStageBytes || (a->R > at_once && bytes <= (a->R > Cfg<kFew>::kCtasPerSm * sms ? 2 : 1) * kShort);
  int cluster = few ? 1 : kMaxCluster;
  while (cluster > 1 && (static_cast<int64_t>(a->R) * cluster > at_once || (cluster - 1) * int64_t{Cfg<kMany>::kStageBytes} >= bytes)) cluster >>= 1;
  auto kernel = few ? (bf16 ? logprobs_kernel<true, kFew> : logprobs_kernel<false, kFew>)
                    : (bf16 ? logprobs_kernel<true, kMany> : logprobs_kernel<false, kMany>);
  e = kda_internal_launch_cluster(kernel, dim3(static_cast<unsigned>(a->R) * cluster),
                                  dim3(few ? Cfg<kFew>::kAllThreads : Cfg<kMany>::kAllThreads),
                                  few ? sizeof(Shared<Cfg<kFew>>) : sizeof(Shared<Cfg<kMany>>), stream, cluster, p, cluster);
  if (e != cudaSuccess) return kda_internal_fail(KDA_ERR_LAUNCH, "launch: %s", cudaGetErrorString(e));
  return KDA_OK;
}
