// kda_tc.cuh -- mbarriers with bounded waits, copies by the tensor memory
// accelerator and tcgen05 products, as the matrix product kernels use them, and
// arithmetic on pairs of floats.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ __forceinline__ uint32_t s32(const void* ptr) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(ptr));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two floats in one instruction.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(s32(b)), "r"(count));
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(s32(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(s32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(s32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase, at most kWaitLimitNs; after any thread of the CTA has
// given up, no thread waits any more.
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, int* failed) {
  if (bar_try(b, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    if (bar_try(b, parity)) return true;
    if (*reinterpret_cast<volatile int*>(failed)) return false;
    uint64_t now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
    if (it == 0) t0 = now;
    else if (now - t0 > kWaitLimitNs) {
      *reinterpret_cast<volatile int*>(failed) = 1;
      return false;
    }
  }
}
// One lane of a warp that is together.  (Code that whole warps run, with one lane
// elected for an instruction, keeps its operands in uniform registers: a product
// takes 40 cycles to issue that way, 60 in code of one lane, and a wait ahead of
// four of them 50 more against 250.)
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
// bar_wait for a warp that is together, which leaves it together.
__device__ __forceinline__ bool warp_wait(uint64_t* b, uint32_t parity, int* failed) {
  return __all_sync(0xffffffffu, bar_wait(b, parity, failed));
}
// The same without regard to others that gave up: for copies already on their way.
__device__ __forceinline__ void bar_drain(uint64_t* b, uint32_t parity) {
  uint64_t t0, now;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  do asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
  while (!bar_try(b, parity) && now - t0 < kWaitLimitNs);
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(s32(b)) : "memory");
}
// Shared-memory matrix descriptor of a K-major operand in rows of 128 bytes
// under the 128-byte swizzle: start in 16-byte units, eight rows (1,024 bytes)
// between groups of rows, version 1, swizzle 2.
__device__ __forceinline__ uint64_t sdesc128(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: f32 accumulator, both operands K-major, e4m3 (kind::f8f6f4) or bf16 (kind::f16).
__host__ __device__ constexpr uint32_t idesc_k(bool e4m3, uint32_t m, uint32_t n) {
  return (1u << 4) | (e4m3 ? 0u : (1u << 7) | (1u << 10)) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
template <bool E4M3>
__device__ __forceinline__ void mma_1cta(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  if constexpr (E4M3)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* b) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(s32(b))
      : "memory");
}
// ---- two CTAs as one: products of 256 rows whose halves, and those of the
// other operand, lie in both CTAs' shared memory, at the same places; the even
// CTA issues them and its barriers count the copies of both.
__device__ __forceinline__ uint32_t in_cta(const void* ptr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(s32(ptr)), "r"(rank));
  return a;
}
// Signals that tensor memory has been read: its loads have ended, and what the thread wrote to memory is none of the
// barrier's business.  (With a release at cluster scope every tile waited for its results to reach memory.)
__device__ __forceinline__ void bar_signal(uint64_t* b) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(s32(b)) : "memory");
}
__device__ __forceinline__ void bar_signal_at(uint32_t b) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(b) : "memory");
}
// Shared memory of this CTA to that of another of the cluster, whose barrier counts the bytes.
__device__ __forceinline__ void send(uint32_t dst, const void* src, uint32_t bytes, uint32_t b) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(s32(src)), "r"(bytes), "r"(b)
               : "memory");
}
__device__ __forceinline__ void commit_both(uint64_t* b, uint32_t even) {  // at the same place in the even CTA and the next
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(s32(b)),
      "h"(static_cast<uint16_t>(3u << even))
      : "memory");
}
template <bool E4M3>
__device__ __forceinline__ void mma_2cta(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  if constexpr (E4M3)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t b) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(b)
      : "memory");
}
__device__ __forceinline__ void tma_3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t b) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(b)
      : "memory");
}
// 8 BLOCKS consecutive columns of this warp's 32 lanes as fragments: thread i gets,
// in r[b][j], lane i / 4 + 8 j, columns 8 b + 2 (i % 4) and the next.  The load
// writes the registers of all 32 threads, so the warp has to be together; load and
// wait are one statement, so that nothing can come between them.
template <int BLOCKS>
__device__ __forceinline__ void tm_fragments(uint32_t addr, float (&r)[BLOCKS][4][2]) {
  static_assert(BLOCKS == 1 || BLOCKS == 2 || BLOCKS == 4, "8, 16 or 32 columns");
  __syncwarp();
  const uint32_t up = addr + (16u << 16);  // the upper 16 lanes
  if constexpr (BLOCKS == 1) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%8];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%4,%5,%6,%7}, [%9];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0][0][0]), "=f"(r[0][0][1]), "=f"(r[0][1][0]), "=f"(r[0][1][1]), "=f"(r[0][2][0]), "=f"(r[0][2][1]),
          "=f"(r[0][3][0]), "=f"(r[0][3][1])
        : "r"(addr), "r"(up)
        : "memory");
  } else if constexpr (BLOCKS == 2) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0][0][0]), "=f"(r[0][0][1]), "=f"(r[0][1][0]), "=f"(r[0][1][1]), "=f"(r[1][0][0]), "=f"(r[1][0][1]),
          "=f"(r[1][1][0]), "=f"(r[1][1][1]), "=f"(r[0][2][0]), "=f"(r[0][2][1]), "=f"(r[0][3][0]), "=f"(r[0][3][1]),
          "=f"(r[1][2][0]), "=f"(r[1][2][1]), "=f"(r[1][3][0]), "=f"(r[1][3][1])
        : "r"(addr), "r"(up)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
        "[%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0][0][0]), "=f"(r[0][0][1]), "=f"(r[0][1][0]), "=f"(r[0][1][1]), "=f"(r[1][0][0]), "=f"(r[1][0][1]),
          "=f"(r[1][1][0]), "=f"(r[1][1][1]), "=f"(r[2][0][0]), "=f"(r[2][0][1]), "=f"(r[2][1][0]), "=f"(r[2][1][1]),
          "=f"(r[3][0][0]), "=f"(r[3][0][1]), "=f"(r[3][1][0]), "=f"(r[3][1][1]), "=f"(r[0][2][0]), "=f"(r[0][2][1]),
          "=f"(r[0][3][0]), "=f"(r[0][3][1]), "=f"(r[1][2][0]), "=f"(r[1][2][1]), "=f"(r[1][3][0]), "=f"(r[1][3][1]),
          "=f"(r[2][2][0]), "=f"(r[2][2][1]), "=f"(r[2][3][0]), "=f"(r[2][3][1]), "=f"(r[3][2][0]), "=f"(r[3][2][1]),
          "=f"(r[3][3][0]), "=f"(r[3][3][1])
        : "r"(addr), "r"(up)
        : "memory");
  }
}
// 32 lanes x 8 columns of accumulators, added to those at `to`, or in their place; tm_put_wait() before they are read.
__device__ __forceinline__ void tm_add(uint32_t from, uint32_t to, bool first) {
  __syncwarp();
  float a[8], b[8];  // (what the second place holds at first is not looked at)
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3]), "=f"(a[4]), "=f"(a[5]), "=f"(a[6]), "=f"(a[7]),
        "=f"(b[0]), "=f"(b[1]), "=f"(b[2]), "=f"(b[3]), "=f"(b[4]), "=f"(b[5]), "=f"(b[6]), "=f"(b[7])
      : "r"(from), "r"(to)
      : "memory");
#pragma unroll
  for (int e = 0; e < 8; ++e) a[e] = first ? a[e] : a[e] + b[e];
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(to), "f"(a[0]), "f"(a[1]), "f"(a[2]), "f"(a[3]), "f"(a[4]), "f"(a[5]), "f"(a[6]), "f"(a[7])
               : "memory");
}
__device__ __forceinline__ void tm_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Four 8 x 8 matrices of 16-bit values between fragments and rows of 16 bytes
// in shared memory, transposed; thread i has the address of row i % 8 of matrix i / 8.
__device__ __forceinline__ void store_transposed(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void load_transposed(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

}  // namespace
