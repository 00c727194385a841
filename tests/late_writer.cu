// A kernel that lets its dependents start at once and writes its result much
// later: sleeps for a given time (at most 10 s), then copies.
#include <cuda_runtime.h>
#include <stdint.h>

namespace {
__global__ void late_copy(uint8_t* dst, const uint8_t* src, int64_t bytes, uint64_t ns) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint64_t t0, now;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  for (int i = 0; i < 100000; ++i) {
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
    if (now - t0 >= ns) break;
    __nanosleep(100000);
  }
  __syncthreads();
  for (int64_t i = threadIdx.x; i < bytes; i += blockDim.x) dst[i] = src[i];
}
}  // namespace

extern "C" int late_writer_copy(void* dst, const void* src, int64_t bytes, uint64_t ns, void* stream) {
  late_copy<<<1, 256, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<uint8_t*>(dst), static_cast<const uint8_t*>(src), bytes, ns);
  return static_cast<int>(cudaGetLastError());
}
