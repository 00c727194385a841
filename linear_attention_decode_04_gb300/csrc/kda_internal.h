// kda_internal.h -- helpers shared by the translation units of the library
// (not part of the C ABI; hidden from the exported symbol table).
#pragma once

#define KDA_INTERNAL __attribute__((visibility("hidden")))

// Record a message for kda_last_error() and return `code`.
KDA_INTERNAL int kda_internal_fail(int code, const char* fmt, ...);
// Clear the message of kda_last_error() at the start of a call.
KDA_INTERNAL void kda_internal_clear_error();

#ifdef __CUDACC__
#include <cuda_runtime.h>

#include <utility>

// Launch `kernel` as a programmatic dependent launch: it may become resident
// while the stream's previous kernel drains, so it must execute
// griddepcontrol.wait before it touches memory.  `cluster` > 1 launches
// clusters of that many CTAs along x.
template <typename... P, typename... A>
static inline cudaError_t kda_internal_launch_cluster(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                                                      void* stream, unsigned cluster, A&&... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}
template <typename... P, typename... A>
static inline cudaError_t kda_internal_launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, void* stream,
                                              A&&... args) {
  return kda_internal_launch_cluster(kernel, grid, block, smem, stream, 1, std::forward<A>(args)...);
}
#endif
