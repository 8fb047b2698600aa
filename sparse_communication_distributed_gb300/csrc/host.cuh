// Host helpers of the calls without a handle: errors, checks of buffers, launches (internal).
#pragma once
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/scape.h"
#include "scape_kernels.cuh"

namespace scape {

// Notes the message for scape_last_error(NULL) of this thread; returns the code.
inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_thread_error(buf);
  return code;
}

inline bool known(int dtype) { return dtype >= SCAPE_BF16 && dtype <= SCAPE_F32; }
inline uint64_t size_of(int dtype) { return dtype == SCAPE_F32 ? 4 : 2; }
inline bool misaligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }
// Whether two buffers of n and m bytes share any.
inline bool ranges_meet(const void* p, uint64_t n, const void* q, uint64_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && n && m && a < b + m && b < a + n;
}

// Launches behind the kernel in front of it, which it waits for on the GPU
// (grid_dependency_wait); in clusters of "cluster" CTAs.
template <class K, class... A>
cudaError_t launch_clusters(K kernel, unsigned grid, unsigned block, uint32_t smem, int cluster, cudaStream_t s,
                            const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}
template <class K, class... A>
cudaError_t launch_behind(K kernel, unsigned grid, unsigned block, cudaStream_t s, const A&... args) {
  return launch_clusters(kernel, grid, block, 0u, 1, s, args...);
}

}  // namespace scape
