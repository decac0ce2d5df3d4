// Launches of the operators over pages: under the stream's last kernel
// (programmatic dependent launch), with what a kernel has to be told once per
// device told once.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace lps {

template <class Kern, class... Args>
cudaError_t launch_early_clusters(Kern kern, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
template <class Kern, class... Args>
cudaError_t launch_early(Kern kern, dim3 grid, int threads, size_t smem, cudaStream_t s, const Args&... args) {
  return launch_early_clusters(kern, grid, threads, smem, 1, s, args...);
}

// The current device's number of SMs (asked for once per device).
inline cudaError_t sm_count(int* n) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool keep = dev >= 0 && dev < 64;
  if (keep && (*n = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && keep) known[dev].store(*n, std::memory_order_relaxed);
  return e;
}

// Lets a kernel use `bytes` of dynamic shared memory on the current device. `told`:
// a bit per device, static beside the kernel's launch.
template <class Kern>
cudaError_t allow_smem(Kern kern, size_t bytes, std::atomic<uint64_t>& told) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (told.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) told.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace lps
