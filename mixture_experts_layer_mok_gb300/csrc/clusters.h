// Launches of kernels in thread-block clusters.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace mok {

// A kernel's launch attributes, and how many clusters of each size are
// resident at once on a device (looked up once).  GB300's SMs come in groups
// of different sizes, so that fewer large clusters fit than the SM count says:
// of the pair split kernel 76 of 2 CTAs, 36 of 4, 23 of 6 and 15 of 8.
struct KernelInfo {
  std::atomic<int> resident[64][9] = {};   // 0: not looked up yet; any thread may be the first
};

template <class K>
cudaError_t resident_clusters(K kern, KernelInfo& info, int threads, int smem, int cluster, int* n) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64 || cluster < 1 || cluster > 8) return cudaErrorInvalidValue;
  std::atomic<int>& at = info.resident[dev][cluster];
  int found = at.load(std::memory_order_acquire);
  if (found == 0) {
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster * 1024);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaOccupancyMaxActiveClusters(&found, kern, &cfg);
    if (err != cudaSuccess) return err;
    if (found <= 0) return cudaErrorInvalidConfiguration;
    at.store(found, std::memory_order_release);
  }
  *n = found;
  return cudaSuccess;
}

template <class K, class... A>
cudaError_t launch_clusters(K kern, dim3 grid, int threads, int smem, int cluster, cudaStream_t st, const A&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace mok
