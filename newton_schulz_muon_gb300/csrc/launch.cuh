// Host-side helpers of the entry points that take no plan: the device they run on,
// and launches with a cluster size or with programmatic dependence on the kernel
// before them in the stream.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

namespace muon {
namespace {

// Multiprocessors of the current device; 0 when it is not sm_103 (or there is none).
inline int device_sms(cudaError_t* err) {
  static int cached[64];  // 0: not asked yet, -1: another architecture
  int dev = 0;
  *err = cudaGetDevice(&dev);
  if (*err != cudaSuccess) return 0;
  if (dev < 64 && cached[dev] != 0) return cached[dev] > 0 ? cached[dev] : 0;
  int major = 0, minor = 0, sms = 0;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  *err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (*err != cudaSuccess) return 0;
  const int found = major == 10 && minor == 3 ? sms : -1;
  if (dev < 64) cached[dev] = found;
  return found > 0 ? found : 0;
}

// dependent = true: the kernel may start while the kernel before it in the stream
// still runs; it must call griddep_wait before it reads that kernel's results, and
// in every thread that writes, so that the two kernels end in order.
template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int grid, int block, size_t smem, cudaStream_t s, int cluster,
                   bool dependent, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace
}  // namespace muon
