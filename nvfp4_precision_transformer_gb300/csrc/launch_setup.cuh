// What launchers look up once (host code alone).
#pragma once

#include "common.cuh"

namespace te {
namespace {

template <typename... P>
[[maybe_unused]] const void* kernel_address(void (*kernel)(P...)) {
  return reinterpret_cast<const void*>(kernel);
}

// Once a device: the shared memory of the two forms of a kernel, and how many clusters of 2, 4 and 8 CTAs
// of the shared form run at once.
struct StreamSetup {
  bool done;
  int most[3];
  te_status set(const void* single, const void* shared, int threads, int smem) {
    if (done) return TE_OK;
    if (cudaFuncSetAttribute(single, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaFuncSetAttribute(shared, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return record_cuda(cudaGetLastError());
    for (int i = 0; i < 3; ++i) {
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim = {2u << i, 1u, 1u};
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2u << i, 1, 1);
      cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
      cfg.dynamicSmemBytes = static_cast<size_t>(smem);
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&most[i], shared, &cfg) != cudaSuccess) {
        cudaGetLastError();   // no such cluster: not taken (the forms without it run all the same)
        most[i] = 0;
      }
    }
    done = true;
    return TE_OK;
  }
};

}  // namespace
}  // namespace te
