// What launchers look up once (host code alone).
#pragma once

#include <atomic>
#include <mutex>

#include "common.cuh"

namespace te {
namespace {

// State of each device that is looked up on the first call there.  Host threads may make that call together:
// one looks up, under the lock, and the flag that it sets last (release) is what the others go by (acquire).
template <typename T>
class PerDevice {
 public:
  // The current device's state, filled by make(T*) the first time.  Where that fails: nullptr, its status in
  // *status, and the next call tries again.
  template <typename Make>
  const T* get(te_status* status, Make make) {
    int d = -1;
    cudaGetDevice(&d);
    if (d < 0 || d >= kDevices) {
      *status = TE_ERR_CUDA;
      return nullptr;
    }
    Slot& slot = slots_[d];
    if (!slot.ready.load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> lock(mutex_);
      if (!slot.ready.load(std::memory_order_relaxed)) {
        *status = make(&slot.value);
        if (*status != TE_OK) return nullptr;
        slot.ready.store(true, std::memory_order_release);
      }
    }
    return &slot.value;
  }

 private:
  static constexpr int kDevices = 64;
  struct Slot {
    std::atomic<bool> ready{false};
    T value{};
  };
  std::mutex mutex_;
  Slot slots_[kDevices];
};

template <typename... P>
[[maybe_unused]] const void* kernel_address(void (*kernel)(P...)) {
  return reinterpret_cast<const void*>(kernel);
}

// A kernel's shared memory beyond 48 KB.
struct SharedMemory {};
[[maybe_unused]] inline te_status allow_shared_memory(SharedMemory*, const void* kernel, int bytes) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return record_cuda(cudaGetLastError());
  return TE_OK;
}

// The shared memory of a GEMM kernel, and the CTA pairs (pair size 1: CTAs) that run at once or, where several
// pairs share a tile, the clusters of two and of four pairs.
struct GemmSetup {
  int units, fours;
  // cfg: the launch's block, shared memory and attributes, the first of them its cluster.
  te_status set(const void* kernel, int pair, bool shared, int smem, cudaLaunchConfig_t cfg) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return record_cuda(cudaGetLastError());
    cudaLaunchAttribute attr[1] = {cfg.attrs[0]};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int sms = num_sms();
    if (shared) {
      for (int pairs = 4; pairs >= 2; pairs -= 2) {
        attr[0].val.clusterDim.x = static_cast<unsigned>(2 * pairs);
        cfg.gridDim = dim3(static_cast<unsigned>(sms / (2 * pairs) * 2 * pairs), 1, 1);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
          cudaGetLastError();   // no such cluster: not taken
          n = 0;
        }
        (pairs == 4 ? fours : units) = n;
      }
      return TE_OK;
    }
    units = sms / pair;
    if (pair > 1) {
      // pairs that can be resident at once (a GPC may leave an SM unpaired)
      cfg.gridDim = dim3(static_cast<unsigned>(pair * units), 1, 1);
      int n = 0;
      const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      if (e != cudaSuccess || n <= 0) {
        cudaGetLastError();
        return record_cuda(e != cudaSuccess ? e : cudaErrorInvalidConfiguration);
      }
      units = n < units ? n : units;
    }
    return TE_OK;
  }
};

// The shared memory of the two forms of a stream kernel, and how many clusters of 2, 4 and 8 CTAs of the shared
// form run at once.
struct StreamSetup {
  int most[3];
  te_status set(const void* single, const void* shared, int threads, int smem) {
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
    return TE_OK;
  }
};

}  // namespace
}  // namespace te
