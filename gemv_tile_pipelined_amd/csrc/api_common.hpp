// api_common.hpp -- what the entry points of api.hip and layer_api.hip share:
// pointer checks, the status of a launch, and the compute units of the current
// device.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/gemvtile.h"

namespace gt {

constexpr int kMaxDevices = 64;
inline std::atomic<int> g_cu_count[kMaxDevices];

inline bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

inline int to_status(hipError_t e) { return e == hipSuccess ? GEMVTILE_OK : GEMVTILE_ERR_LAUNCH; }

// Compute units of the current device, cached per device.
inline int current_cu_count(int *out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return GEMVTILE_ERR_DEVICE;
  if (dev >= 0 && dev < kMaxDevices) {
    const int cached = g_cu_count[dev].load(std::memory_order_relaxed);
    if (cached > 0) {
      *out = cached;
      return GEMVTILE_OK;
    }
  }
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
    return GEMVTILE_ERR_DEVICE;
  if (dev >= 0 && dev < kMaxDevices) g_cu_count[dev].store(cus, std::memory_order_relaxed);
  *out = cus;
  return GEMVTILE_OK;
}

}  // namespace gt
