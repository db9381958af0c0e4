// What the launchers of the operators share: the device, its CUs, LDS past the default.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace moe {

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// the current device, or -1
inline int device() {
  int dev = -1;
  return hipGetDevice(&dev) == hipSuccess ? dev : -1;
}

inline int cu_count(int dev) {
  static std::atomic<int> known[64];  // asked for once per device
  int cus = dev >= 0 && dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (cus > 0) return cus;
  if (dev < 0 || hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
    return 256;
  if (dev < 64) known[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

// Dynamic LDS beyond the default, allowed once per kernel (its `done`) and device.
template <typename K>
hipError_t allow_lds(K* kernel, int bytes, int dev, std::atomic<uint64_t>& done) {
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return hipSuccess;
  const hipError_t e =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace moe
