// dynamic_lds.h -- launches of kernels with more dynamic LDS than the default.
#pragma once
#include <atomic>
#include <hip/hip_runtime.h>

namespace moe {

// Allows a kernel more than the default dynamic LDS, once per device, and
// gives the device's number of compute units.  Calls of several threads may
// come here at once: one word says that it has been done, and is the number.
template <auto KERN>
hipError_t allow_lds(int bytes, int* cus) {
  static std::atomic<int> count[64] = {};  // 0: not yet
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  const bool known = dev >= 0 && dev < 64;
  *cus = known ? count[dev].load(std::memory_order_acquire) : 0;
  if (*cus > 0) return hipSuccess;
  err = hipFuncSetAttribute((const void*)KERN, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err != hipSuccess) return err;
  err = hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (err == hipSuccess && known) count[dev].store(*cus, std::memory_order_release);
  return err;
}

}  // namespace moe
