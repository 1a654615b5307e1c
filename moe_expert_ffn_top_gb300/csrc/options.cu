// What kernels have to be allowed before a launch (see options.h), once per kernel and device.
#include <stdint.h>

#include <atomic>

#include "options.h"

namespace moelora {

namespace {

constexpr int kSlots = 1024;  // a few hundred kernels ask; one that finds no slot asks every time
struct Slot {
  std::atomic<const void*> kernel;
  std::atomic<uint64_t> devices;  // bit d: allowed on device d
};
Slot slots[kSlots];

std::atomic<uint64_t>* devices_of(const void* kernel) {
  for (size_t h = (reinterpret_cast<uintptr_t>(kernel) >> 4) % kSlots, n = 0; n < kSlots; ++n, h = (h + 1) % kSlots) {
    const void* key = slots[h].kernel.load(std::memory_order_acquire);
    if (!key && slots[h].kernel.compare_exchange_strong(key, kernel)) return &slots[h].devices;
    if (key == kernel) return &slots[h].devices;  // there before, or another thread's a moment ago
  }
  return nullptr;
}

}  // namespace

cudaError_t allow_options(const void* kernel, bool again) {
  int dev = 0, most = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::atomic<uint64_t>* devices = devices_of(kernel);
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (!again && devices && (devices->load(std::memory_order_acquire) & bit)) return cudaSuccess;
  cudaFuncAttributes at;
  e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, kernel);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)at.sharedSizeBytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && devices) devices->fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace moelora
