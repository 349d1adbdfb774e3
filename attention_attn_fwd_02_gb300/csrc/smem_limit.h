// smem_limit.h -- dynamic shared-memory limits of the kernels, remembered.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

namespace attn {

// Raises a kernel's dynamic shared-memory limit to `bytes` on the current
// device once; the setting lasts for the process, so later launches only look
// it up (the attribute call costs microseconds, which small problems feel).
// The table is hashed by kernel and device and holds every kernel of the
// library (some 300) on sixteen devices; a pair that finds it full pays the
// attribute call each time.
inline cudaError_t ensure_smem(const void* kern, int bytes) {
  struct Entry {
    const void* k;
    int dev, bytes;
  };
  constexpr uint32_t kSlots = 8192, kProbes = 64;
  static std::mutex mu;
  static Entry tab[kSlots];   // k == nullptr: free
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const uint64_t h = ((uint64_t)(uintptr_t)kern + (uint64_t)dev) * 0x9E3779B97F4A7C15ull;
  const uint32_t first = (uint32_t)(h >> 51);   // 13 bits
  auto find = [&]() -> Entry* {                 // the pair's entry, or the free one where it goes, or null
    for (uint32_t i = 0; i < kProbes; ++i) {
      Entry& e = tab[(first + i) % kSlots];
      if (!e.k || (e.k == kern && e.dev == dev)) return &e;
    }
    return nullptr;
  };
  {
    std::lock_guard<std::mutex> lock(mu);
    const Entry* e = find();
    if (e && e->k && e->bytes >= bytes) return cudaSuccess;
  }
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess) {
    std::lock_guard<std::mutex> lock(mu);
    Entry* e = find();
    if (e && (!e->k || e->bytes < bytes)) *e = {kern, dev, bytes};
  }
  return err;
}

}  // namespace attn
