// A kernel's limit of dynamic shared memory.  Host code on the C runtime calls
// alone, so that a test can run it on a runtime of its own.
#pragma once

#include <atomic>
#include <mutex>

#include <cuda_runtime_api.h>

namespace moe_router {

// Allow `kern` the dynamic shared memory `smem` (above the 48 KB default
// only), once per device and size: `granted` is the calling launcher's own
// record (one per kernel instantiation), the largest size set per device.
// The limit is assigned, not raised: check, set and record are one step under a
// lock, so that a smaller size of another host thread is never set behind a
// larger one that is recorded.
constexpr int kSmemDevs = 64;
inline std::mutex g_smem_mu;

template <typename Kern>
cudaError_t allow_smem(Kern kern, size_t smem, std::atomic<int>* granted) {
  if (smem <= 48 * 1024) return cudaSuccess;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return cudaErrorInvalidDevice;
  const int want = static_cast<int>(smem);
  std::atomic<int>* const known = dev < kSmemDevs ? &granted[dev] : nullptr;
  if (known != nullptr && known->load(std::memory_order_acquire) >= want) return cudaSuccess;
  std::lock_guard<std::mutex> lock(g_smem_mu);
  if (known != nullptr && known->load(std::memory_order_relaxed) >= want) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, want);
  if (e == cudaSuccess && known != nullptr) known->store(want, std::memory_order_release);
  return e;
}

}  // namespace moe_router
