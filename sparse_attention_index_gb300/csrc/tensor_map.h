// The driver's encoder of tensor maps, looked up at run time (libdsa.so does not link the driver's library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

namespace dsa {

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// nullptr where the driver has none. Any thread may ask; those that ask first at the same time find the
// same function, each by itself.
inline EncodeTiled encode_tiled() {
  static std::atomic<EncodeTiled> known{nullptr};
  EncodeTiled fn = known.load(std::memory_order_relaxed);
  if (fn != nullptr) return fn;
  void* ptr = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                       &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess)
    return nullptr;
  fn = reinterpret_cast<EncodeTiled>(ptr);
  known.store(fn, std::memory_order_relaxed);
  return fn;
}

}  // namespace dsa
