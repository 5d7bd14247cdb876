// The driver's encoder of tensor maps, found through the runtime (the library is
// not linked with the driver's).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

namespace nf {

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                            CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                            CUtensorMapFloatOOBfill);

inline cudaError_t encoder(Encode* out) {
  static std::atomic<void*> kept{nullptr};
  void* fn = kept.load(std::memory_order_relaxed);
  if (fn == nullptr) {
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
    kept.store(fn, std::memory_order_relaxed);
  }
  *out = reinterpret_cast<Encode>(fn);
  return cudaSuccess;
}

}  // namespace nf
