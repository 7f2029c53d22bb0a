// Host set-up that is needed once, kept only where it succeeded: after a failure (a device
// that is out of memory or not ready yet) the next call tries again.
#pragma once

#include <atomic>

#include <cuda.h>
#include <cuda_runtime_api.h>

namespace qsw {

// The devices for which a set-up is done.
struct DeviceOnce {
  std::atomic<bool> done[64];
};

// Sets the current device up by `set_up`, which two threads may run at once.
template <class F>
cudaError_t once_per_device(DeviceOnce &once, F set_up) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (once.done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = set_up();
  if (e == cudaSuccess) once.done[dev].store(true, std::memory_order_release);
  return e;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled of the driver; null where there is none.
inline EncodeTiledFn encode_tiled_fn() {
  static std::atomic<EncodeTiledFn> held{nullptr};
  EncodeTiledFn fn = held.load(std::memory_order_acquire);
  if (fn) return fn;
  void *ptr = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess) {
    fn = reinterpret_cast<EncodeTiledFn>(ptr);
    held.store(fn, std::memory_order_release);
  }
  return fn;
}

}  // namespace qsw
