// tensor_map.cu -- the driver's tensor-map encoder, and the check of addresses.
#include "tensor_map.h"

#include <cuda_runtime.h>

#include <atomic>

namespace gbn {

norm_status_t map_encoder(MapEncoder *out) {
  static std::atomic<MapEncoder> found{nullptr};
  MapEncoder enc = found.load(std::memory_order_relaxed);
  if (!enc) {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn) {
      cudaGetLastError();
      return NORM_ERR_CUDA;
    }
    enc = reinterpret_cast<MapEncoder>(fn);
    found.store(enc, std::memory_order_relaxed);
  }
  *out = enc;
  return NORM_OK;
}

norm_status_t check_device_memory(const void *p, int dev) {
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();
    return NORM_ERR_MEMORY;
  }
  if (a.type == cudaMemoryTypeManaged) return NORM_OK;
  return a.type == cudaMemoryTypeDevice && a.device == dev ? NORM_OK : NORM_ERR_MEMORY;
}

}  // namespace gbn
