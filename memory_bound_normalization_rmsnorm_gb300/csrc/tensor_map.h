// tensor_map.h -- host side of tiled tensor copies (gemm.cu).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include "../../include/gbnorm.h"

namespace gbn {

// The driver's cuTensorMapEncodeTiled, looked up once.
norm_status_t tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000 *out);

// NORM_OK where p is memory that a tensor map of device `dev` can address.
norm_status_t check_device_memory(const void *p, int dev);

}  // namespace gbn
