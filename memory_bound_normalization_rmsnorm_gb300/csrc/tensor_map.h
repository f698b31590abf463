// tensor_map.h -- what every launch with tensor copies needs from the driver.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include "../../include/gbnorm.h"

namespace gbn {

using MapEncoder = PFN_cuTensorMapEncodeTiled_v12000;

// The driver's encoder of tensor maps.  Found once; a failed lookup is not kept.
norm_status_t map_encoder(MapEncoder *out);

// Tensor maps take addresses that this GPU can reach: device memory of the current
// device `dev`, or managed memory.  Host memory, another device's memory and
// addresses unknown to CUDA are NORM_ERR_MEMORY.
norm_status_t check_device_memory(const void *p, int dev);

}  // namespace gbn
