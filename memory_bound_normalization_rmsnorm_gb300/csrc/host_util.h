// host_util.h -- host-side helpers shared by the entry points that live
// outside api.cu.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gbnorm.h"

namespace gbn {

struct DropArgs;

inline bool aligned_to_16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Validates p and offset_dev and forms the kernel argument (dropout.cu).
norm_status_t make_drop(float p, uint64_t seed, uint64_t offset, const void *offset_dev,
                        DropArgs *out);

// Ordinal, SM count, opt-in shared memory per block, device error word and
// context identity of the current device (api.cu).
norm_status_t device_context(int *dev, int *sms, int *smem_optin, unsigned **err,
                             unsigned long long *ctx);

// The attributes a kernel with opt-in shared memory or a large cluster needs,
// set once per device and context (api.cu).
norm_status_t function_ready(int dev, const void *fn, int smem_optin);

// One launch with programmatic stream serialisation allowed (the kernel waits
// for its predecessor before touching global memory), as clusters of
// `cluster` CTAs when that is above 1 (api.cu).
norm_status_t launch_serial(const void *fn, dim3 grid, dim3 block, size_t smem, int cluster,
                            void **args, cudaStream_t s);

// One launch whose CTAs are all resident at once (grid-wide barriers) (api.cu).
norm_status_t launch_cooperative(const void *fn, dim3 grid, dim3 block, size_t smem, void **args,
                                 cudaStream_t s);

// Fixed-order column sum of P fp32 rows [P][n] (and, with dbeta, of the P
// rows that follow them) into dgamma (dbeta), on `s` (api.cu).
norm_status_t reduce_rows(const float *rows, int P, int n, float *dgamma, float *dbeta,
                          cudaStream_t s);

}  // namespace gbn
