// elem.cuh -- 16-byte chunks of the element types the group-normalisation and
// dropout kernels take (bf16, fp16, fp32) as packed fp32 pairs.
#pragma once
#include <cuda_fp16.h>

#include "rowops.cuh"

namespace gbn {

// Element types, with the values of norm_dtype_t.
constexpr int kBF16 = 0;
constexpr int kFP16 = 1;
constexpr int kFP32 = 2;

__host__ __device__ constexpr int elem_bytes(int dt) { return dt == kFP32 ? 4 : 2; }
// Elements per 16-byte chunk.
__host__ __device__ constexpr int chunk_elems(int dt) { return 16 / elem_bytes(dt); }

// Chunk -> exact fp32 pairs (lower address first).
template <int DT>
__device__ __forceinline__ void unpack(const uint4 &c, float2 (&v)[chunk_elems(DT) / 2]) {
  if constexpr (DT == kBF16) {
    chunk_to_f2(c, v);
  } else if constexpr (DT == kFP16) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = __half22float2(*reinterpret_cast<const __half2 *>(&w[p]));
  } else {
    v[0] = make_float2(__uint_as_float(c.x), __uint_as_float(c.y));
    v[1] = make_float2(__uint_as_float(c.z), __uint_as_float(c.w));
  }
}

// fp32 pairs -> chunk, rounded to nearest even.
template <int DT>
__device__ __forceinline__ uint4 pack(const float2 (&v)[chunk_elems(DT) / 2]) {
  if constexpr (DT == kBF16) {
    return f2_to_chunk(v);
  } else if constexpr (DT == kFP16) {
    uint32_t w[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const __half2 h = __floats2half2_rn(v[p].x, v[p].y);
      w[p] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                      __float_as_uint(v[1].y));
  }
}

// One element, for the ragged end of a flat tensor.
template <int DT>
__device__ __forceinline__ float load_elem(const void *p, int64_t i) {
  if constexpr (DT == kBF16)
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
  else if constexpr (DT == kFP16)
    return __half2float(static_cast<const __half *>(p)[i]);
  else
    return static_cast<const float *>(p)[i];
}
template <int DT>
__device__ __forceinline__ void store_elem(void *p, int64_t i, float v) {
  if constexpr (DT == kBF16)
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else if constexpr (DT == kFP16)
    static_cast<__half *>(p)[i] = __float2half_rn(v);
  else
    static_cast<float *>(p)[i] = v;
}

}  // namespace gbn
