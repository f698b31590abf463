// fold.cuh -- sums of the columns of partial rows in a fixed order.
#pragma once
#include <cstdint>

namespace gbn {

// For a block of 1024 threads: out[c] = the sum of column c of `rows` rows of n fp32
// values at src, for the 32 columns of block blockIdx.x.  32 rows are added side by
// side (each warp takes every 32nd), then the 32 sums in order.  out may be null.
__device__ __forceinline__ void fold_columns(const float *src, int rows, int n, float *out) {
  __shared__ float sum[32][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x / 32;
  const int col = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (out && col < n) {
#pragma unroll 4
    for (int r = row; r < rows; r += 32) v += __ldcg(src + static_cast<int64_t>(r) * n + col);
  }
  sum[row][lane] = v;
  __syncthreads();
  if (row == 0 && out && col < n) {
    v = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) v += sum[r][lane];
    out[col] = v;
  }
}

}  // namespace gbn
