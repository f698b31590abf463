// linear_grad.cu -- what the products of norm_linear_bwd need beside them: dz =
// dy act'(z) with the column sums that are dbias, and copies of operands that
// tensor copies cannot address.
#include <cuda_runtime.h>

#include "fold.cuh"
#include "linear.cuh"

namespace gbn {

namespace {

constexpr int kGradRows = 4;  // rows in flight per thread

// Bound by HBM: one read of dy and z, one write of dz.  A warp takes rows of 256
// columns (32 with V = 1), the CTA's 8 warps every 8th row of a chunk; a
// thread's sums are those of its V columns, joined over the warps in order into
// one row of partials per chunk.  Sums are of the unrounded dz.  dz itself is
// rounded to the operands' 16-bit type, since kind::f16 takes no wider one: the
// errors of dx and dW are those of two roundings in place of one (1.41 times), where
// dz as the sum of two 16-bit values would double their products.
template <int DT, int V>
__global__ void __launch_bounds__(kGradThreads) linear_grad_kernel(const GradArgs a) {
  constexpr int W = kGradThreads / 32;
  __shared__ float fold[W][32 * V];
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int col = (blockIdx.x * 32 + lane) * V;
  const int r0 = int(int64_t(a.M) * blockIdx.y / a.chunks);
  const int r1 = int(int64_t(a.M) * (blockIdx.y + 1) / a.chunks);
  const bool on = col < a.N;
  const uint16_t *dy = static_cast<const uint16_t *>(a.dy) + col;
  const uint16_t *z = static_cast<const uint16_t *>(a.z) + col;
  uint16_t *dz = static_cast<uint16_t *>(a.dz) + col;
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.f;
  for (int r = r0 + warp; r < r1; r += W * kGradRows) {
    uint4 vd[kGradRows], vz[kGradRows];
#pragma unroll
    for (int u = 0; u < kGradRows; ++u) {
      const int64_t row = r + u * W;
      if (on && row < r1) {
        if constexpr (V == 8) {
          vd[u] = ld_global_nc_v4(dy + row * a.lddy);
          if (a.act != kLinNone) vz[u] = ld_global_nc_v4(z + row * a.ldz);
        } else {
          vd[u].x = dy[row * a.lddy];
          if (a.act != kLinNone) vz[u].x = z[row * a.ldz];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kGradRows; ++u) {
      const int64_t row = r + u * W;
      if (!on || row >= r1) continue;
      const uint32_t wd[4] = {vd[u].x, vd[u].y, vd[u].z, vd[u].w};
      const uint32_t wz[4] = {vz[u].x, vz[u].y, vz[u].z, vz[u].w};
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 d = lin_unpack<DT>(wd[i / 2]);
        f[i] = (i & 1) ? d.y : d.x;
        if (a.act != kLinNone) {
          const float2 zz = lin_unpack<DT>(wz[i / 2]);
          f[i] *= lin_act_grad((i & 1) ? zz.y : zz.x, a.act);
        }
        sum[i] += f[i];
      }
      if (a.dz) {
        if constexpr (V == 8)
          *reinterpret_cast<uint4 *>(dz + row * a.lddz) =
              make_uint4(lin_pack<DT>(f[0], f[1]), lin_pack<DT>(f[2], f[3]),
                         lin_pack<DT>(f[4], f[5]), lin_pack<DT>(f[6], f[7]));
        else
          store_elem<DT>(dz + row * a.lddz, 0, f[0]);
      }
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < V; ++i) fold[warp][lane * V + i] = sum[i];
  __syncthreads();
  for (int c = threadIdx.x; c < 32 * V; c += kGradThreads) {
    const int at = blockIdx.x * 32 * V + c;
    if (at >= a.N) break;
    float v = fold[0][c];
#pragma unroll
    for (int w = 1; w < W; ++w) v += fold[w][c];
    a.part[int64_t(blockIdx.y) * a.N + at] = v;
  }
}

// Adds the chunks' rows in order.
__global__ void __launch_bounds__(1024)
    linear_fold_kernel(const float *part, int n, int rows, float *out) {
  grid_launch_dependents();
  grid_dependency_wait();
  fold_columns(part, rows, n, out);
}

// 16-bit rows to rows whose stride and address tensor copies take; one or two
// matrices, one after the other along the grid's x.  T: one element, or two where
// every row starts on a multiple of four bytes.  A warp takes 256 T of a row.
template <typename T>
__global__ void __launch_bounds__(256) linear_pack_kernel(const __grid_constant__ PackArgs a) {
  constexpr int E = sizeof(T) / 2;
  grid_launch_dependents();
  grid_dependency_wait();
  const bool second = static_cast<int>(blockIdx.x) >= a.strips[0];
  const T *src = reinterpret_cast<const T *>(second ? a.src[1] : a.src[0]);
  T *dst = reinterpret_cast<T *>(second ? a.dst[1] : a.dst[0]);
  const int64_t ld = (second ? a.ld[1] : a.ld[0]) / E, ldd = (second ? a.ldd[1] : a.ldd[0]) / E;
  const int rows = second ? a.rows[1] : a.rows[0];
  const int cols = (second ? a.cols[1] : a.cols[0]) / E;
  const int c0 = (static_cast<int>(blockIdx.x) - (second ? a.strips[0] : 0)) * 256 + (threadIdx.x & 31);
  for (int r = blockIdx.y * 8 + threadIdx.x / 32; r < rows; r += gridDim.y * 8) {
    T v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (c0 + 32 * u < cols) v[u] = src[r * ld + c0 + 32 * u];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (c0 + 32 * u < cols) dst[r * ldd + c0 + 32 * u] = v[u];
  }
}

}  // namespace

const void *linear_grad_kernel_ptr(bool bf16, bool vec) {
  if (bf16)
    return vec ? reinterpret_cast<const void *>(&linear_grad_kernel<kBF16, 8>)
               : reinterpret_cast<const void *>(&linear_grad_kernel<kBF16, 1>);
  return vec ? reinterpret_cast<const void *>(&linear_grad_kernel<kFP16, 8>)
             : reinterpret_cast<const void *>(&linear_grad_kernel<kFP16, 1>);
}
const void *linear_fold_kernel_ptr() { return reinterpret_cast<const void *>(&linear_fold_kernel); }
const void *linear_pack_kernel_ptr(bool two) {
  return two ? reinterpret_cast<const void *>(&linear_pack_kernel<uint32_t>)
             : reinterpret_cast<const void *>(&linear_pack_kernel<uint16_t>);
}

}  // namespace gbn
