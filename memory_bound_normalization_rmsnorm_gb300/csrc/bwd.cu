// bwd.cu -- backward RMSNorm / LayerNorm: one fused row pass (dx, plus
// per-CTA partial column sums for dgamma and dbeta) and a fixed-order
// reduction of those partials.
//
// Follows the backward-pass paragraphs of "PyTorch atinge desempenho SOTA
// em normalizacao com torch.compile" (matsubara.tec.br):
//   - dX, dW and dB computed in ONE kernel so that dy and x are read once
//     (the fused-reduction paragraph);
//   - the column reduction split across CTAs, each CTA summing many rows
//     into a partial row of a workspace that a second kernel reduces,
//     without atomics (the split-reduction paragraph);
//   - rows per partial set by how many CTAs run (the SPLIT_SIZE paragraph)
//     and several loads kept in flight (the num_stages paragraph).
// The saved rstd (and mean) of the forward pass are reused, not recomputed.
#include "bwd_kernel.cuh"

namespace gbn {

namespace {

// Self-test of the bounded-wait failure path: waits on phase 0 of an
// mbarrier that expects one arrival which never comes.
__global__ void selftest_wait_kernel(unsigned *err, uint32_t polls) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) mbar_wait(&bar, 0, err, &abort_flag, polls);
}

constexpr int kReduceWarps = 32;
constexpr int kReduceBatch = 8;  // partial rows a lane loads before adding

// dgamma[j] = sum over p of ws[p][j] (blockIdx.y = 0) and dbeta[j] = sum
// over p of ws[P + p][j] (blockIdx.y = 1).  Warp w of the block sums the
// contiguous range p in [P*w/32, P*(w+1)/32) in increasing p (loads of a
// batch issued together, then added in order); the 32 warp sums are then
// added in warp order: a fixed order for a given P, so the result is bitwise
// reproducible.  Each lane owns 4 consecutive columns.
__global__ void __launch_bounds__(kReduceWarps * 32) reduce_partials_kernel(
    const float *__restrict__ ws, int P, int N, float *__restrict__ dgamma,
    float *__restrict__ dbeta) {
  __shared__ float4 part[kReduceWarps][32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int w = threadIdx.x >> 5;
  const float *src = ws + static_cast<size_t>(blockIdx.y) * P * N;
  float *dst = blockIdx.y ? dbeta : dgamma;
  const int col = (blockIdx.x * 32 + lane) * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < N) {
    const int p0 = static_cast<int>((static_cast<int64_t>(P) * w) / kReduceWarps);
    const int p1 = static_cast<int>((static_cast<int64_t>(P) * (w + 1)) / kReduceWarps);
    for (int p = p0; p < p1; p += kReduceBatch) {
      float4 v[kReduceBatch];
#pragma unroll
      for (int u = 0; u < kReduceBatch; ++u)
        v[u] = (p + u < p1) ? __ldcg(reinterpret_cast<const float4 *>(
                                  src + static_cast<size_t>(p + u) * N + col))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < kReduceBatch; ++u) {
        if (p + u < p1) {
          acc.x += v[u].x; acc.y += v[u].y; acc.z += v[u].z; acc.w += v[u].w;
        }
      }
    }
  }
  part[w][lane] = acc;
  __syncthreads();
  if (w == 0 && col < N) {
    float4 s = part[0][lane];
#pragma unroll
    for (int u = 1; u < kReduceWarps; ++u) {
      s.x += part[u][lane].x; s.y += part[u][lane].y;
      s.z += part[u][lane].z; s.w += part[u][lane].w;
    }
    *reinterpret_cast<float4 *>(dst + col) = s;
  }
}

template <int MODE, int K, bool CLUSTER, bool RESID>
const void *pick_exact(bool e) {
  return e ? reinterpret_cast<const void *>(&norm_bwd_kernel<MODE, K, CLUSTER, true, RESID>)
           : reinterpret_cast<const void *>(&norm_bwd_kernel<MODE, K, CLUSTER, false, RESID>);
}

template <int MODE, int K, bool CLUSTER>
const void *pick_variant(bool e, bool r) {
  if (r) return CLUSTER ? nullptr : pick_exact<MODE, K, false, true>(e);  // no cluster variants
  return pick_exact<MODE, K, CLUSTER, false>(e);
}

template <int MODE, bool CLUSTER>
const void *pick_bwd(int K, bool e, bool r) {
  switch (K) {
    case 1: return pick_variant<MODE, 1, CLUSTER>(e, r);
    case 2: return pick_variant<MODE, 2, CLUSTER>(e, r);
    case 3: return pick_variant<MODE, 3, CLUSTER>(e, r);
    case 4: return pick_variant<MODE, 4, CLUSTER>(e, r);
    default: return nullptr;
  }
}

}  // namespace

const void *bwd_kernel_ptr(int mode, int K, bool cluster, bool exact, bool resid) {
  if (mode == kRMS)
    return cluster ? pick_bwd<kRMS, true>(K, exact, resid) : pick_bwd<kRMS, false>(K, exact, resid);
  return cluster ? pick_bwd<kLayer, true>(K, exact, resid)
                 : pick_bwd<kLayer, false>(K, exact, resid);
}

const void *reduce_kernel_ptr() {
  return reinterpret_cast<const void *>(&reduce_partials_kernel);
}

int reduce_threads() { return kReduceWarps * 32; }

const void *selftest_kernel_ptr() {
  return reinterpret_cast<const void *>(&selftest_wait_kernel);
}

}  // namespace gbn
