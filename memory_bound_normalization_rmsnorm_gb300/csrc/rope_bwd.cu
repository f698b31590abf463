// rope_bwd.cu -- backward of the head normalisation and rotation (rope.cuh).
//
//   dn = dy turned back,  g = dn gamma,  xhat = (x - mean) rstd
//   dx = rstd (g - mean(g) - xhat mean(g xhat))   (mean(g) for LayerNorm only)
//   dgamma = sum of dn xhat,  dbeta = sum of dn over all rows of the side
//
// The statistics are taken again from x, which has to be read anyway: nothing
// is kept from the forward pass.  Each CTA works on one side (queries or keys),
// so that a thread's running sums are those of one gamma; they are joined over
// the CTA in a fixed order, and rope_fold_kernel adds the CTAs' rows in order.
#include <cuda_runtime.h>

#include "rope.cuh"

namespace gbn {

namespace {

constexpr int kRopeBwdBatch = 2;  // rows in flight per thread

template <int DT, int V, int MODE>
__global__ void __launch_bounds__(kRopeThreads) rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int NU = rope_units(V);
  constexpr int B = kRopeBwdBatch;
  __shared__ uint64_t turns[kRopeMaxD / 2];
  extern __shared__ float fold[];
  grid_launch_dependents();
  grid_dependency_wait();
  rope_table(a, turns);
  __syncthreads();
  const RopeLane<V> l(a);
  const int warps = kRopeThreads / 32, warp = threadIdx.x / 32;
  const int side = static_cast<int>(blockIdx.x) >= a.ctas[0] ? 1 : 0;
  const RopeSide &s = a.side[side];
  const int cta = static_cast<int>(blockIdx.x) - (side ? a.ctas[0] : 0);
  const int chunks = a.chunks[side];
  const int64_t items = a.T * chunks;
  float g[NU][2 * V], dg[NU][2 * V], db[NU][2 * V];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    RopeVec<DT, V> v;
    v.zero();
    if (l.in1[i]) v.load(s.gamma, l.o1[i]);
    v.get(g[i]);
    v.zero();
    if (l.in2[i]) v.load(s.gamma, l.o2[i]);
    v.get(g[i] + V);
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) dg[i][e] = db[i][e] = 0.f;
  }
  for (int64_t item = static_cast<int64_t>(cta) * warps + warp; item < items;
       item += static_cast<int64_t>(a.ctas[side]) * warps) {
    const int64_t t = item / chunks;
    const int c = static_cast<int>(item - t * chunks);
    RopeAngles<V> ang;
    ang.at(a, l, turns, t);
    const int r0 = s.rounds * c / chunks, r1 = s.rounds * (c + 1) / chunks;
    for (int r = r0; r < r1; r += B) {
      RopeVec<DT, V> vx[B][NU][2], vd[B][NU][2];
#pragma unroll
      for (int n = 0; n < B; ++n) {
        const int h = ((r + n) << (5 - a.lanes_log2)) + l.group;
        const bool row = r + n < r1 && h < s.H;
        const int64_t ax = t * s.xt + h * s.xh, ad = t * s.dt + h * s.dh;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            vx[n][i][k].zero();
            vd[n][i][k].zero();
            if (row && (k ? l.in2[i] : l.in1[i])) {
              vx[n][i][k].load(s.x, ax + (k ? l.o2[i] : l.o1[i]));
              vd[n][i][k].load(s.dy, ad + (k ? l.o2[i] : l.o1[i]));
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < B; ++n) {
        if (r + n >= r1) break;
        const int h = ((r + n) << (5 - a.lanes_log2)) + l.group;
        float f[NU][2 * V], d[NU][2 * V];
#pragma unroll
        for (int i = 0; i < NU; ++i) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            vx[n][i][k].get(f[i] + k * V);
            vd[n][i][k].get(d[i] + k * V);
          }
          if (l.pair[i] >= 0) {
            if (a.inter)
              ang.turn(i, true, d[i]);
            else
              ang.turn(i, false, d[i]);
          }
        }
        const float rstd = rope_stats<MODE, V>(a, l, f);
        // Lanes beyond the last head hold zeros; with eps = 0 their rstd is infinite.
        const float rs = h < s.H ? rstd : 0.f;
        float c1 = 0.f, c0 = 0.f;
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) {
            f[i][e] *= rs;  // xhat
            dg[i][e] = fmaf(d[i][e], f[i][e], dg[i][e]);
            if (MODE == kLayer) db[i][e] += d[i][e];
            d[i][e] *= g[i][e];
            c1 = fmaf(d[i][e], f[i][e], c1);
            if (MODE == kLayer) c0 += d[i][e];
          }
        c1 = rope_sum(c1, a.lanes_log2) * a.invD;
        if (MODE == kLayer) c0 = rope_sum(c0, a.lanes_log2) * a.invD;
        if (h >= s.H) continue;
        const int64_t at = t * s.ot + h * s.oh;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) {
            const float m = MODE == kLayer ? d[i][e] - c0 : d[i][e];
            d[i][e] = rs * fmaf(-f[i][e], c1, m);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            vd[n][i][k].set(d[i] + k * V);
            if (k ? l.in2[i] : l.in1[i]) vd[n][i][k].store(s.out, at + (k ? l.o2[i] : l.o1[i]));
          }
        }
      }
    }
  }
  // The warp's groups first (lanes that hold the same elements), then the warps.
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        if (o >= (1 << a.lanes_log2)) {
          dg[i][e] += __shfl_xor_sync(0xffffffffu, dg[i][e], o);
          if (MODE == kLayer) db[i][e] += __shfl_xor_sync(0xffffffffu, db[i][e], o);
        }
      }
      if (l.group == 0 && (e < V ? l.in1[i] : l.in2[i])) {
        const int at = warp * a.D + (e < V ? l.o1[i] + e : l.o2[i] + e - V);
        fold[at] = dg[i][e];
        if (MODE == kLayer) fold[warps * a.D + at] = db[i][e];
      }
    }
  __syncthreads();
  const int n = a.D * (MODE == kLayer ? 2 : 1);
  for (int i = threadIdx.x; i < n; i += kRopeThreads) {
    const int which = i >= a.D, e = i - which * a.D;
    float v = 0.f;
    for (int w = 0; w < warps; ++w) v += fold[(which * warps + w) * a.D + e];
    a.part[(static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * a.D + e] = v;
  }
}

// Adds the CTAs' rows: block y = 0 dgamma of q, 1 of k, 2 and 3 dbeta of them;
// 32 columns per block, 32 rows side by side, joined in order.
__global__ void __launch_bounds__(1024)
    rope_fold_kernel(const float *part, int n, int cq, int ck, float *dgq, float *dgk, float *dbq,
                     float *dbk) {
  __shared__ float sum[32][33];
  grid_launch_dependents();
  grid_dependency_wait();
  const int which = blockIdx.y >> 1, side = blockIdx.y & 1;
  float *out = which ? (side ? dbk : dbq) : (side ? dgk : dgq);
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x / 32;
  const int rows = side ? ck : cq;
  const float *src = part + (static_cast<int64_t>(which) * (cq + ck) + (side ? cq : 0)) * n;
  float v = 0.f;
  if (out && col < n) {
#pragma unroll 4
    for (int r = row; r < rows; r += 32) v += __ldcg(src + static_cast<int64_t>(r) * n + col);
  }
  sum[row][threadIdx.x & 31] = v;
  __syncthreads();
  if (row == 0 && out && col < n) {
    v = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) v += sum[r][threadIdx.x & 31];
    out[col] = v;
  }
}

template <int DT, int V>
const void *pick_mode(int mode) {
  return mode == kLayer ? reinterpret_cast<const void *>(&rope_bwd_kernel<DT, V, kLayer>)
                        : reinterpret_cast<const void *>(&rope_bwd_kernel<DT, V, kRMS>);
}

template <int DT>
const void *pick_width(int V, int mode) {
  switch (V) {
    case 8:
      if constexpr (DT != kFP32) return pick_mode<DT, 8>(mode);
      return nullptr;
    case 4: return pick_mode<DT, 4>(mode);
    case 2: return pick_mode<DT, 2>(mode);
    default: return pick_mode<DT, 1>(mode);
  }
}

}  // namespace

const void *rope_bwd_kernel_ptr(int dt, int V, int mode) {
  switch (dt) {
    case kBF16: return pick_width<kBF16>(V, mode);
    case kFP16: return pick_width<kFP16>(V, mode);
    default: return pick_width<kFP32>(V, mode);
  }
}

const void *rope_fold_kernel_ptr() { return reinterpret_cast<const void *>(&rope_fold_kernel); }

}  // namespace gbn
