// group_bwd.cu -- backward group normalisation with an activation (and
// dropout) on channels-last tensors, from the forward's saved statistics:
//   dz = drop(dy) act'(z),  z = xhat gamma + beta,  g = dz gamma,
//   dgamma = sum over (b, s) of dz xhat,  dbeta = sum of dz,
//   dx = rstd (g - mean(g) - xhat mean(g xhat)), means over (s, channels of
//   the group).
// Both group means are sums over the channels of the per-channel sums that
// dgamma and dbeta need, so one set of accumulators serves both.  dz is
// recomputed in the second pass (from x and dy in shared memory or L2)
// rather than kept: kept in 16 bits it would be rounded.
#include "common.cuh"
#include "group.cuh"

namespace gbn {

namespace {

// Per-channel constants of a thread's chunk.
template <int V>
struct BwdConst {
  float2 nmu[V / 2], rs[V / 2], gf[V / 2], bf[V / 2];
};

template <int DT>
__device__ __forceinline__ void load_const(const GroupArgs &a, int b, int chunk,
                                           BwdConst<chunk_elems(DT)> &k) {
  constexpr int V = chunk_elems(DT);
  load_affine<DT>(a, chunk, k.gf, k.bf);
  const int64_t base = static_cast<int64_t>(b) * a.G;
#pragma unroll
  for (int p = 0; p < V / 2; ++p) {
    const int c = chunk * V + 2 * p;
    const int g0 = c / a.D, g1 = (c + 1) / a.D;
    k.nmu[p] = make_float2(-__ldg(a.mean + base + g0), -__ldg(a.mean + base + g1));
    k.rs[p] = make_float2(__ldg(a.rstd + base + g0), __ldg(a.rstd + base + g1));
  }
}

// xhat and dz of one chunk.
template <int DT, int ACT, bool DROP>
__device__ __forceinline__ void grad_chunk(const uint4 &xv, const uint4 &dv,
                                           const BwdConst<chunk_elems(DT)> &k, const DropGen &gen,
                                           int64_t elem, float2 (&xh)[chunk_elems(DT) / 2],
                                           float2 (&dz)[chunk_elems(DT) / 2]) {
  constexpr int V = chunk_elems(DT);
  unpack<DT>(xv, xh);
  unpack<DT>(dv, dz);
  if (DROP) gen.template chunk<V>(dz, static_cast<uint64_t>(elem));
#pragma unroll
  for (int p = 0; p < V / 2; ++p) {
    xh[p] = mul2(add2(xh[p], k.nmu[p]), k.rs[p]);
    if (ACT != kActNone) {
      const float2 z = fma2(xh[p], k.gf[p], k.bf[p]);
      dz[p] = mul2(dz[p], make_float2(act_grad<ACT>(z.x), act_grad<ACT>(z.y)));
    }
  }
}

// dx of one chunk: rstd gamma dz - rstd m1 - xhat (rstd m2), with the group
// constants ra = -rstd m1 and rc = -rstd m2.
template <int DT, int ACT, bool DROP>
__device__ __forceinline__ uint4 dx_chunk(const uint4 &xv, const uint4 &dv,
                                          const BwdConst<chunk_elems(DT)> &k,
                                          const float2 (&ra)[chunk_elems(DT) / 2],
                                          const float2 (&rc)[chunk_elems(DT) / 2],
                                          const DropGen &gen, int64_t elem) {
  constexpr int V = chunk_elems(DT);
  float2 xh[V / 2], dz[V / 2];
  grad_chunk<DT, ACT, DROP>(xv, dv, k, gen, elem, xh, dz);
#pragma unroll
  for (int p = 0; p < V / 2; ++p)
    dz[p] = fma2(xh[p], rc[p], fma2(mul2(dz[p], k.gf[p]), k.rs[p], ra[p]));
  return pack<DT>(dz);
}

// Group constants of the dx pass from gst = (-rstd m1, -rstd m2) per group.
template <int DT>
__device__ __forceinline__ void dx_constants(const GroupArgs &a, const float2 *gst, int g0,
                                             int chunk, float2 (&ra)[chunk_elems(DT) / 2],
                                             float2 (&rc)[chunk_elems(DT) / 2]) {
  constexpr int V = chunk_elems(DT);
#pragma unroll
  for (int p = 0; p < V / 2; ++p) {
    const int c = chunk * V + 2 * p;
    const float2 s0 = gst[c / a.D - g0], s1 = gst[(c + 1) / a.D - g0];
    ra[p] = make_float2(s0.x, s1.x);
    rc[p] = make_float2(s0.y, s1.y);
  }
}

// Sum over a group's D channels of gamma-weighted channel sums, by one warp.
template <int DT>
__device__ __forceinline__ float2 weighted_group(const GroupArgs &a, const float *cb,
                                                 const float *cg, int c0, int c) {
  const int lane = threadIdx.x & 31;
  float s1 = 0.f, s2 = 0.f;
  for (int j = lane; j < a.D; j += 32) {
    const float gm = load_elem<DT>(a.gamma, c0 + c + j);
    s1 = fmaf(gm, cb[c + j], s1);
    s2 = fmaf(gm, cg[c + j], s2);
  }
  return make_float2(warp_sum(s1), warp_sum(s2));
}

template <int V>
__device__ __forceinline__ void put_channels(float *cb, float *cg, int c, const float2 (&s1)[V / 2],
                                             const float2 (&s2)[V / 2]) {
#pragma unroll
  for (int p = 0; p < V / 2; ++p) {
    *reinterpret_cast<float2 *>(cb + c + 2 * p) = s1[p];
    *reinterpret_cast<float2 *>(cg + c + 2 * p) = s2[p];
  }
}

template <int DT, int ACT, bool DROP>
__global__ void __launch_bounds__(kGroupThreads, 1) group_bwd_kernel(const GroupArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int V = chunk_elems(DT);
  const int nthr = blockDim.x;
  const int tid = threadIdx.x;
  const int nact = a.ncs * a.R;  // threads that own a chunk column
  const int unit = static_cast<int>(blockIdx.x) / a.k;
  const int q = static_cast<int>(blockIdx.x) - unit * a.k;
  const int b = unit / a.nslab;
  const int slab = unit - b * a.nslab;
  const int rl = tid / a.ncs;
  const int cc = tid - rl * a.ncs;
  const int chunk0 = slab * a.ncs;
  const int ncs_me = min(a.ncs, a.nc - chunk0);
  const int g0 = slab * a.sg;
  const int ng = min(a.sg, a.G - g0);
  const bool on = rl < a.R && cc < ncs_me;
  const int64_t s0 = part_begin(a.S, q, a.k);
  const int nrow = static_cast<int>(part_begin(a.S, q + 1, a.k) - s0);
  const int nr = (on && rl < nrow) ? (nrow - rl + a.R - 1) / a.R : 0;

  // slot i of this thread: x at data[2 i nact], dy at data[(2 i + 1) nact]
  uint4 *data = reinterpret_cast<uint4 *>(smem) + tid;
  unsigned char *fold = smem + static_cast<size_t>(a.slots) * nact * 32;
  float2 *gst = reinterpret_cast<float2 *>(fold + group_fold_bytes(a.R, a.ncs, V));
  float2 *gfin = gst + a.sg;

  grid_launch_dependents();
  grid_dependency_wait();

  const int64_t e0 = group_elem(a, b, s0 + rl, chunk0 + cc, V);
  const int64_t estep = static_cast<int64_t>(a.R) * a.C;
  const int64_t bstep = estep * elem_bytes(DT);
  const unsigned char *xs = static_cast<const unsigned char *>(a.x) + e0 * elem_bytes(DT);
  const unsigned char *ds = static_cast<const unsigned char *>(a.dy) + e0 * elem_bytes(DT);
  for (int i = 0; i < nr; ++i) {
    cp_async_16(data + static_cast<size_t>(2 * i) * nact, xs + i * bstep);
    cp_async_16(data + static_cast<size_t>(2 * i + 1) * nact, ds + i * bstep);
    if (i & 1) cp_async_commit();
  }
  cp_async_commit();

  BwdConst<V> k;
  if (on) load_const<DT>(a, b, chunk0 + cc, k);
  const DropGen gen(a.drop);
  float2 s1[V / 2], s2[V / 2];
#pragma unroll
  for (int p = 0; p < V / 2; ++p) s1[p] = s2[p] = splat2(0.f);
  auto take = [&](int i) {
    float2 xh[V / 2], dz[V / 2];
    grad_chunk<DT, ACT, DROP>(data[static_cast<size_t>(2 * i) * nact],
                              data[static_cast<size_t>(2 * i + 1) * nact], k, gen, e0 + i * estep,
                              xh, dz);
#pragma unroll
    for (int p = 0; p < V / 2; ++p) {
      s1[p] = add2(s1[p], dz[p]);
      s2[p] = fma2(dz[p], xh[p], s2[p]);
    }
  };
  const int npair = nr >> 1;
  for (int j = 0; j < npair; ++j) {
    cp_async_wait_upto(npair - j);
    take(2 * j);
    take(2 * j + 1);
  }
  cp_async_wait<0>();
  if (nr & 1) take(nr - 1);

  fold_sums<V>(s1, s2, fold, a.R, rl, cc, a.ncs, on);
  float *cb = reinterpret_cast<float *>(fold);  // sum dz per channel
  float *cg = cb + a.ncs * V;                   // sum dz xhat per channel
  if (on && rl == 0) put_channels<V>(cb, cg, cc * V, s1, s2);
  __syncthreads();
  const int ch0 = chunk0 * V;
  for (int g = tid >> 5; g < ng; g += nthr >> 5) {
    const float2 r = weighted_group<DT>(a, cb, cg, ch0, g * a.D);
    if ((tid & 31) == 0) gst[g] = r;
  }
  if (a.k > 1) cluster_sync(); else __syncthreads();
  const float inv = 1.0f / (static_cast<float>(a.S) * static_cast<float>(a.D));
  for (int g = tid; g < ng; g += nthr) {
    float2 t = gst[g];
    if (a.k > 1) {
      t = make_float2(0.f, 0.f);
      for (int r = 0; r < a.k; ++r) t = add2(t, ld_cluster_f2(gst + g, r));
    }
    const float rs = __ldg(a.rstd + static_cast<int64_t>(b) * a.G + g0 + g);
    gfin[g] = make_float2(-rs * (t.x * inv), -rs * (t.y * inv));
  }
  // dgamma / dbeta row of this sample: CTA q sums every k-th channel pair of
  // the slab over the cluster, in rank order.
  for (int j = q * nthr + tid; j < ncs_me * (V / 2); j += a.k * nthr) {
    float2 tg = make_float2(0.f, 0.f), tb = tg;
    const float2 *pg = reinterpret_cast<const float2 *>(cg) + j;
    const float2 *pb = reinterpret_cast<const float2 *>(cb) + j;
    if (a.k == 1) {
      tg = *pg;
      tb = *pb;
    } else {
      for (int r = 0; r < a.k; ++r) {
        tg = add2(tg, ld_cluster_f2(pg, r));
        tb = add2(tb, ld_cluster_f2(pb, r));
      }
    }
    const int64_t at = static_cast<int64_t>(b) * a.C + ch0 + 2 * j;
    *reinterpret_cast<float2 *>(a.cpart + at) = tg;
    if (a.dbeta_part) *reinterpret_cast<float2 *>(a.dbeta_part + at) = tb;
  }
  __syncthreads();
  if (a.k > 1) cluster_arrive_release();

  if (nr) {
    float2 ra[V / 2], rc[V / 2];
    dx_constants<DT>(a, gfin, g0, chunk0 + cc, ra, rc);
    unsigned char *dst = static_cast<unsigned char *>(a.out) + e0 * elem_bytes(DT);
#pragma unroll 2
    for (int i = 0; i < nr; ++i)
      st_global_cs_v4(dst + i * bstep,
                      dx_chunk<DT, ACT, DROP>(data[static_cast<size_t>(2 * i) * nact],
                                              data[static_cast<size_t>(2 * i + 1) * nact], k, ra,
                                              rc, gen, e0 + i * estep));
  }
  if (a.k > 1) cluster_wait_acquire();
}

// Streamed form, first pass: per-channel sums of one row range of one sample
// (a partial row of dgamma and dbeta) and the group sums they add up to.
template <int DT, int ACT, bool DROP>
__global__ void __launch_bounds__(kGroupThreads, 1) group_sums_kernel(const GroupArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int V = chunk_elems(DT);
  const int tid = threadIdx.x;
  const int b = static_cast<int>(blockIdx.x) / a.splits;
  const int sp = static_cast<int>(blockIdx.x) - b * a.splits;
  const int rl = tid / a.ncs;
  const int cc = tid - rl * a.ncs;
  const int64_t s0 = part_begin(a.S, sp, a.splits);
  const int nrow = static_cast<int>(part_begin(a.S, sp + 1, a.splits) - s0);
  float *cb = reinterpret_cast<float *>(smem);
  float *cg = cb + a.C;
  unsigned char *fold = smem + static_cast<size_t>(a.C) * 8;

  grid_launch_dependents();
  grid_dependency_wait();
  const DropGen gen(a.drop);

  for (int col = 0; col < a.nc; col += a.ncs) {
    const bool on = rl < a.R && cc < min(a.ncs, a.nc - col);
    const int nr = (on && rl < nrow) ? (nrow - rl + a.R - 1) / a.R : 0;
    const int64_t c0 = (static_cast<int64_t>(b) * a.S + s0 + rl) * a.nc + col + cc;
    const int64_t step = static_cast<int64_t>(a.R) * a.nc;
    const uint4 *xs = static_cast<const uint4 *>(a.x) + c0;
    const uint4 *ds = static_cast<const uint4 *>(a.dy) + c0;
    float2 s1[V / 2], s2[V / 2];
#pragma unroll
    for (int p = 0; p < V / 2; ++p) s1[p] = s2[p] = splat2(0.f);
    BwdConst<V> k;
    if (on) load_const<DT>(a, b, col + cc, k);
    auto take = [&](const uint4 &xv, const uint4 &dv, int i) {
      float2 xh[V / 2], dz[V / 2];
      grad_chunk<DT, ACT, DROP>(xv, dv, k, gen, (c0 + i * step) * V, xh, dz);
#pragma unroll
      for (int p = 0; p < V / 2; ++p) {
        s1[p] = add2(s1[p], dz[p]);
        s2[p] = fma2(dz[p], xh[p], s2[p]);
      }
    };
    int i = 0;
    for (; i + 4 <= nr; i += 4) {
      uint4 xv[4], dv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        xv[u] = __ldg(xs + (i + u) * step);
        dv[u] = __ldg(ds + (i + u) * step);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) take(xv[u], dv[u], i + u);
    }
    for (; i < nr; ++i) take(__ldg(xs + i * step), __ldg(ds + i * step), i);
    fold_sums<V>(s1, s2, fold, a.R, rl, cc, a.ncs, on);
    if (on && rl == 0) put_channels<V>(cb, cg, (col + cc) * V, s1, s2);
  }
  __syncthreads();
  float2 *out = reinterpret_cast<float2 *>(a.gpart) + static_cast<int64_t>(blockIdx.x) * a.G;
  for (int g = tid >> 5; g < a.G; g += blockDim.x >> 5) {
    const float2 r = weighted_group<DT>(a, cb, cg, 0, g * a.D);
    if ((tid & 31) == 0) out[g] = r;
  }
  float *rg = a.cpart + static_cast<int64_t>(blockIdx.x) * a.C;
  float *rb = a.dbeta_part ? a.dbeta_part + static_cast<int64_t>(blockIdx.x) * a.C : nullptr;
  for (int j = tid; j < a.C / 4; j += blockDim.x) {
    reinterpret_cast<float4 *>(rg)[j] = reinterpret_cast<const float4 *>(cg)[j];
    if (rb) reinterpret_cast<float4 *>(rb)[j] = reinterpret_cast<const float4 *>(cb)[j];
  }
}

// Streamed form, second pass: dx of one row range, last row first.
template <int DT, int ACT, bool DROP>
__global__ void __launch_bounds__(kGroupThreads, 1) group_dx_kernel(const GroupArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int V = chunk_elems(DT);
  const int tid = threadIdx.x;
  const int lane = tid & 31;
  const int b = static_cast<int>(blockIdx.x) / a.splits;
  const int sp = static_cast<int>(blockIdx.x) - b * a.splits;
  const int rl = tid / a.ncs;
  const int cc = tid - rl * a.ncs;
  const int64_t s0 = part_begin(a.S, sp, a.splits);
  const int nrow = static_cast<int>(part_begin(a.S, sp + 1, a.splits) - s0);
  float2 *gfin = reinterpret_cast<float2 *>(smem);

  grid_launch_dependents();
  grid_dependency_wait();

  const float2 *part =
      reinterpret_cast<const float2 *>(a.gpart) + static_cast<int64_t>(b) * a.splits * a.G;
  const float inv = 1.0f / (static_cast<float>(a.S) * static_cast<float>(a.D));
  for (int g = tid >> 5; g < a.G; g += blockDim.x >> 5) {
    float2 t = splat2(0.f);
    for (int r = lane; r < a.splits; r += 32)
      t = add2(t, __ldcg(part + static_cast<int64_t>(r) * a.G + g));
    t.x = warp_sum(t.x);
    t.y = warp_sum(t.y);
    if (lane == 0) {
      const float rs = __ldg(a.rstd + static_cast<int64_t>(b) * a.G + g);
      gfin[g] = make_float2(-rs * (t.x * inv), -rs * (t.y * inv));
    }
  }
  __syncthreads();

  const DropGen gen(a.drop);
  for (int col = 0; col < a.nc; col += a.ncs) {
    if (rl >= a.R || cc >= min(a.ncs, a.nc - col) || rl >= nrow) continue;
    const int nr = (nrow - rl + a.R - 1) / a.R;
    BwdConst<V> k;
    load_const<DT>(a, b, col + cc, k);
    float2 ra[V / 2], rc[V / 2];
    dx_constants<DT>(a, gfin, 0, col + cc, ra, rc);
    const int64_t c0 = (static_cast<int64_t>(b) * a.S + s0 + rl) * a.nc + col + cc;
    const int64_t step = static_cast<int64_t>(a.R) * a.nc;
    const uint4 *xs = static_cast<const uint4 *>(a.x);
    const uint4 *ds = static_cast<const uint4 *>(a.dy);
    uint4 *dst = static_cast<uint4 *>(a.out);
    int i = nr;
    for (; i >= 2; i -= 2) {
      uint4 xv[2], dv[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t c = c0 + (i - 1 - u) * step;
        xv[u] = __ldcs(xs + c);
        dv[u] = __ldcs(ds + c);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t c = c0 + (i - 1 - u) * step;
        st_global_cs_v4(dst + c, dx_chunk<DT, ACT, DROP>(xv[u], dv[u], k, ra, rc, gen, c * V));
      }
    }
    if (i == 1)
      st_global_cs_v4(dst + c0,
                      dx_chunk<DT, ACT, DROP>(__ldcs(xs + c0), __ldcs(ds + c0), k, ra, rc, gen, c0 * V));
  }
}

constexpr int kFormBwd = 0, kFormSums = 1, kFormDx = 2;

template <int DT, int ACT, bool DROP>
const void *pick_form(int form) {
  switch (form) {
    case kFormSums: return reinterpret_cast<const void *>(&group_sums_kernel<DT, ACT, DROP>);
    case kFormDx: return reinterpret_cast<const void *>(&group_dx_kernel<DT, ACT, DROP>);
    default: return reinterpret_cast<const void *>(&group_bwd_kernel<DT, ACT, DROP>);
  }
}

template <int DT>
const void *pick_act(int act, bool drop, int form) {
  switch (act) {
    case kActSilu:
      return drop ? pick_form<DT, kActSilu, true>(form) : pick_form<DT, kActSilu, false>(form);
    case kActGelu:
      return drop ? pick_form<DT, kActGelu, true>(form) : pick_form<DT, kActGelu, false>(form);
    default:
      return drop ? pick_form<DT, kActNone, true>(form) : pick_form<DT, kActNone, false>(form);
  }
}

const void *pick(int dt, int act, bool drop, int form) {
  switch (dt) {
    case kBF16: return pick_act<kBF16>(act, drop, form);
    case kFP16: return pick_act<kFP16>(act, drop, form);
    default: return pick_act<kFP32>(act, drop, form);
  }
}

}  // namespace

const void *group_bwd_kernel_ptr(int dt, int act, bool drop) { return pick(dt, act, drop, kFormBwd); }
const void *group_sums_kernel_ptr(int dt, int act, bool drop) {
  return pick(dt, act, drop, kFormSums);
}
const void *group_dx_kernel_ptr(int dt, int act, bool drop) { return pick(dt, act, drop, kFormDx); }

}  // namespace gbn
