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
//
// Bound by instruction latency at 16 warps per SM (128 registers: a chunk
// column's constants and sums stay in them).  A chunk (8 elements of 16 bits)
// costs a thread 95 instructions over both passes, 203 with SiLU, 281 with
// dropout too (22 an element are the formulas' own with SiLU), and a thread about
// 800 more for its start, constants and folds, which 11 rows share at 16 x 1024 x
// 640: half of the issue slots are used, each warp waiting for its own results.
// Resident form: 16 x 1024 x 640 bf16, SiLU and p = 0.1: 33.3 us (63 MB, 28 % of
// the measured copy bandwidth).  2 x 221 x 88 fp16 GELU: 4.6 us in one launch.
// Streamed form: 4 x 4096 x 8192 bf16 in one group, SiLU: 310 us (282 without
// activation).
#include "common.cuh"
#include "group_rows.cuh"

namespace gbn {

namespace {

template <int DT, int ACT, bool DROP>
__global__ void __launch_bounds__(kGroupThreads, 1) group_bwd_kernel(const GroupArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int V = chunk_elems(DT);
  const int nthr = blockDim.x;
  const int tid = threadIdx.x;
  const int nact = a.ncs * a.R;  // threads that own a chunk column
  // A cluster owns a slab of cb samples (one, or all of a small batch), k CTAs
  // each.
  const int csize = a.cb * a.k;
  const int unit = a.by_csize(blockIdx.x);
  const int rank = static_cast<int>(blockIdx.x) - unit * csize;
  const int bl = a.by_k(rank);
  const int q = rank - bl * a.k;
  const int ub = a.by_nslab(unit);
  const int b = ub * a.cb + bl;
  const int slab = unit - ub * a.nslab;
  const int rl = a.by_ncs(tid);
  const int cc = tid - rl * a.ncs;
  const int chunk0 = slab * a.ncs;
  const int ncs_me = min(a.ncs, a.nc - chunk0);
  const int g0 = slab * a.sg;
  const int ng = min(a.sg, a.G - g0);
  const bool on = rl < a.R && cc < ncs_me;
  const Parts parts(a);
  const int s0 = parts.begin(q), nrow = parts.rows(q);
  const int nr = (on && rl < nrow) ? a.by_R(nrow - rl + a.R - 1) : 0;

  // slot i of this thread: x at data[2 i nact], dy at data[(2 i + 1) nact]
  uint4 *data = reinterpret_cast<uint4 *>(smem) + tid;
  unsigned char *fold = smem + static_cast<size_t>(a.slots) * nact * 32;
  float *cb = reinterpret_cast<float *>(fold + group_fold_bytes(a.R, a.ncs, V));
  float *cg = cb + a.ncs * V;  // cb: sum dz per channel, cg: sum dz xhat
  float2 *gst = reinterpret_cast<float2 *>(cg + a.ncs * V);
  float2 *gfin = gst + a.sg;

  grid_launch_dependents();
  grid_dependency_wait();

  const int64_t e0 = group_elem(a, b, s0 + rl, chunk0 + cc, V);
  const int64_t estep = static_cast<int64_t>(a.R) * a.C;
  const int64_t bstep = estep * elem_bytes(DT);
  const unsigned char *xs = static_cast<const unsigned char *>(a.x) + e0 * elem_bytes(DT);
  const unsigned char *ds = static_cast<const unsigned char *>(a.dy) + e0 * elem_bytes(DT);
  {
    uint4 *to = data;
    for (int i = 0; i < nr; ++i) {
      cp_async_16(to, xs);
      cp_async_16(to + nact, ds);
      to += 2 * nact;
      xs += bstep;
      ds += bstep;
      if (i & 1) cp_async_commit();
    }
  }
  cp_async_commit();

  BwdConst<V> k;
  if (on) load_const<DT>(a, b, chunk0 + cc, k);
  DropGen gen(a.drop);
  if (DROP) gen.start();
  float2 s1[V / 2], s2[V / 2];
#pragma unroll
  for (int p = 0; p < V / 2; ++p) s1[p] = s2[p] = splat2(0.f);
  // dy in a slot, its dropped elements zeroed -- in the slot too, so that the
  // dx pass need not ask the generator again.
  auto take_d = [&](uint4 &slot, int64_t e) {
    uint4 v = slot;
    if (DROP) {
      gen.template mask<DT>(v, static_cast<uint64_t>(e));
      slot = v;
    }
    return v;
  };
  const int npair = nr >> 1;
  {
    uint4 *at = data;
    int64_t e = e0;
#pragma unroll 1
    for (int j = npair; j > 0; --j) {
      cp_async_wait_upto(j);
      const uint4 da = take_d(at[nact], e), db = take_d(at[3 * nact], e + estep);
      sum_rows<DT, ACT>(at[0], da, at[2 * nact], db, true, k, s1, s2);
      at += 4 * nact;
      e += 2 * estep;
    }
    cp_async_wait<0>();
    if (nr & 1) {
      const uint4 xv = at[0], dv = take_d(at[nact], e);
      sum_rows<DT, ACT>(xv, dv, xv, dv, false, k, s1, s2);
    }
  }

  const int ch0 = chunk0 * V;
  channel_sums<V>(s1, s2, fold, cb, cg, a.R, rl, cc, a.ncs, on, ncs_me * V, sum_factor<DROP>(a),
                  [&](int j) { return xhat_factor<DROP>(a, b, ch0 + j); });
  __syncthreads();
  group_sums<DT>(a, cb, cg, ch0, ng, [&](int g, float2 v) { gst[g] = v; });
  if (csize > 1) cluster_sync(); else __syncthreads();
  // (eight lanes per group, each with the partial of one CTA of the sample)
  each_group(ng, 3, [&](int g, int r, bool in) {
    float2 t = make_float2(0.f, 0.f);
    if (a.k == 1) {
      if (in) t = gst[g];
    } else {
      if (in && r < a.k) t = ld_cluster_f2(gst + g, bl * a.k + r);
      t.x = lanes_sum(t.x, 3);
      t.y = lanes_sum(t.y, 3);
    }
    if (in && r == 0) {
      const float rs = __ldg(a.rstd + static_cast<int64_t>(b) * a.G + g0 + g);
      gfin[g] = make_float2(-rs * a.f_SD(t.x), -rs * rs * a.f_SD(t.y));
    }
  });
  // dgamma / dbeta row of this cluster's samples: the CTAs share its channel
  // pairs out among them and sum over the cluster in rank order (by the last
  // warps: the first have the groups).  Only sums that are stored are read: the
  // store waits for the peers' values, so none is still on its way when this CTA
  // arrives at the barrier that lets the peers leave.
  const bool want_b = a.dbeta_part != nullptr;
#pragma unroll 1
  for (int j = rank * nthr + nthr - 1 - tid; j < ncs_me * (V / 2); j += csize * nthr) {
    float2 tg = make_float2(0.f, 0.f), tb = tg;
    const float2 *pg = reinterpret_cast<const float2 *>(cg) + j;
    const float2 *pb = reinterpret_cast<const float2 *>(cb) + j;
    if (csize == 1) {
      tg = *pg;
      tb = *pb;
    } else if (want_b) {
      // (at most kMaxGroupCluster: all loads in flight together)
#pragma unroll
      for (int r = 0; r < kMaxGroupCluster; ++r) {
        if (r < csize) {
          tg = add2(tg, ld_cluster_f2(pg, r));
          tb = add2(tb, ld_cluster_f2(pb, r));
        }
      }
    } else {
#pragma unroll
      for (int r = 0; r < kMaxGroupCluster; ++r)
        if (r < csize) tg = add2(tg, ld_cluster_f2(pg, r));
    }
    const int64_t at = static_cast<int64_t>(ub) * a.C + ch0 + 2 * j;
    *reinterpret_cast<float2 *>(a.cpart + at) = tg;
    if (want_b) *reinterpret_cast<float2 *>(a.dbeta_part + at) = tb;
  }
  __syncthreads();
  if (csize > 1) cluster_arrive_leave();

  if (nr) {
    float2 ra[V / 2], rc[V / 2];
    dx_constants<DT>(a, gfin, g0, chunk0 + cc, ra, rc);
    unsigned char *dst = static_cast<unsigned char *>(a.out) + e0 * elem_bytes(DT);
    const uint4 *at = data;
#pragma unroll 1
    for (int left = nr; left > 0; left -= 2) {
      const int o = left > 1 ? 2 * nact : 0;  // (a last row alone is taken twice)
      uint4 xa = at[0], xb = at[o];
      dx_rows<DT, ACT, DROP>(a, xa, at[nact], xb, at[o + nact], k, ra, rc);
      st_global_cs_v4(dst, xa);
      if (left > 1) st_global_cs_v4(dst + bstep, xb);
      at += 4 * nact;
      dst += 2 * bstep;
    }
  }
  if (csize > 1) cluster_wait_acquire();
}

// Streamed form, first pass: per-channel sums of one row range of one sample
// (a partial row of dgamma and dbeta) and the group sums they add up to.
template <int DT, int ACT, bool DROP>
__global__ void __launch_bounds__(kGroupThreads, 1) group_sums_kernel(const GroupArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int V = chunk_elems(DT);
  const int tid = threadIdx.x;
  const int b = a.by_splits(blockIdx.x);
  const int sp = static_cast<int>(blockIdx.x) - b * a.splits;
  const int rl = a.by_ncs(tid);
  const int cc = tid - rl * a.ncs;
  const Parts parts(a);
  const int s0 = parts.begin(sp), nrow = parts.rows(sp);
  float *cb = reinterpret_cast<float *>(smem);
  float *cg = cb + a.C;
  unsigned char *fold = smem + static_cast<size_t>(a.C) * 8;

  grid_launch_dependents();
  grid_dependency_wait();
  DropGen gen(a.drop);
  if (DROP) gen.start();

  for (int col = 0; col < a.nc; col += a.ncs) {
    const bool on = rl < a.R && cc < min(a.ncs, a.nc - col);
    const int nr = (on && rl < nrow) ? a.by_R(nrow - rl + a.R - 1) : 0;
    const int64_t c0 = (static_cast<int64_t>(b) * a.S + s0 + rl) * a.nc + col + cc;
    const int64_t step = static_cast<int64_t>(a.R) * a.nc;
    const uint4 *xs = static_cast<const uint4 *>(a.x) + c0;
    const uint4 *ds = static_cast<const uint4 *>(a.dy) + c0;
    float2 s1[V / 2], s2[V / 2];
#pragma unroll
    for (int p = 0; p < V / 2; ++p) s1[p] = s2[p] = splat2(0.f);
    BwdConst<V> k;
    if (on) load_const<DT>(a, b, col + cc, k);
    int i = 0;
    for (; i + 4 <= nr; i += 4) {
      uint4 xv[4], dv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        xv[u] = __ldg(xs + (i + u) * step);
        dv[u] = __ldg(ds + (i + u) * step);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (DROP) gen.template mask<DT>(dv[u], static_cast<uint64_t>((c0 + (i + u) * step) * V));
#pragma unroll
      for (int u = 0; u < 4; u += 2)
        sum_rows<DT, ACT>(xv[u], dv[u], xv[u + 1], dv[u + 1], true, k, s1, s2);
    }
    for (; i < nr; ++i) {
      const uint4 xv = __ldg(xs + i * step);
      uint4 dv = __ldg(ds + i * step);
      if (DROP) gen.template mask<DT>(dv, static_cast<uint64_t>((c0 + i * step) * V));
      sum_rows<DT, ACT>(xv, dv, xv, dv, false, k, s1, s2);
    }
    channel_sums<V>(s1, s2, fold, cb + col * V, cg + col * V, a.R, rl, cc, a.ncs, on,
                    min(a.ncs, a.nc - col) * V, sum_factor<DROP>(a),
                    [&](int j) { return xhat_factor<DROP>(a, b, col * V + j); });
    __syncthreads();  // the fold buffer is free again
  }
  float2 *out = reinterpret_cast<float2 *>(a.gpart) + static_cast<int64_t>(blockIdx.x) * a.G;
  group_sums<DT>(a, cb, cg, 0, a.G, [&](int g, float2 v) { out[g] = v; });
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
  const int b = a.by_splits(blockIdx.x);
  const int sp = static_cast<int>(blockIdx.x) - b * a.splits;
  const int rl = a.by_ncs(tid);
  const int cc = tid - rl * a.ncs;
  const Parts parts(a);
  const int s0 = parts.begin(sp), nrow = parts.rows(sp);
  float2 *gfin = reinterpret_cast<float2 *>(smem);

  grid_launch_dependents();
  grid_dependency_wait();

  const float2 *part =
      reinterpret_cast<const float2 *>(a.gpart) + static_cast<int64_t>(b) * a.splits * a.G;
  for (int g = tid >> 5; g < a.G; g += blockDim.x >> 5) {
    float2 t = splat2(0.f);
    for (int r = lane; r < a.splits; r += 32)
      t = add2(t, __ldcg(part + static_cast<int64_t>(r) * a.G + g));
    t.x = warp_sum(t.x);
    t.y = warp_sum(t.y);
    if (lane == 0) {
      const float rs = __ldg(a.rstd + static_cast<int64_t>(b) * a.G + g);
      gfin[g] = make_float2(-rs * a.f_SD(t.x), -rs * rs * a.f_SD(t.y));
    }
  }
  __syncthreads();

  DropGen gen(a.drop);
  if (DROP) gen.start();
  for (int col = 0; col < a.nc; col += a.ncs) {
    if (rl >= a.R || cc >= min(a.ncs, a.nc - col) || rl >= nrow) continue;
    const int nr = a.by_R(nrow - rl + a.R - 1);
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
      const int64_t c = c0 + (i - 1) * step;
      if (DROP) {
        gen.template mask<DT>(dv[0], static_cast<uint64_t>(c * V));
        gen.template mask<DT>(dv[1], static_cast<uint64_t>((c - step) * V));
      }
      dx_rows<DT, ACT, DROP>(a, xv[0], dv[0], xv[1], dv[1], k, ra, rc);
      st_global_cs_v4(dst + c, xv[0]);
      st_global_cs_v4(dst + c - step, xv[1]);
    }
    if (i == 1) {
      uint4 xa = __ldcs(xs + c0), xb = xa;
      uint4 dv = __ldcs(ds + c0);
      if (DROP) gen.template mask<DT>(dv, static_cast<uint64_t>(c0 * V));
      dx_rows<DT, ACT, DROP>(a, xa, dv, xb, dv, k, ra, rc);
      st_global_cs_v4(dst + c0, xa);
    }
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
