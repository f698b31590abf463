// group_fwd.cu -- forward group normalisation with an activation (and
// dropout) on channels-last tensors: y = drop(act(xhat * gamma + beta)),
// xhat = (x - mean) * rstd with the statistics of each (sample, group).
//
// Resident form: x is read once, so the bytes are the minimum, and what bounds
// it is latency: a call is little more than one wave of CTAs, whose phases
// (copy in, fold, cluster exchange, output) follow each other.  Smaller CTAs,
// several per SM, overlap them; group.cu chooses by an estimate.  8 x 4096 x
// 320 bf16 SiLU: 13.6 us, of which the two passes over HBM need 6.2; copy in
// about 4.3, fold and exchange 2, output 4 to 5, launch 2 (42 MB, 45 % of the
// measured copy bandwidth).  1 x 64 x 1280: 3.4 us.
//
// Streamed form (groups wider than a CTA's 512 chunk columns): x is read twice,
// the second time newest row first, partly from L2.  4 x 4096 x 8192 bf16 in one
// group, SiLU: 159 us (537 MB + a second read of 268 MB; 50 % of the copy
// bandwidth by the minimum bytes).
#include "common.cuh"
#include "group_rows.cuh"

namespace gbn {

namespace {

template <int DT, int ACT, bool DROP>
__global__ void __launch_bounds__(kGroupThreads, 1) group_fwd_kernel(const GroupArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int V = chunk_elems(DT);
  const int tid = threadIdx.x;
  const int nact = a.ncs * a.R;  // threads that own a chunk column
  const int unit = a.by_k(blockIdx.x);
  const int q = static_cast<int>(blockIdx.x) - unit * a.k;
  const int b = a.by_nslab(unit);
  const int slab = unit - b * a.nslab;
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

  uint4 *data = reinterpret_cast<uint4 *>(smem) + tid;  // slot i of this thread: data[i * nact]
  unsigned char *fold = smem + static_cast<size_t>(a.slots) * nact * 16;
  float *chm = reinterpret_cast<float *>(fold + group_fold_bytes(a.R, a.ncs, V));
  float *chq = chm + a.ncs * V;
  float2 *gst = reinterpret_cast<float2 *>(chq + a.ncs * V);
  float2 *gfin = gst + a.sg;

  grid_launch_dependents();
  grid_dependency_wait();

  const int64_t e0 = group_elem(a, b, s0 + rl, chunk0 + cc, V);  // this thread's first element
  const int64_t estep = static_cast<int64_t>(a.R) * a.C;
  const unsigned char *src = static_cast<const unsigned char *>(a.x) + e0 * elem_bytes(DT);
  const int64_t bstep = estep * elem_bytes(DT);
  {
    uint4 *to = data;
    for (int i = 0; i < nr; ++i) {
      cp_async_16(to, src);
      to += nact;
      src += bstep;
      if ((i & 3) == 3) cp_async_commit();
    }
  }
  cp_async_commit();

  AffineRaw aff;  // (their latency hides behind the statistics)
  if (on) aff = load_affine_raw(a, chunk0 + cc);

  // Statistics of this thread's channels, four rows at a time as they land.
  ChannelStats<V> st;
  st.clear();
  const int nblk = nr >> 2;
  for (int j = 0; j < nblk; ++j) {
    cp_async_wait_upto(nblk - j);  // groups after this block's: nblk - j - 1 and the last
    float2 f[4][V / 2];
#pragma unroll
    for (int u = 0; u < 4; ++u) unpack<DT>(data[static_cast<size_t>(4 * j + u) * nact], f[u]);
    st.add4(f[0], f[1], f[2], f[3]);
  }
  cp_async_wait<0>();
  for (int i = 4 * nblk; i < nr; ++i) {
    float2 f[V / 2];
    unpack<DT>(data[static_cast<size_t>(i) * nact], f);
    st.add1(f);
  }

  // Row lanes -> channels -> groups -> cluster.
  channel_stats<V>(st, fold, chm, chq, a.R, rl, cc, a.ncs, on, ncs_me * V,
                   parts.by_rows(q));
  __syncthreads();
  groups_of_channels(a, chm, chq, ng, static_cast<float>(nrow),
                     [&](int g, float m, float m2) { gst[g] = make_float2(m, m2); });
  if (a.k > 1) cluster_sync(); else __syncthreads();
  const float fD = static_cast<float>(a.D);
  // Eight lanes per group, each with the partial of one CTA of the cluster
  // (counts: that CTA's rows, times D): one round trip to the peers' shared
  // memory, and the mean first, then the deviations from it.
  each_group(ng, 3, [&](int g, int r, bool in) {
    const bool mine = in && r < a.k;
    const float2 v = !mine ? make_float2(0.f, 0.f) : a.k == 1 ? gst[g] : ld_cluster_f2(gst + g, r);
    const float n = mine ? static_cast<float>(parts.rows(r)) : 0.f;
    const float m = a.k == 1 ? v.x : a.f_S(lanes_sum(n * v.x, 3));
    const float e = v.x - m;
    const float m2 =
        a.k == 1 ? v.y : lanes_sum(fmaf(n * fD * e, e, v.y), 3);
    if (in && r == 0) {
      const float rs = group_rstd(a, m2);
      gfin[g] = make_float2(m, rs);
      if (q == 0) {
        a.mean[static_cast<int64_t>(b) * a.G + g0 + g] = m;
        a.rstd[static_cast<int64_t>(b) * a.G + g0 + g] = rs;
      }
    }
  });
  __syncthreads();
  if (a.k > 1) cluster_arrive_leave();  // this CTA has read its peers' partials

  if (nr) {
    float2 nmu[V / 2], sc[V / 2], bf[V / 2];
    out_constants<DT>(a, aff, gfin, g0, chunk0 + cc, nmu, sc, bf);
    DropGen gen(a.drop);
    if (DROP) gen.start();
    unsigned char *dst = static_cast<unsigned char *>(a.out) + e0 * elem_bytes(DT);
    const uint4 *at = data;
    int64_t e = e0;
#pragma unroll 2
    for (int left = nr; left > 0; left -= 2) {
      uint4 va = at[0], vb = at[left > 1 ? nact : 0];  // (a last row alone is taken twice)
      out_rows<DT, ACT, DROP>(va, vb, nmu, sc, bf, gen, e, e + estep);
      st_global_cs_v4(dst, va);
      if (left > 1) st_global_cs_v4(dst + bstep, vb);
      at += 2 * nact;
      e += 2 * estep;
      dst += 2 * bstep;
    }
  }
  if (a.k > 1) cluster_wait_acquire();  // no CTA leaves while a peer may read it
}

// Streamed form, first pass: (mean, M2) of every group over one row range of
// one sample.  Chunk columns beyond the CTA's width are taken in turn.
template <int DT>
__global__ void __launch_bounds__(kGroupThreads, 1) group_stats_kernel(const GroupArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int V = chunk_elems(DT);
  const int tid = threadIdx.x;
  const int b = a.by_splits(blockIdx.x);
  const int sp = static_cast<int>(blockIdx.x) - b * a.splits;
  const int rl = a.by_ncs(tid);
  const int cc = tid - rl * a.ncs;
  const Parts parts(a);
  const int s0 = parts.begin(sp), nrow = parts.rows(sp);
  float *chm = reinterpret_cast<float *>(smem);
  float *chq = chm + a.C;
  unsigned char *fold = smem + static_cast<size_t>(a.C) * 8;

  grid_launch_dependents();
  grid_dependency_wait();

  for (int col = 0; col < a.nc; col += a.ncs) {
    const bool on = rl < a.R && cc < min(a.ncs, a.nc - col);
    const int nr = (on && rl < nrow) ? a.by_R(nrow - rl + a.R - 1) : 0;
    const uint4 *src = static_cast<const uint4 *>(a.x) +
                       (static_cast<int64_t>(b) * a.S + s0 + rl) * a.nc + col + cc;
    const int64_t step = static_cast<int64_t>(a.R) * a.nc;
    ChannelStats<V> st;
    st.clear();
    int i = 0;
    for (; i + 8 <= nr; i += 8) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = __ldg(src + (i + u) * step);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 f[4][V / 2];
#pragma unroll
        for (int u = 0; u < 4; ++u) unpack<DT>(v[4 * h + u], f[u]);
        st.add4(f[0], f[1], f[2], f[3]);
      }
    }
    for (; i < nr; ++i) {
      float2 f[V / 2];
      unpack<DT>(__ldg(src + i * step), f);
      st.add1(f);
    }
    channel_stats<V>(st, fold, chm + col * V, chq + col * V, a.R, rl, cc, a.ncs, on,
                     min(a.ncs, a.nc - col) * V, parts.by_rows(sp));
    __syncthreads();  // the fold buffer is free again
  }
  float2 *out = reinterpret_cast<float2 *>(a.gpart) + static_cast<int64_t>(blockIdx.x) * a.G;
  groups_of_channels(a, chm, chq, a.G, static_cast<float>(nrow),
                     [&](int g, float m, float m2) { out[g] = make_float2(m, m2); });
}

// Streamed form, second pass: folds the splits' statistics, then the output
// of one row range, last row first (the first pass read it first row first).
template <int DT, int ACT, bool DROP>
__global__ void __launch_bounds__(kGroupThreads, 1) group_apply_kernel(const GroupArgs a) {
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
    float acc = 0.f;
    for (int r = lane; r < a.splits; r += 32) {
      const float n = static_cast<float>(parts.rows(r));
      acc = fmaf(n, __ldcg(part + static_cast<int64_t>(r) * a.G + g).x, acc);
    }
    const float m = a.f_S(warp_sum(acc));
    float m2 = 0.f;
    for (int r = lane; r < a.splits; r += 32) {
      const float n = static_cast<float>(parts.rows(r)) * static_cast<float>(a.D);
      const float2 v = __ldcg(part + static_cast<int64_t>(r) * a.G + g);
      m2 += fmaf(n * (v.x - m), v.x - m, v.y);
    }
    m2 = warp_sum(m2);
    if (lane == 0) {
      const float rs = group_rstd(a, m2);
      gfin[g] = make_float2(m, rs);
      if (sp == 0) {
        a.mean[static_cast<int64_t>(b) * a.G + g] = m;
        a.rstd[static_cast<int64_t>(b) * a.G + g] = rs;
      }
    }
  }
  __syncthreads();

  DropGen gen(a.drop);
  if (DROP) gen.start();
  for (int col = 0; col < a.nc; col += a.ncs) {
    if (rl >= a.R || cc >= min(a.ncs, a.nc - col) || rl >= nrow) continue;
    const int nr = a.by_R(nrow - rl + a.R - 1);
    float2 nmu[V / 2], sc[V / 2], bf[V / 2];
    out_constants<DT>(a, load_affine_raw(a, col + cc), gfin, 0, col + cc, nmu, sc, bf);
    const int64_t row = static_cast<int64_t>(b) * a.S + s0 + rl;
    const int64_t c0 = row * a.nc + col + cc;
    const int64_t step = static_cast<int64_t>(a.R) * a.nc;
    const uint4 *src = static_cast<const uint4 *>(a.x);
    uint4 *dst = static_cast<uint4 *>(a.out);
    int i = nr;
    for (; i >= 4; i -= 4) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = __ldcs(src + c0 + (i - 1 - u) * step);
#pragma unroll
      for (int u = 0; u < 4; u += 2) {
        const int64_t c = c0 + (i - 1 - u) * step;
        out_rows<DT, ACT, DROP>(v[u], v[u + 1], nmu, sc, bf, gen, c * V, (c - step) * V);
        st_global_cs_v4(dst + c, v[u]);
        st_global_cs_v4(dst + c - step, v[u + 1]);
      }
    }
    for (; i > 0; --i) {
      const int64_t c = c0 + (i - 1) * step;
      uint4 va = __ldcs(src + c), vb = va;
      out_rows<DT, ACT, DROP>(va, vb, nmu, sc, bf, gen, c * V, c * V);
      st_global_cs_v4(dst + c, va);
    }
  }
}

template <int DT, int ACT>
const void *pick_fwd(bool drop, bool streamed) {
  if (streamed)
    return drop ? reinterpret_cast<const void *>(&group_apply_kernel<DT, ACT, true>)
                : reinterpret_cast<const void *>(&group_apply_kernel<DT, ACT, false>);
  return drop ? reinterpret_cast<const void *>(&group_fwd_kernel<DT, ACT, true>)
              : reinterpret_cast<const void *>(&group_fwd_kernel<DT, ACT, false>);
}

template <int DT>
const void *pick_act(int act, bool drop, bool streamed) {
  switch (act) {
    case kActSilu: return pick_fwd<DT, kActSilu>(drop, streamed);
    case kActGelu: return pick_fwd<DT, kActGelu>(drop, streamed);
    default: return pick_fwd<DT, kActNone>(drop, streamed);
  }
}

const void *pick(int dt, int act, bool drop, bool streamed) {
  switch (dt) {
    case kBF16: return pick_act<kBF16>(act, drop, streamed);
    case kFP16: return pick_act<kFP16>(act, drop, streamed);
    default: return pick_act<kFP32>(act, drop, streamed);
  }
}

}  // namespace

const void *group_fwd_kernel_ptr(int dt, int act, bool drop) { return pick(dt, act, drop, false); }
const void *group_apply_kernel_ptr(int dt, int act, bool drop) { return pick(dt, act, drop, true); }

const void *group_stats_kernel_ptr(int dt) {
  switch (dt) {
    case kBF16: return reinterpret_cast<const void *>(&group_stats_kernel<kBF16>);
    case kFP16: return reinterpret_cast<const void *>(&group_stats_kernel<kFP16>);
    default: return reinterpret_cast<const void *>(&group_stats_kernel<kFP32>);
  }
}

}  // namespace gbn
