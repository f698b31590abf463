// group_rows.cuh -- the arithmetic of the group-normalisation passes on one
// chunk column of two rows, shared by their forms (group_fwd.cu,
// group_bwd.cu, group_ring.cu).
#pragma once
#include "group.cuh"

namespace gbn {

// The groups of consecutive channels, with one division for the first.
struct GroupWalk {
  int g, left, D;
  __device__ __forceinline__ GroupWalk(const GroupArgs &a, int c)
      : g(c / a.D), left(a.D - (c - g * a.D)), D(a.D) {}
  __device__ __forceinline__ int next() {
    const int r = g;
    if (--left == 0) {
      ++g;
      left = D;
    }
    return r;
  }
};

// ------------------------------------------------------------- forward
// y of the same chunk column in two rows: z = (x - mean) * (rstd gamma) +
// beta, activation, dropout.
template <int DT, int ACT, bool DROP>
__device__ __forceinline__ void out_rows(uint4 &xa, uint4 &xb, const float2 (&nmu)[chunk_elems(DT) / 2],
                                         const float2 (&sc)[chunk_elems(DT) / 2],
                                         const float2 (&bf)[chunk_elems(DT) / 2],
                                         const DropGen &gen, int64_t ea, int64_t eb) {
  constexpr int V = chunk_elems(DT);
  float2 fa[V / 2], fb[V / 2];
  unpack<DT>(xa, fa);
  unpack<DT>(xb, fb);
#pragma unroll
  for (int p = 0; p < V / 2; ++p) {
    fa[p] = fma2(add2(fa[p], nmu[p]), sc[p], bf[p]);
    fb[p] = fma2(add2(fb[p], nmu[p]), sc[p], bf[p]);
    act_rows<ACT>(fa[p], fb[p]);
  }
  if (DROP) {
    gen.template chunk<V>(fa, static_cast<uint64_t>(ea));
    gen.template chunk<V>(fb, static_cast<uint64_t>(eb));
  }
  xa = pack<DT>(fa);
  xb = pack<DT>(fb);
}

// Per-channel constants of the output pass: -mean, rstd gamma, beta.
// `gst` holds (mean, rstd) of the groups from g0 on.
template <int DT>
__device__ __forceinline__ void out_constants(const GroupArgs &a, const float2 *gst, int g0,
                                              int chunk, float2 (&nmu)[chunk_elems(DT) / 2],
                                              float2 (&sc)[chunk_elems(DT) / 2],
                                              float2 (&bf)[chunk_elems(DT) / 2]) {
  constexpr int V = chunk_elems(DT);
  load_affine<DT>(a, chunk, sc, bf);
  GroupWalk g(a, chunk * V);
#pragma unroll
  for (int p = 0; p < V / 2; ++p) {
    const float2 s0 = gst[g.next() - g0], s1 = gst[g.next() - g0];
    nmu[p] = make_float2(-s0.x, -s1.x);
    sc[p] = mul2(sc[p], make_float2(s0.y, s1.y));
  }
}

// ------------------------------------------------------------ backward
// Per-channel constants of a thread's chunk: -mean, rstd gamma and beta.  With
// d = x - mean, z = d (rstd gamma) + beta; the sums are taken of dz and dz d
// (rstd, constant over them, goes in once at the end), and dx = dz (rstd
// gamma) + ra + d rc with ra = -rstd m1 and rc = -rstd^2 m2: three operations
// fewer per element than by way of xhat.
template <int V>
struct BwdConst {
  float2 nmu[V / 2], sc[V / 2], bf[V / 2];
};

template <int DT>
__device__ __forceinline__ void load_const(const GroupArgs &a, int b, int chunk,
                                           BwdConst<chunk_elems(DT)> &k) {
  constexpr int V = chunk_elems(DT);
  load_affine<DT>(a, chunk, k.sc, k.bf);
  const int64_t base = static_cast<int64_t>(b) * a.G;
  GroupWalk g(a, chunk * V);
#pragma unroll
  for (int p = 0; p < V / 2; ++p) {
    const int g0 = g.next(), g1 = g.next();
    k.nmu[p] = make_float2(-__ldg(a.mean + base + g0), -__ldg(a.mean + base + g1));
    k.sc[p] = mul2(k.sc[p], make_float2(__ldg(a.rstd + base + g0), __ldg(a.rstd + base + g1)));
  }
}

// Sums of dz and dz d as sum_rows leaves them -> sums of dz and dz xhat.
template <int DT, bool DROP>
__device__ __forceinline__ void scale_sums(const GroupArgs &a, int b, int chunk,
                                           float2 (&s1)[chunk_elems(DT) / 2],
                                           float2 (&s2)[chunk_elems(DT) / 2]) {
  const float *rs = a.rstd + static_cast<int64_t>(b) * a.G;
  GroupWalk g(a, chunk * chunk_elems(DT));
#pragma unroll
  for (int p = 0; p < chunk_elems(DT) / 2; ++p) {
    const int g0 = g.next(), g1 = g.next();
    s2[p] = mul2(s2[p], make_float2(__ldg(rs + g0), __ldg(rs + g1)));
    if (DROP) {
      s1[p] = mul2(s1[p], splat2(a.drop.scale));
      s2[p] = mul2(s2[p], splat2(a.drop.scale));
    }
  }
}

// d = x - mean and dz of the same chunk column in two rows.  With dropout the
// dropped elements of dy are 0 already and dz lacks the kept ones' factor.
template <int DT, int ACT>
__device__ __forceinline__ void grad_rows(
    const uint4 &xa, const uint4 &da, const uint4 &xb, const uint4 &db,
    const BwdConst<chunk_elems(DT)> &k, float2 (&ca)[chunk_elems(DT) / 2],
    float2 (&dza)[chunk_elems(DT) / 2], float2 (&cb)[chunk_elems(DT) / 2],
    float2 (&dzb)[chunk_elems(DT) / 2]) {
  constexpr int V = chunk_elems(DT);
  unpack<DT>(xa, ca);
  unpack<DT>(da, dza);
  unpack<DT>(xb, cb);
  unpack<DT>(db, dzb);
#pragma unroll
  for (int p = 0; p < V / 2; ++p) {
    ca[p] = add2(ca[p], k.nmu[p]);
    cb[p] = add2(cb[p], k.nmu[p]);
    if (ACT != kActNone) {
      float2 za = fma2(ca[p], k.sc[p], k.bf[p]), zb = fma2(cb[p], k.sc[p], k.bf[p]);
      act_grad_rows<ACT>(za, zb);
      dza[p] = mul2(dza[p], za);
      dzb[p] = mul2(dzb[p], zb);
    }
  }
}

// dx of the same chunk column in two rows, left in xa and xb (dropped elements
// of dy are 0 already).
template <int DT, int ACT, bool DROP>
__device__ __forceinline__ void dx_rows(const GroupArgs &a, uint4 &xa, const uint4 &da, uint4 &xb,
                                        const uint4 &db, const BwdConst<chunk_elems(DT)> &k,
                                        const float2 (&ra)[chunk_elems(DT) / 2],
                                        const float2 (&rc)[chunk_elems(DT) / 2]) {
  constexpr int V = chunk_elems(DT);
  float2 ca[V / 2], dza[V / 2], cb[V / 2], dzb[V / 2];
  grad_rows<DT, ACT>(xa, da, xb, db, k, ca, dza, cb, dzb);
#pragma unroll
  for (int p = 0; p < V / 2; ++p) {
    if (DROP) {
      dza[p] = mul2(dza[p], splat2(a.drop.scale));
      dzb[p] = mul2(dzb[p], splat2(a.drop.scale));
    }
    dza[p] = fma2(ca[p], rc[p], fma2(dza[p], k.sc[p], ra[p]));
    dzb[p] = fma2(cb[p], rc[p], fma2(dzb[p], k.sc[p], ra[p]));
  }
  xa = pack<DT>(dza);
  xb = pack<DT>(dzb);
}

// Adds dz and dz d of two rows (`two`: the second counts) to the sums.
template <int DT, int ACT>
__device__ __forceinline__ void sum_rows(const uint4 &xa, const uint4 &da, const uint4 &xb,
                                         const uint4 &db, bool two,
                                         const BwdConst<chunk_elems(DT)> &k,
                                         float2 (&s1)[chunk_elems(DT) / 2],
                                         float2 (&s2)[chunk_elems(DT) / 2]) {
  constexpr int V = chunk_elems(DT);
  float2 ca[V / 2], dza[V / 2], cb[V / 2], dzb[V / 2];
  grad_rows<DT, ACT>(xa, da, xb, db, k, ca, dza, cb, dzb);
#pragma unroll
  for (int p = 0; p < V / 2; ++p) {
    s1[p] = add2(s1[p], dza[p]);
    s2[p] = fma2(dza[p], ca[p], s2[p]);
  }
  if (two) {
#pragma unroll
    for (int p = 0; p < V / 2; ++p) {
      s1[p] = add2(s1[p], dzb[p]);
      s2[p] = fma2(dzb[p], cb[p], s2[p]);
    }
  }
}

// Group constants of the dx pass from gst = (ra, rc) per group.
template <int DT>
__device__ __forceinline__ void dx_constants(const GroupArgs &a, const float2 *gst, int g0,
                                             int chunk, float2 (&ra)[chunk_elems(DT) / 2],
                                             float2 (&rc)[chunk_elems(DT) / 2]) {
  constexpr int V = chunk_elems(DT);
  GroupWalk g(a, chunk * V);
#pragma unroll
  for (int p = 0; p < V / 2; ++p) {
    const float2 s0 = gst[g.next() - g0], s1 = gst[g.next() - g0];
    ra[p] = make_float2(s0.x, s1.x);
    rc[p] = make_float2(s0.y, s1.y);
  }
}

// Gamma-weighted sums over each group of the per-channel sums of dz (cb) and
// dz xhat (cg), handed to out(g, sums) by one lane per group.  ch0: the
// slab's first channel.
template <int DT, typename Out>
__device__ __forceinline__ void group_sums(const GroupArgs &a, const float *cb, const float *cg,
                                           int ch0, int ng, Out out) {
  each_group(ng, a.lsh, [&](int g, int l, bool in) {
    float s1 = 0.f, s2 = 0.f;
    if (in) {
#pragma unroll 1
      for (int j = g * a.D + l; j < (g + 1) * a.D; j += 1 << a.lsh) {
        const float gm = load_elem<DT>(a.gamma, ch0 + j);
        s1 = fmaf(gm, cb[j], s1);
        s2 = fmaf(gm, cg[j], s2);
      }
    }
    s1 = lanes_sum(s1, a.lsh);
    s2 = lanes_sum(s2, a.lsh);
    if (in && l == 0) out(g, make_float2(s1, s2));
  });
}

}  // namespace gbn
