// group_rows.cuh -- the arithmetic of the group-normalisation passes on one
// chunk column of two rows, shared by their forms (group_fwd.cu,
// group_bwd.cu, group_ring.cu).
#pragma once
#include "group.cuh"

namespace gbn {

// The groups of consecutive channels.
struct GroupWalk {
  int g, left, D;
  __device__ __forceinline__ GroupWalk(const GroupArgs &a, int c)
      : g(a.by_D(c)), left(a.D - (c - g * a.D)), D(a.D) {}
  __device__ __forceinline__ int next() {
    const int r = g;
    if (--left == 0) {
      ++g;
      left = D;
    }
    return r;
  }
};

// A 16-byte chunk taken pair by pair, so that few of its channels are live as
// fp32 at a time.
template <int DT>
struct Pairs {
  uint32_t w[4];
  __device__ __forceinline__ explicit Pairs(const uint4 &c) : w{c.x, c.y, c.z, c.w} {}
  __device__ __forceinline__ uint4 chunk() const { return make_uint4(w[0], w[1], w[2], w[3]); }
  __device__ __forceinline__ float2 get(int p) const {
    if constexpr (DT == kBF16) {
      return bf2_to_f2(w[p]);
    } else if constexpr (DT == kFP16) {
      return __half22float2(*reinterpret_cast<const __half2 *>(&w[p]));
    } else {
      return make_float2(__uint_as_float(w[2 * p]), __uint_as_float(w[2 * p + 1]));
    }
  }
  __device__ __forceinline__ void set(int p, float2 v) {
    if constexpr (DT == kBF16) {
      w[p] = f2_to_bf2(v);
    } else if constexpr (DT == kFP16) {
      const __half2 h = __floats2half2_rn(v.x, v.y);
      w[p] = *reinterpret_cast<const uint32_t *>(&h);
    } else {
      w[2 * p] = __float_as_uint(v.x);
      w[2 * p + 1] = __float_as_uint(v.y);
    }
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
  Pairs<DT> ta(xa), tb(xb);
  float2 fa[V / 2], fb[V / 2];
#pragma unroll
  for (int p = 0; p < V / 2; ++p) {
    fa[p] = fma2(add2(ta.get(p), nmu[p]), sc[p], bf[p]);
    fb[p] = fma2(add2(tb.get(p), nmu[p]), sc[p], bf[p]);
    act_rows<ACT>(fa[p], fb[p]);
    if (!DROP) {
      ta.set(p, fa[p]);
      tb.set(p, fb[p]);
    }
  }
  if (DROP) {
    gen.template chunk<V>(fa, static_cast<uint64_t>(ea));
    gen.template chunk<V>(fb, static_cast<uint64_t>(eb));
    xa = pack<DT>(fa);
    xb = pack<DT>(fb);
  } else {
    xa = ta.chunk();
    xb = tb.chunk();
  }
}

// Per-channel constants of the output pass: -mean, rstd gamma, beta.
// `gst` holds (mean, rstd) of the groups from g0 on.
template <int DT>
__device__ __forceinline__ void out_constants(const GroupArgs &a, const AffineRaw &aff,
                                              const float2 *gst, int g0, int chunk, float2 (&nmu)[chunk_elems(DT) / 2],
                                              float2 (&sc)[chunk_elems(DT) / 2],
                                              float2 (&bf)[chunk_elems(DT) / 2]) {
  constexpr int V = chunk_elems(DT);
  unpack<DT>(aff.g, sc);
  unpack<DT>(aff.b, bf);
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

// What turns a channel's sums of dz and dz d, as sum_rows leaves them, into
// those of dz and dz xhat: the kept elements' factor of the dropout, and with
// it rstd of the channel's group (of sample b; c counts within the tensor).
template <bool DROP>
__device__ __forceinline__ float sum_factor(const GroupArgs &a) {
  return DROP ? a.drop.scale : 1.0f;
}
template <bool DROP>
__device__ __forceinline__ float xhat_factor(const GroupArgs &a, int b, int c) {
  return __ldg(a.rstd + static_cast<int64_t>(b) * a.G + a.by_D(c)) * sum_factor<DROP>(a);
}

// d = x - mean and dz of the same two channels in two rows, from x in ca and
// cb and dy in dza and dzb.  With dropout the dropped elements of dy are 0
// already and dz lacks the kept ones' factor.
template <int ACT>
__device__ __forceinline__ void grad_pairs(float2 nmu, float2 sc, float2 bf, float2 &ca, float2 &dza,
                                           float2 &cb, float2 &dzb) {
  ca = add2(ca, nmu);
  cb = add2(cb, nmu);
  if (ACT != kActNone) {
    float2 za = fma2(ca, sc, bf), zb = fma2(cb, sc, bf);
    act_grad_rows<ACT>(za, zb);
    dza = mul2(dza, za);
    dzb = mul2(dzb, zb);
  }
}

// dx of the same chunk column in two rows, left in xa and xb (dropped elements
// of dy are 0 already).
template <int DT, int ACT, bool DROP>
__device__ __forceinline__ void dx_rows(const GroupArgs &a, uint4 &xa, const uint4 &da, uint4 &xb,
                                        const uint4 &db, const BwdConst<chunk_elems(DT)> &k,
                                        const float2 (&ra)[chunk_elems(DT) / 2],
                                        const float2 (&rc)[chunk_elems(DT) / 2]) {
  Pairs<DT> tx(xa), ux(xb);
  const Pairs<DT> td(da), ud(db);
#pragma unroll
  for (int p = 0; p < chunk_elems(DT) / 2; ++p) {
    float2 ca = tx.get(p), cb = ux.get(p), dza = td.get(p), dzb = ud.get(p);
    grad_pairs<ACT>(k.nmu[p], k.sc[p], k.bf[p], ca, dza, cb, dzb);
    if (DROP) {
      dza = mul2(dza, splat2(a.drop.scale));
      dzb = mul2(dzb, splat2(a.drop.scale));
    }
    tx.set(p, fma2(ca, rc[p], fma2(dza, k.sc[p], ra[p])));
    ux.set(p, fma2(cb, rc[p], fma2(dzb, k.sc[p], ra[p])));
  }
  xa = tx.chunk();
  xb = ux.chunk();
}

// Adds dz and dz d of two rows to the sums.  `two`: the second counts (else
// it is the first again, and its dy is taken as zero).
template <int DT, int ACT>
__device__ __forceinline__ void sum_rows(const uint4 &xa, const uint4 &da, const uint4 &xb,
                                         uint4 db, bool two, const BwdConst<chunk_elems(DT)> &k,
                                         float2 (&s1)[chunk_elems(DT) / 2],
                                         float2 (&s2)[chunk_elems(DT) / 2]) {
  if (!two) db = make_uint4(0, 0, 0, 0);
  const Pairs<DT> tx(xa), ux(xb), td(da), ud(db);
#pragma unroll
  for (int p = 0; p < chunk_elems(DT) / 2; ++p) {
    float2 ca = tx.get(p), cb = ux.get(p), dza = td.get(p), dzb = ud.get(p);
    grad_pairs<ACT>(k.nmu[p], k.sc[p], k.bf[p], ca, dza, cb, dzb);
    s1[p] = add2(s1[p], add2(dza, dzb));
    s2[p] = fma2(dzb, cb, fma2(dza, ca, s2[p]));
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
