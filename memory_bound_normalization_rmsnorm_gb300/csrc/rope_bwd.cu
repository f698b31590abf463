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

#include "fold.cuh"
#include "rope.cuh"

namespace gbn {

namespace {

template <int DT, int V, int MODE, int MIX>
__global__ void __launch_bounds__(kRopeThreads, kRopeBwdCtas)
    rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int NU = rope_units(V), NP = RopeUnit<V>::NP, S = kRopeBwdStages;
  constexpr int es = elem_bytes(DT);
  extern __shared__ uint4 smem[];
  RopeShared &sh = *reinterpret_cast<RopeShared *>(smem);
  uint4 *ring_mem = smem + sizeof(RopeShared) / 16;  // the ring, then the fold of the sums
  float *fold = reinterpret_cast<float *>(ring_mem);
  grid_launch_dependents();
  grid_dependency_wait();
  const int warps = kRopeThreads / 32, warp = threadIdx.x / 32;
  const int side = static_cast<int>(blockIdx.x) >= a.ctas[0] ? 1 : 0;
  const RopeSide &s = a.side[side];
  const RopeLane<DT, V, NU, MIX> l(a);
  const int groups = 32 >> a.lanes_log2;
  const int first = warp * groups + l.group, per = warps * groups;
  RopeTiles<V> tile;
  tile.start(a, side, static_cast<int>(blockIdx.x) - (side ? a.ctas[0] : 0));
  RopeRing<DT, V, NU, MIX, 2, S> ring;
  ring.start(a, side, l, ring_mem, tile.t, first, per);
  for (int n = 0; n < S - 1; ++n) ring.fetch(a, side, l, first, per);
  RopeVec<DT, V> g[NU][2];
  l.load(g, static_cast<const char *>(s.gamma), true);
  RopeRow<1> out;
  {
    const void *base = s.out;
    out.start<DT>(a, side, &base, &s.ot, &s.oh, first, per);
  }
  RopeUnit<V> dg[NU], db[NU];
  l.param(dg, nullptr);
  l.param(db, nullptr);
  for (; tile.any(a); tile.t += tile.step) {
    tile.angles(a, side, sh);
    out.at(tile.t);
    for (int left = tile.n * s.H; left > 0; left -= per) {
      const bool on = first < left;
      RopeUnit<V> f[NU], d[NU];
      RopeVec<DT, V> v[NU][2];
      ring.template wait<S - 2>();
      ring.read(v, 0);
      l.get(f, v);
      ring.read(v, 1);
      l.get(d, v);
      if (MIX != kMixed) ring.step();  // else trade needs the round's slots
      ring.fetch(a, side, l, first, per);
      {
        RopeAngles<V, NU> ang;
        ang.get(a, l, sh.cs + (on ? out.tok * 2 * a.pairs : 0));
#pragma unroll
        for (int i = 0; i < NU; ++i)
          if (l.pair[i] >= 0) ang.turn(i, d[i]);
      }
      // Lanes beyond the last head hold zeros; with eps = 0 their rstd is infinite.
      const float rstd = rope_stats<MODE>(a, l, f);
      const float rs = on ? rstd : 0.f;
      RopeUnit<V> gf[NU];
      l.get(gf, g);
      float2 s1 = make_float2(0.f, 0.f), s0 = s1;
#pragma unroll
      for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int e = 0; e < 2 * NP; ++e) {
          float2 &x = e < NP ? f[i].u[e] : f[i].w[e - NP], &y = e < NP ? d[i].u[e] : d[i].w[e - NP];
          float2 &sg = e < NP ? dg[i].u[e] : dg[i].w[e - NP];
          x = mul2(x, splat2(rs));  // xhat
          sg = fma2(y, x, sg);
          if (MODE == kLayer) {
            float2 &sb = e < NP ? db[i].u[e] : db[i].w[e - NP];
            sb = add2(sb, y);
          }
          y = mul2(y, e < NP ? gf[i].u[e] : gf[i].w[e - NP]);
          s1 = fma2(y, x, s1);
          if (MODE == kLayer) s0 = add2(s0, y);
        }
      // dx = rstd g - rstd mean(g) - xhat (rstd mean(g xhat))
      const float2 c1 = splat2(-rs * (rope_sum(s1.x + s1.y, a.lanes_log2) * a.invD));
      float2 c0 = make_float2(0.f, 0.f);
      if (MODE == kLayer) c0 = splat2(-rs * (rope_sum(s0.x + s0.y, a.lanes_log2) * a.invD));
      RopeVec<DT, V> o[NU][2];
#pragma unroll
      for (int i = 0; i < NU; ++i) {
#pragma unroll
        for (int e = 0; e < 2 * NP; ++e) {
          float2 &x = e < NP ? f[i].u[e] : f[i].w[e - NP], &y = e < NP ? d[i].u[e] : d[i].w[e - NP];
          y = fma2(y, splat2(rs), MODE == kLayer ? fma2(x, c1, c0) : mul2(x, c1));
        }
        d[i].template set<MIX>(o[i], l.mix[i]);
      }
      if (MIX == kMixed) {
        ring.trade(o);
        ring.step();
      }
      if (on) l.store(o, const_cast<char *>(out.p[0]));
      out.next();
    }
  }
  __syncthreads();  // every round has been read
  // The warp's groups first (lanes that hold the same elements), then the warps.
  const auto join = [&](RopeUnit<V> (&u)[NU], float *out) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
#pragma unroll
      for (int e = 0; e < 2 * NP; ++e) {
        float2 &x = e < NP ? u[i].u[e] : u[i].w[e - NP];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          if (o >= (1 << a.lanes_log2)) {
            x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
            x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
          }
        }
      }
      if (l.group != 0) continue;
      const int e1 = l.o1[i] / es, e2 = l.o2[i] / es;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float x = e & 1 ? u[i].u[e / 2].y : u[i].u[e / 2].x;
        const float y = e & 1 ? u[i].w[e / 2].y : u[i].w[e / 2].x;
        if (V > 1 && rope_mixed(MIX, l.mix[i])) {  // neighbours
          if (2 * e < V ? l.in1[i] : l.in2[i]) {
            const int at = 2 * e < V ? e1 + 2 * e : e2 + 2 * e - V;
            out[at] = x;
            out[at + 1] = y;
          }
        } else {
          if (l.in1[i]) out[e1 + e] = x;
          if (l.in2[i]) out[e2 + e] = y;
        }
      }
    }
  };
  join(dg, fold + warp * a.D);
  if (MODE == kLayer) join(db, fold + (warps + warp) * a.D);
  __syncthreads();
  const int n = a.D * (MODE == kLayer ? 2 : 1);
  for (int i = threadIdx.x; i < n; i += kRopeThreads) {
    const int which = i >= a.D, e = i - which * a.D;
    float v = 0.f;
    for (int w = 0; w < warps; ++w) v += fold[(which * warps + w) * a.D + e];
    a.part[(static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * a.D + e] = v;
  }
}

// Adds the CTAs' rows: block y = 0 dgamma of q, 1 of k, 2 and 3 dbeta of them.
__global__ void __launch_bounds__(1024)
    rope_fold_kernel(const float *part, int n, int cq, int ck, float *dgq, float *dgk, float *dbq,
                     float *dbk) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int which = blockIdx.y >> 1, side = blockIdx.y & 1;
  float *out = which ? (side ? dbk : dbq) : (side ? dgk : dgq);
  const float *src = part + (static_cast<int64_t>(which) * (cq + ck) + (side ? cq : 0)) * n;
  fold_columns(src, side ? ck : cq, n, out);
}

template <int DT, int V, int MIX>
const void *pick_mode(int mode) {
  return mode == kLayer ? reinterpret_cast<const void *>(&rope_bwd_kernel<DT, V, kLayer, MIX>)
                        : reinterpret_cast<const void *>(&rope_bwd_kernel<DT, V, kRMS, MIX>);
}

template <int DT, int V>
const void *pick_mix(int mode, bool inter) {
  return inter ? pick_mode<DT, V, kMixed>(mode) : pick_mode<DT, V, kApart>(mode);
}

template <int DT>
const void *pick_width(int V, int mode, bool inter) {
  switch (V) {
    case 8:
      if constexpr (DT != kFP32) return pick_mix<DT, 8>(mode, inter);
      return nullptr;
    case 4: return pick_mix<DT, 4>(mode, inter);
    case 2: return pick_mode<DT, 2, kEither>(mode);
    default: return pick_mode<DT, 1, kApart>(mode);
  }
}

}  // namespace

const void *rope_bwd_kernel_ptr(int dt, int V, int mode, bool inter) {
  switch (dt) {
    case kBF16: return pick_width<kBF16>(V, mode, inter);
    case kFP16: return pick_width<kFP16>(V, mode, inter);
    default: return pick_width<kFP32>(V, mode, inter);
  }
}

const void *rope_fold_kernel_ptr() { return reinterpret_cast<const void *>(&rope_fold_kernel); }

}  // namespace gbn
