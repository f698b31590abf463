// rope.cu -- forward of the head normalisation and rotation (rope.cuh), and the
// entry points norm_rope_fwd / norm_rope_bwd.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/gbnorm.h"
#include "common.cuh"
#include "host_util.h"
#include "rope.cuh"

namespace gbn {

namespace {

// One pass: read a row, normalise it in registers, turn its pairs, write it.
template <int DT, int V, int NU, int MODE, int MIX>
__global__ void __launch_bounds__(kRopeThreads, rope_fwd_ctas(MODE, V, NU, MIX == kMixed))
    rope_fwd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int NP = RopeUnit<V>::NP, S = rope_fwd_stages(NU);
  extern __shared__ uint4 smem[];
  RopeShared &sh = *reinterpret_cast<RopeShared *>(smem);
  uint4 *ring_mem = smem + sizeof(RopeShared) / 16;
  grid_launch_dependents();
  grid_dependency_wait();
  const int side = static_cast<int>(blockIdx.x) >= a.ctas[0] ? 1 : 0;
  const RopeSide &s = a.side[side];
  const RopeLane<DT, V, NU, MIX> l(a);
  const int groups = 32 >> a.lanes_log2;
  const int first = threadIdx.x / 32 * groups + l.group, per = kRopeThreads / 32 * groups;
  RopeTiles<V> tile;
  tile.start(a, side, static_cast<int>(blockIdx.x) - (side ? a.ctas[0] : 0));
  RopeRing<DT, V, NU, MIX, 1, S> ring;
  ring.start(a, side, l, ring_mem, tile.t, first, per);
  for (int n = 0; n < S - 1; ++n) ring.fetch(a, side, l, first, per);
  RopeUnit<V> g[NU];
  RopeVec<DT, V> b[NU][2];
  if (MODE != kNoNorm) l.param(g, s.gamma);
  if (MODE == kLayer) l.load(b, static_cast<const char *>(s.beta), s.beta != nullptr);
  RopeRow<1> out;
  {
    const void *base = s.out;
    out.start<DT>(a, side, &base, &s.ot, &s.oh, first, per);
  }
  for (; tile.any(a); tile.t += tile.step) {
    tile.angles(a, side, sh);
    out.at(tile.t);
    for (int left = tile.n * s.H; left > 0; left -= per) {
      RopeUnit<V> f[NU];
      RopeVec<DT, V> o[NU][2];
      ring.template wait<S - 2>();
      ring.read(o, 0);
      l.get(f, o);
      if (MIX != kMixed) ring.step();  // else trade needs the round's slots
      ring.fetch(a, side, l, first, per);
      if constexpr (MODE != kNoNorm) {
        const float2 rstd = splat2(rope_stats<MODE>(a, l, f));
        RopeUnit<V> bf[NU];
        if (MODE == kLayer) l.get(bf, b);
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            const float2 u = mul2(f[i].u[e], rstd), w = mul2(f[i].w[e], rstd);
            f[i].u[e] = MODE == kLayer ? fma2(u, g[i].u[e], bf[i].u[e]) : mul2(u, g[i].u[e]);
            f[i].w[e] = MODE == kLayer ? fma2(w, g[i].w[e], bf[i].w[e]) : mul2(w, g[i].w[e]);
          }
      }
      const bool on = first < left;
      RopeAngles<V, NU> ang;
      ang.get(a, l, sh.cs + (on ? out.tok * 2 * a.pairs : 0));
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        if (l.pair[i] >= 0) ang.turn(i, f[i]);
        f[i].template set<MIX>(o[i], l.mix[i]);
      }
      if (MIX == kMixed) {
        ring.trade(o);
        ring.step();
      }
      if (on) l.store(o, const_cast<char *>(out.p[0]));
      out.next();
    }
  }
}

template <int DT, int V, int NU, int MIX>
const void *pick_mode(int mode) {
  switch (mode) {
    case kRMS: return reinterpret_cast<const void *>(&rope_fwd_kernel<DT, V, NU, kRMS, MIX>);
    case kLayer: return reinterpret_cast<const void *>(&rope_fwd_kernel<DT, V, NU, kLayer, MIX>);
    default: return reinterpret_cast<const void *>(&rope_fwd_kernel<DT, V, NU, kNoNorm, MIX>);
  }
}

template <int DT, int V, int NU>
const void *pick_mix(int mode, bool inter) {
  return inter ? pick_mode<DT, V, NU, kMixed>(mode) : pick_mode<DT, V, NU, kApart>(mode);
}

template <int DT>
const void *pick_width(int V, int NU, int mode, bool inter) {
  switch (V) {
    case 8:
      if constexpr (DT != kFP32) return pick_mix<DT, 8, 1>(mode, inter);
      return nullptr;
    case 4: return NU == 3 ? pick_mix<DT, 4, 3>(mode, inter) : pick_mix<DT, 4, 1>(mode, inter);
    case 2: return pick_mode<DT, 2, rope_units(2), kEither>(mode);
    default: return pick_mode<DT, 1, rope_units(1), kApart>(mode);
  }
}

}  // namespace

const void *rope_fwd_kernel_ptr(int dt, int V, int NU, int mode, bool inter) {
  switch (dt) {
    case kBF16: return pick_width<kBF16>(V, NU, mode, inter);
    case kFP16: return pick_width<kFP16>(V, NU, mode, inter);
    default: return pick_width<kFP32>(V, NU, mode, inter);
  }
}

namespace {

// What both entry points check, and the arguments that the shape alone gives.
norm_status_t rope_shape(int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t rd,
                         norm_mode_t mode, norm_dtype_t dtype) {
  if (mode != NORM_RMS && mode != NORM_LAYER) return NORM_ERR_MODE;
  if (dtype != NORM_BF16 && dtype != NORM_FP16 && dtype != NORM_FP32) return NORM_ERR_ARG;
  if (T < 1 || T > (int64_t(1) << 31) || Hq < 1 || Hq > 65536 || Hk < 0 || Hk > 65536)
    return NORM_ERR_SHAPE;
  if (D < 2 || D > kRopeMaxD || rd < 2 || rd > D || rd % 2) return NORM_ERR_SHAPE;
  return NORM_OK;
}

struct Widest {
  int V;
  int es;
  void address(const void *p) {
    while (V > 1 && (reinterpret_cast<uintptr_t>(p) % (V * es))) V /= 2;
  }
  void count(int64_t n) {
    while (V > 1 && n % V) V /= 2;
  }
  bool heads(const norm_heads_t *h, int64_t T, int64_t H) {
    if (reinterpret_cast<uintptr_t>(h->data) % es) return false;
    address(h->data);
    if (T > 1) count(h->token_stride);
    if (H > 1) count(h->head_stride);
    return true;
  }
};

// The strides that kernels step by.  A single token's or head's says nothing: lanes
// beyond the last row form addresses with it, for copies of no bytes that have to
// be aligned all the same.
int64_t token_step(const norm_heads_t *h, int64_t T) { return T > 1 ? h->token_stride : 0; }
int64_t head_step(const norm_heads_t *h, int64_t H) { return H > 1 ? h->head_stride : 0; }

bool strides_ok(const norm_heads_t *h) {
  const int64_t most = int64_t(1) << 40;
  return h->token_stride >= 0 && h->token_stride <= most && h->head_stride >= 0 &&
         h->head_stride <= most;
}

// No two rows of an output may share elements: heads inside a token's stride, or
// tokens inside a head's.
bool rows_apart(const norm_heads_t *h, int64_t T, int64_t H, int64_t D) {
  const int64_t ts = h->token_stride, hs = h->head_stride;
  if (H > 1 && hs < D) return false;
  if (T > 1 && ts < D) return false;
  if (H == 1 || T == 1) return true;
  // (the products pass 64 bits: the second as a quotient, ts >= D >= 2)
  return ts >= (H - 1) * hs + D || (hs >= D && (hs - D) / ts >= T - 1);
}

int pow2_log(int n) {
  int l = 0;
  while ((1 << l) < n) ++l;
  return l;
}

norm_status_t rope_args(const void *pos, int pos_bits, int64_t pos_stride, const double *inv_freq,
                        const uint8_t *pair_axis, int axes, int interleaved, int64_t T, int64_t Hq,
                        int64_t Hk, int64_t D, int64_t rd, float eps, Widest *w, RopeArgs *a) {
  if (!pos || !inv_freq) return NORM_ERR_NULL;
  if (axes < 1 || axes > kRopeMaxAxes || (pos_bits != 32 && pos_bits != 64) || pos_stride < 0 ||
      pos_stride > (int64_t(1) << 40) || (interleaved != 0 && interleaved != 1))
    return NORM_ERR_ARG;
  if (axes > 1 && !pair_axis) return NORM_ERR_NULL;
  if (!std::isfinite(eps) || eps < 0.f) return NORM_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(pos) % (pos_bits / 8) ||
      reinterpret_cast<uintptr_t>(inv_freq) % 8)
    return NORM_ERR_ALIGN;
  *a = RopeArgs{};
  a->pos = pos;
  a->pos64 = pos_bits == 64;
  a->pos_stride = pos_stride;
  a->inv_freq = inv_freq;
  a->axes = axes;
  a->T = T;
  a->D = static_cast<int>(D);
  a->rd = static_cast<int>(rd);
  a->pairs = a->rd / 2;
  a->inter = interleaved;
  a->sign = 1.f;
  a->eps = eps;
  a->invD = 1.f / static_cast<float>(D);
  if (pair_axis)
    for (int p = 0; p < a->pairs; ++p) {
      if (pair_axis[p] >= axes) return NORM_ERR_ARG;
      a->axis[p >> 5] |= uint64_t(pair_axis[p]) << ((p & 31) * 2);
    }
  w->count(a->pairs);
  w->count(D - rd);
  a->side[0].H = static_cast<int>(Hq);
  a->side[1].H = static_cast<int>(Hk);
  return NORM_OK;
}

// Lanes per row, once the chunk width and the units per lane are known.
void rope_lanes(RopeArgs *a, int V, int NU) {
  const int units = a->pairs / V + (a->D - a->rd + 2 * V - 1) / (2 * V);
  a->lanes_log2 = pow2_log((units + NU - 1) / NU);
  a->pairs_log2 = pow2_log(a->pairs);
}

// Units per lane of the forward kernels, and the lanes: three units of chunks of
// four where those leave fewer lanes without a unit than one unit each (heads of
// 48, 72, 80, 96, 112, 144, 160, ... elements).  32768 tokens of 16 + 16 heads,
// RMSNorm, one unit and three, us: bf16 heads of 72 101 and 64, 80 86 and 64, 160
// 155 and 114; fp32, whose copies of two lanes are too short, 48 66 and 68, from
// four lanes on 72 105 and 107, 80 104 and 105, 160 224 and 228, but with
// LayerNorm 128 and 109, 128 and 106, 243 and 230, and 1500 tokens of 80 9.0 and
// 7.5.  (The backward kernels would spill their sums: bf16, 32768 tokens of 80 128
// us with one unit, 156 with three.)
int rope_fwd_units(RopeArgs *a, int *V, int dtype) {
  const int one = rope_units(*V);
  rope_lanes(a, *V, one);
  if (*V < 4) return one;
  const int slots = *V << a->lanes_log2;
  RopeArgs b = *a;
  rope_lanes(&b, 4, 3);
  if ((12 << b.lanes_log2) >= slots || (dtype == NORM_FP32 && b.lanes_log2 < 2)) return one;
  a->lanes_log2 = b.lanes_log2;
  *V = 4;
  return 3;
}

// CTAs of each side: `per_sm` per SM in all, shared in proportion to the sides'
// work.  A token's angles cost about as much as two of its rows: at 32768 tokens
// of 32 + 8 heads the forward takes 126, 120, 117, 120 and 124 us where they are
// counted as 0, 1, 2, 3 and 6.
void rope_ctas(int64_t T, int64_t Hq, int64_t Hk, int sms, int per_sm, int *cq, int *ck) {
  const int64_t most = int64_t(sms) * per_sm;
  int64_t q = Hk ? (most * (Hq + 2) + (Hq + Hk + 4) / 2) / (Hq + Hk + 4) : most;
  if (q > most - (Hk ? 1 : 0)) q = most - (Hk ? 1 : 0);
  if (q < 1) q = 1;
  *cq = static_cast<int>(q < T ? q : T);
  *ck = Hk ? static_cast<int>(most - q < T ? most - q : T) : 0;
}

// Tokens per tile: all of a CTA's where shared memory holds their angles (5476
// tokens of 16 + 16 heads of 80, one unit per lane: 30 us in one tile, 32 in two),
// else `rows` rows or so, few enough for the CTAs to end together.  Few rows mean
// many barriers, many rows CTAs that drift apart and a wider stretch of memory in
// use.  Forward: 128 rows (32768 tokens of 32 + 8 heads of 128, bf16: 96 rows 113
// us, 128 108, 192 118; 16384 of 16 + 16: 45, 44 with 192), eight rounds where a
// round has 64 rows or more (heads of 64 with LayerNorm, 128 rows 31 us, 512 27),
// six of three units per lane in fp32 (32768 tokens of 80, LayerNorm: two rounds
// 116 us, six 106), twelve in 16 bits (two rounds 104, six 88, twelve 85).
// Backward: 512 rows (16384 tokens of 32 + 8 heads of 128: 256 rows 82.4 us, 384
// 81.1, 512 80.1, 768 81.7), sixteen rounds at least.
void rope_tiles(RopeArgs *a, int rows) {
  for (int i = 0; i < 2; ++i) {
    const int H = a->side[i].H;
    if (H == 0) continue;
    a->by_H[i].set(H);
    const int64_t per_cta = (a->T + a->ctas[i] - 1) / a->ctas[i];  // tokens
    int most = kRopeMaxAngles / a->pairs;
    if (most > kRopeMaxTile) most = kRopeMaxTile;
    if (per_cta > most && most > rows / H) most = rows / H;
    if (most < 1) most = 1;
    const int64_t tiles = (per_cta + most - 1) / most;
    a->tile[i] = static_cast<int>((per_cta + tiles - 1) / tiles);
  }
}

norm_status_t rope_launch_fwd(RopeArgs *a, int V, int mode, int dtype, int dev, int sms, int optin,
                              cudaStream_t s) {
  const int NU = rope_fwd_units(a, &V, dtype);
  const void *fn = rope_fwd_kernel_ptr(dtype, V, NU, mode, a->inter);
  const norm_status_t st = function_ready(dev, fn, optin);
  if (st != NORM_OK) return st;
  // With few tokens per CTA a third CTA per SM costs more to start than it brings
  // (333 tokens: 4.7 us with three, 3.2 with two).
  const int per_sm = a->T < int64_t(sms) * 16 ? 2 : rope_fwd_ctas(mode, V, NU, a->inter);
  rope_ctas(a->T, a->side[0].H, a->side[1].H, sms, per_sm, &a->ctas[0], &a->ctas[1]);
  const int narrow = a->lanes_log2 <= 2 ? 8 * kRopeThreads >> a->lanes_log2 : 128;
  rope_tiles(a, NU == 3 ? 1536 / elem_bytes(dtype) : narrow);
  void *args[] = {a};
  return launch_serial(fn, dim3(unsigned(a->ctas[0] + a->ctas[1])), dim3(kRopeThreads),
                       sizeof(RopeShared) + rope_ring_bytes(dtype, V, NU, rope_fwd_stages(NU)), 1,
                       args, s);
}

}  // namespace

}  // namespace gbn

using namespace gbn;

extern "C" {

norm_status_t norm_rope_fwd(const norm_heads_t *q, const norm_heads_t *k, int64_t T, int64_t Hq,
                            int64_t Hk, int64_t D, int64_t rd, const void *pos, int pos_bits,
                            int64_t pos_stride, const double *inv_freq, const uint8_t *pair_axis,
                            int axes, int interleaved, const void *gamma_q, const void *gamma_k,
                            const void *beta_q, const void *beta_k, float eps, norm_mode_t mode,
                            norm_dtype_t dtype, const norm_heads_t *yq, const norm_heads_t *yk,
                            norm_stream_t stream) {
  norm_status_t st = rope_shape(T, Hq, Hk, D, rd, mode, dtype);
  if (st != NORM_OK) return st;
  if (!q || !yq || !q->data || !yq->data) return NORM_ERR_NULL;
  if (Hk > 0 && (!k || !yk || !k->data || !yk->data)) return NORM_ERR_NULL;
  const bool norm = gamma_q != nullptr;
  if (norm ? (Hk > 0 && !gamma_k) : gamma_k != nullptr) return NORM_ERR_NULL;
  if ((beta_q || beta_k) && (mode == NORM_RMS || !norm)) return NORM_ERR_MODE;
  if (Hk == 0 && (gamma_k || beta_k)) return NORM_ERR_ARG;
  Widest w{dtype == NORM_FP32 ? 4 : 8, elem_bytes(dtype)};
  RopeArgs a;
  st = rope_args(pos, pos_bits, pos_stride, inv_freq, pair_axis, axes, interleaved, T, Hq, Hk, D, rd,
                 eps, &w, &a);
  if (st != NORM_OK) return st;
  const norm_heads_t *x[2] = {q, k}, *y[2] = {yq, yk};
  const void *gamma[2] = {gamma_q, gamma_k}, *beta[2] = {beta_q, beta_k};
  for (int i = 0; i < (Hk > 0 ? 2 : 1); ++i) {
    RopeSide &s = a.side[i];
    if (!strides_ok(x[i]) || !strides_ok(y[i]) || !rows_apart(y[i], T, s.H, D))
      return NORM_ERR_SHAPE;
    if (!w.heads(x[i], T, s.H) || !w.heads(y[i], T, s.H)) return NORM_ERR_ALIGN;
    for (const void *p : {gamma[i], beta[i]}) {
      if (reinterpret_cast<uintptr_t>(p) % w.es) return NORM_ERR_ALIGN;
      w.address(p);
    }
    s.x = x[i]->data;
    s.xt = token_step(x[i], T);
    s.xh = head_step(x[i], s.H);
    s.out = y[i]->data;
    s.ot = token_step(y[i], T);
    s.oh = head_step(y[i], s.H);
    s.gamma = gamma[i];
    s.beta = beta[i];
  }
  int dev = 0, sms = 0, optin = 0;
  unsigned *err = nullptr;
  if ((st = device_context(&dev, &sms, &optin, &err, nullptr)) != NORM_OK) return st;
  return rope_launch_fwd(&a, w.V, norm ? mode : kNoNorm, dtype, dev, sms, optin,
                         reinterpret_cast<cudaStream_t>(stream));
}

norm_status_t norm_rope_bwd_workspace_bytes(int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                                            int normed, norm_mode_t mode, size_t *bytes) {
  if (!bytes) return NORM_ERR_NULL;
  norm_status_t st = rope_shape(T, Hq, Hk, D, D - D % 2, mode, NORM_BF16);
  if (st != NORM_OK) return st;
  *bytes = 0;
  if (!normed) return NORM_OK;
  int dev = 0, sms = 0, optin = 0;
  unsigned *err = nullptr;
  if ((st = device_context(&dev, &sms, &optin, &err, nullptr)) != NORM_OK) return st;
  int cq = 0, ck = 0;
  rope_ctas(T, Hq, Hk, sms, kRopeBwdCtas, &cq, &ck);
  *bytes = size_t(cq + ck) * size_t(D) * 4 * (mode == NORM_LAYER ? 2 : 1);
  return NORM_OK;
}

norm_status_t norm_rope_bwd(const norm_heads_t *dyq, const norm_heads_t *dyk, const norm_heads_t *q,
                            const norm_heads_t *k, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                            int64_t rd, const void *pos, int pos_bits, int64_t pos_stride,
                            const double *inv_freq, const uint8_t *pair_axis, int axes,
                            int interleaved, const void *gamma_q, const void *gamma_k, float eps,
                            norm_mode_t mode, norm_dtype_t dtype, const norm_heads_t *dq,
                            const norm_heads_t *dk, float *dgamma_q, float *dgamma_k,
                            float *dbeta_q, float *dbeta_k, void *workspace,
                            size_t workspace_bytes, norm_stream_t stream) {
  norm_status_t st = rope_shape(T, Hq, Hk, D, rd, mode, dtype);
  if (st != NORM_OK) return st;
  const bool norm = gamma_q != nullptr;
  const int sides = Hk > 0 ? 2 : 1;
  const norm_heads_t *dy[2] = {dyq, dyk}, *x[2] = {q, k}, *out[2] = {dq, dk};
  const void *gamma[2] = {gamma_q, gamma_k};
  float *dgamma[2] = {dgamma_q, dgamma_k}, *dbeta[2] = {dbeta_q, dbeta_k};
  for (int i = 0; i < sides; ++i) {
    if (!dy[i] || !dy[i]->data || !out[i] || !out[i]->data) return NORM_ERR_NULL;
    if (norm && (!x[i] || !x[i]->data || !gamma[i] || !dgamma[i])) return NORM_ERR_NULL;
  }
  if (!norm && (gamma_k || dgamma_q || dgamma_k || dbeta_q || dbeta_k)) return NORM_ERR_MODE;
  if (mode == NORM_RMS && (dbeta_q || dbeta_k)) return NORM_ERR_MODE;
  if (Hk == 0 && (gamma_k || dgamma_k || dbeta_k)) return NORM_ERR_ARG;
  Widest w{dtype == NORM_FP32 ? 4 : 8, elem_bytes(dtype)};
  RopeArgs a;
  st = rope_args(pos, pos_bits, pos_stride, inv_freq, pair_axis, axes, interleaved, T, Hq, Hk, D, rd,
                 eps, &w, &a);
  if (st != NORM_OK) return st;
  for (int i = 0; i < sides; ++i) {
    RopeSide &s = a.side[i];
    if (!strides_ok(dy[i]) || !strides_ok(out[i]) || !rows_apart(out[i], T, s.H, D) ||
        (norm && !strides_ok(x[i])))
      return NORM_ERR_SHAPE;
    if (!w.heads(dy[i], T, s.H) || !w.heads(out[i], T, s.H) || (norm && !w.heads(x[i], T, s.H)))
      return NORM_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(gamma[i]) % w.es) return NORM_ERR_ALIGN;
    w.address(gamma[i]);
    for (const float *p : {dgamma[i], dbeta[i]})
      if (reinterpret_cast<uintptr_t>(p) % 4) return NORM_ERR_ALIGN;
    s.out = out[i]->data;
    s.ot = token_step(out[i], T);
    s.oh = head_step(out[i], s.H);
    s.dy = dy[i]->data;
    s.dt = token_step(dy[i], T);
    s.dh = head_step(dy[i], s.H);
    s.gamma = gamma[i];
    if (norm) {
      s.x = x[i]->data;
      s.xt = token_step(x[i], T);
      s.xh = head_step(x[i], s.H);
    } else {  // the gradient turns back: the forward kernel with the other sign
      s.x = s.dy;
      s.xt = s.dt;
      s.xh = s.dh;
    }
  }
  int dev = 0, sms = 0, optin = 0;
  unsigned *err = nullptr;
  if ((st = device_context(&dev, &sms, &optin, &err, nullptr)) != NORM_OK) return st;
  a.sign = -1.f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!norm) return rope_launch_fwd(&a, w.V, kNoNorm, dtype, dev, sms, optin, s);
  size_t need = 0;
  if ((st = norm_rope_bwd_workspace_bytes(T, Hq, Hk, D, 1, mode, &need)) != NORM_OK) return st;
  if (!workspace || workspace_bytes < need) return NORM_ERR_WORKSPACE;
  if (!aligned_to_16(workspace)) return NORM_ERR_ALIGN;
  a.part = static_cast<float *>(workspace);
  rope_lanes(&a, w.V, rope_units(w.V));
  rope_ctas(T, Hq, Hk, sms, kRopeBwdCtas, &a.ctas[0], &a.ctas[1]);
  const int per = kRopeThreads >> a.lanes_log2;  // rows of a round
  rope_tiles(&a, 16 * per > 512 ? 16 * per : 512);
  const bool layer = mode == NORM_LAYER;
  const void *fn = rope_bwd_kernel_ptr(dtype, w.V, mode, a.inter);
  if ((st = function_ready(dev, fn, optin)) != NORM_OK) return st;
  const uint32_t ring = rope_ring_bytes(dtype, w.V, rope_units(w.V), 2 * kRopeBwdStages);
  const uint32_t fold_bytes = rope_fold_floats(a.D, layer) * 4;
  void *args[] = {&a};
  st = launch_serial(fn, dim3(a.ctas[0] + a.ctas[1]), dim3(kRopeThreads),
                     sizeof(RopeShared) + (ring > fold_bytes ? ring : fold_bytes), 1, args, s);
  if (st != NORM_OK) return st;
  const float *part = a.part;
  int n = a.D, cq = a.ctas[0], ck = a.ctas[1];
  void *fold[] = {&part, &n, &cq, &ck, &dgamma[0], &dgamma[1], &dbeta[0], &dbeta[1]};
  return launch_serial(rope_fold_kernel_ptr(), dim3((n + 31) / 32, layer ? 4 : 2), dim3(1024), 0, 1,
                       fold, s);
}

}  // extern "C"
