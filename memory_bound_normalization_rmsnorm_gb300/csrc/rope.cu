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

constexpr int kRopeBatch = 4;  // rows in flight per thread

// One pass: read a row, normalise it in registers, turn its pairs, write it.
// A warp takes a token (or, where tokens are few, a share of its heads): the
// angles are computed once for all heads of the token, queries and keys.
template <int DT, int V, int MODE>
__global__ void __launch_bounds__(kRopeThreads) rope_fwd_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int NU = rope_units(V);
  __shared__ uint64_t turns[kRopeMaxD / 2];
  grid_launch_dependents();
  grid_dependency_wait();
  rope_table(a, turns);
  __syncthreads();
  const RopeLane<V> l(a);
  const int warps = kRopeThreads / 32;
  const int chunks = a.chunks[0];
  const int64_t items = a.T * chunks;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * warps + threadIdx.x / 32; item < items;
       item += static_cast<int64_t>(gridDim.x) * warps) {
    const int64_t t = item / chunks;
    const int c = static_cast<int>(item - t * chunks);
    RopeAngles<V> ang;
    ang.at(a, l, turns, t);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const RopeSide &s = a.side[side];
      if (s.H == 0) continue;
      const int r0 = s.rounds * c / chunks, r1 = s.rounds * (c + 1) / chunks;
      if (r0 == r1) continue;
      float g[NU][2 * V], b[NU][2 * V];
      if constexpr (MODE != kNoNorm) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          RopeVec<DT, V> v;
          v.zero();
          if (l.in1[i]) v.load(s.gamma, l.o1[i]);
          v.get(g[i]);
          v.zero();
          if (l.in2[i]) v.load(s.gamma, l.o2[i]);
          v.get(g[i] + V);
          if constexpr (MODE == kLayer) {
            v.zero();
            if (l.in1[i] && s.beta) v.load(s.beta, l.o1[i]);
            v.get(b[i]);
            v.zero();
            if (l.in2[i] && s.beta) v.load(s.beta, l.o2[i]);
            v.get(b[i] + V);
          }
        }
      }
      for (int r = r0; r < r1; r += kRopeBatch) {
        RopeVec<DT, V> v[kRopeBatch][NU][2];
#pragma unroll
        for (int n = 0; n < kRopeBatch; ++n) {
          const int h = ((r + n) << (5 - a.lanes_log2)) + l.group;
          const bool row = r + n < r1 && h < s.H;
          const int64_t at = t * s.xt + h * s.xh;
#pragma unroll
          for (int i = 0; i < NU; ++i) {
            v[n][i][0].zero();
            v[n][i][1].zero();
            if (row && l.in1[i]) v[n][i][0].load(s.x, at + l.o1[i]);
            if (row && l.in2[i]) v[n][i][1].load(s.x, at + l.o2[i]);
          }
        }
#pragma unroll
        for (int n = 0; n < kRopeBatch; ++n) {
          if (r + n >= r1) break;
          const int h = ((r + n) << (5 - a.lanes_log2)) + l.group;
          float f[NU][2 * V];
#pragma unroll
          for (int i = 0; i < NU; ++i) {
            v[n][i][0].get(f[i]);
            v[n][i][1].get(f[i] + V);
          }
          if constexpr (MODE != kNoNorm) {
            const float rstd = rope_stats<MODE, V>(a, l, f);
#pragma unroll
            for (int i = 0; i < NU; ++i)
#pragma unroll
              for (int e = 0; e < 2 * V; ++e)
                f[i][e] = MODE == kLayer ? fmaf(f[i][e] * rstd, g[i][e], b[i][e])
                                         : f[i][e] * rstd * g[i][e];
          }
          if (h >= s.H) continue;
          const int64_t at = t * s.ot + h * s.oh;
#pragma unroll
          for (int i = 0; i < NU; ++i) {
            if (l.pair[i] >= 0) {
              if (a.inter)
                ang.turn(i, true, f[i]);
              else
                ang.turn(i, false, f[i]);
            }
            v[n][i][0].set(f[i]);
            v[n][i][1].set(f[i] + V);
            if (l.in1[i]) v[n][i][0].store(s.out, at + l.o1[i]);
            if (l.in2[i]) v[n][i][1].store(s.out, at + l.o2[i]);
          }
        }
      }
    }
  }
}

template <int DT, int V>
const void *pick_mode(int mode) {
  switch (mode) {
    case kRMS: return reinterpret_cast<const void *>(&rope_fwd_kernel<DT, V, kRMS>);
    case kLayer: return reinterpret_cast<const void *>(&rope_fwd_kernel<DT, V, kLayer>);
    default: return reinterpret_cast<const void *>(&rope_fwd_kernel<DT, V, kNoNorm>);
  }
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

const void *rope_fwd_kernel_ptr(int dt, int V, int mode) {
  switch (dt) {
    case kBF16: return pick_width<kBF16>(V, mode);
    case kFP16: return pick_width<kFP16>(V, mode);
    default: return pick_width<kFP32>(V, mode);
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
  return ts >= (H - 1) * hs + D || hs >= (T - 1) * ts + D;
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

// Lanes per row and rounds, once the chunk width is known.
void rope_lanes(RopeArgs *a, int V) {
  a->units = a->pairs / V + (a->D - a->rd + 2 * V - 1) / (2 * V);
  const int l = pow2_log(a->units);
  a->lanes_log2 = l < 5 ? l : 5;
  for (RopeSide &s : a->side) {
    const int groups = 32 >> a->lanes_log2;
    s.rounds = (s.H + groups - 1) / groups;
  }
}

constexpr int kRopeWarps = kRopeThreads / 32;

// Warps that share a token: one where the tokens fill the GPU (the angles are
// then computed once), else up to one per round of its longer side.
int rope_chunks(int64_t T, int rounds, int sms) {
  const int64_t want = int64_t(sms) * 16;
  const int64_t c = (want + T - 1) / T;
  return static_cast<int>(c < 1 ? 1 : c > rounds ? rounds : c);
}

norm_status_t rope_launch_fwd(RopeArgs *a, int V, int mode, int dtype, int sms, cudaStream_t s) {
  const int rounds = a->side[0].rounds > a->side[1].rounds ? a->side[0].rounds : a->side[1].rounds;
  a->chunks[0] = rope_chunks(a->T, rounds, sms);
  const int64_t items = a->T * a->chunks[0];
  const int64_t ctas = (items + kRopeWarps - 1) / kRopeWarps;
  const int64_t most = int64_t(sms) * 8;
  void *args[] = {a};
  return launch_serial(rope_fwd_kernel_ptr(dtype, V, mode),
                       dim3(static_cast<unsigned>(ctas < most ? ctas : most)), dim3(kRopeThreads), 0,
                       1, args, s);
}

// CTAs of each side of the backward, in proportion to its rows.
void rope_bwd_ctas(int64_t T, int64_t Hq, int64_t Hk, int sms, int *cq, int *ck) {
  const int64_t most = int64_t(sms) * 3;
  const int64_t rows[2] = {T * Hq, T * Hk};
  int *out[2] = {cq, ck};
  for (int i = 0; i < 2; ++i) {
    int64_t c = (most * rows[i] + rows[0] + rows[1] - 1) / (rows[0] + rows[1]);
    const int64_t use = (rows[i] + 15) / 16;  // two rows or more per warp
    if (c > use) c = use;
    *out[i] = static_cast<int>(c);
  }
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
    s.xt = x[i]->token_stride;
    s.xh = x[i]->head_stride;
    s.out = y[i]->data;
    s.ot = y[i]->token_stride;
    s.oh = y[i]->head_stride;
    s.gamma = gamma[i];
    s.beta = beta[i];
  }
  int dev = 0, sms = 0, optin = 0;
  unsigned *err = nullptr;
  if ((st = device_context(&dev, &sms, &optin, &err, nullptr)) != NORM_OK) return st;
  rope_lanes(&a, w.V);
  return rope_launch_fwd(&a, w.V, norm ? mode : kNoNorm, dtype, sms,
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
  rope_bwd_ctas(T, Hq, Hk, sms, &cq, &ck);
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
    s.ot = out[i]->token_stride;
    s.oh = out[i]->head_stride;
    s.dy = dy[i]->data;
    s.dt = dy[i]->token_stride;
    s.dh = dy[i]->head_stride;
    s.gamma = gamma[i];
    if (norm) {
      s.x = x[i]->data;
      s.xt = x[i]->token_stride;
      s.xh = x[i]->head_stride;
    } else {  // the gradient turns back: the forward kernel with the other sign
      s.x = s.dy;
      s.xt = s.dt;
      s.xh = s.dh;
    }
  }
  int dev = 0, sms = 0, optin = 0;
  unsigned *err = nullptr;
  if ((st = device_context(&dev, &sms, &optin, &err, nullptr)) != NORM_OK) return st;
  rope_lanes(&a, w.V);
  a.sign = -1.f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!norm) return rope_launch_fwd(&a, w.V, kNoNorm, dtype, sms, s);
  size_t need = 0;
  if ((st = norm_rope_bwd_workspace_bytes(T, Hq, Hk, D, 1, mode, &need)) != NORM_OK) return st;
  if (!workspace || workspace_bytes < need) return NORM_ERR_WORKSPACE;
  if (!aligned_to_16(workspace)) return NORM_ERR_ALIGN;
  a.part = static_cast<float *>(workspace);
  rope_bwd_ctas(T, Hq, Hk, sms, &a.ctas[0], &a.ctas[1]);
  for (int i = 0; i < 2; ++i) {
    // warps that share a token: as many as leave every warp of the side work
    const int64_t warps = int64_t(a.ctas[i]) * kRopeWarps;
    int64_t c = (warps + T - 1) / T;
    if (c > a.side[i].rounds) c = a.side[i].rounds;
    a.chunks[i] = static_cast<int>(c < 1 ? 1 : c);
  }
  const bool layer = mode == NORM_LAYER;
  void *args[] = {&a};
  st = launch_serial(rope_bwd_kernel_ptr(dtype, w.V, mode), dim3(a.ctas[0] + a.ctas[1]),
                     dim3(kRopeThreads), rope_fold_floats(a.D, layer) * 4, 1, args, s);
  if (st != NORM_OK) return st;
  const float *part = a.part;
  int n = a.D, cq = a.ctas[0], ck = a.ctas[1];
  void *fold[] = {&part, &n, &cq, &ck, &dgamma[0], &dgamma[1], &dbeta[0], &dbeta[1]};
  return launch_serial(rope_fold_kernel_ptr(), dim3((n + 31) / 32, layer ? 4 : 2), dim3(1024), 0, 1,
                       fold, s);
}

}  // extern "C"
