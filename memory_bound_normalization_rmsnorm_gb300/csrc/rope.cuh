// rope.cuh -- normalisation of query and key heads and their rotation by
// positions of up to four axes (norm_rope_fwd, norm_rope_bwd): arguments, lane
// layout, angles and the arithmetic that both directions share.
//
// A head row has D elements of one token and head.  Its first rd elements are
// rd / 2 pairs (p and p + rd / 2, or neighbours 2p and 2p + 1); pair p turns by
// the angle pos[axis(p)][token] * inv_freq[p], the others stay.
//
// Layout.  A unit is two chunks of V elements: the 2V elements of V pairs, or
// 2V elements behind rd.  The rows are short (D <= 256), so L = 4 to 32 lanes
// of a warp share one, a unit (or kUnits, for the narrow V of odd sizes) per
// lane: both elements of every pair lie in one thread, a row's statistics take
// log2 L shuffles, and the 32 / L groups of a warp read heads side by side.  V
// is the widest chunk (up to 16 bytes) that the pair count, the unturned rest,
// every stride and every address are whole multiples of.
#pragma once
#include <cstdint>

#include "elem.cuh"

namespace gbn {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxD = 256;
constexpr int kRopeMaxAxes = 4;
constexpr int kNoNorm = 2;  // mode beside kRMS and kLayer: rotation alone

struct RopeSide {
  const void *x;   // forward input
  const void *dy;  // backward: gradient of the output
  void *out;       // y, or dx
  const void *gamma, *beta;
  int64_t xt, xh, dt, dh, ot, oh;  // token and head strides, in elements
  int H;
  int rounds;  // ceil(H / groups per warp)
};

struct RopeArgs {
  RopeSide side[2];  // q, k (H = 0: none)
  const void *pos;
  const double *inv_freq;
  int64_t pos_stride;   // between axes, in elements
  uint64_t axis[4];     // two bits per pair
  int64_t T;
  float *part;          // backward: partial rows of dgamma, then of dbeta
  int ctas[2];          // backward: CTAs of each side
  int chunks[2];        // warps that share a token's rounds (forward: [0] for both sides)
  int D, rd, pairs, units;
  int lanes_log2;       // log2 L
  int axes;
  int pos64;
  int inter;            // pairs of neighbours
  float sign;           // -1: the inverse rotation
  float eps, invD;
};

__host__ __device__ constexpr int rope_units(int V) { return V >= 4 ? 1 : 4 / V; }

// --------------------------------------------------------------- chunks
// V elements at p (a whole multiple of V elements from an address aligned to
// V elements) as fp32.
template <int DT, int V>
struct RopeVec {
  static constexpr int kBytes = V * elem_bytes(DT);
  static constexpr int kWords = (kBytes + 3) / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const void *base, int64_t i) {
    const char *p = static_cast<const char *>(base) + i * elem_bytes(DT);
    if constexpr (kBytes == 16) {
      const uint4 v = *reinterpret_cast<const uint4 *>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2 *>(p);
      w[0] = v.x, w[1] = v.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void get(float *f) const {
    if constexpr (DT == kFP32) {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        float2 p;
        if constexpr (DT == kBF16)
          p = bf2_to_f2(w[i]);
        else
          p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        f[2 * i] = p.x;
        if (V > 1) f[2 * i + 1] = p.y;
      }
    }
  }
  // rounded to nearest even
  __device__ __forceinline__ void set(const float *f) {
    if constexpr (DT == kFP32) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const float2 p = make_float2(f[2 * i], V > 1 ? f[2 * i + 1] : 0.f);
        if constexpr (DT == kBF16) {
          w[i] = f2_to_bf2(p);
        } else {
          const __half2 h = __floats2half2_rn(p.x, p.y);
          w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
      }
    }
  }
  __device__ __forceinline__ void store(void *base, int64_t i) const {
    char *p = static_cast<char *>(base) + i * elem_bytes(DT);
    if constexpr (kBytes == 16)
      *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kBytes == 8)
      *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else if constexpr (kBytes == 4)
      *reinterpret_cast<uint32_t *>(p) = w[0];
    else
      *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(w[0]);
  }
};

// ----------------------------------------------------------------- lanes
// Where the units of this lane lie in a row.
template <int V>
struct RopeLane {
  static constexpr int NU = rope_units(V);
  int o1[NU], o2[NU];     // elements of the two chunks
  int pair[NU];           // first pair of the unit, or -1: not turned
  bool in1[NU], in2[NU];  // the chunk exists
  int group;              // this lane's row among the warp's

  __device__ __forceinline__ explicit RopeLane(const RopeArgs &a) {
    const int lane = threadIdx.x & 31;
    const int L = 1 << a.lanes_log2;
    group = lane >> a.lanes_log2;
    const int punits = a.pairs / V;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = (lane & (L - 1)) + i * L;
      if (u < punits) {
        pair[i] = u * V;
        o1[i] = a.inter ? 2 * V * u : V * u;
        o2[i] = a.inter ? o1[i] + V : a.pairs + V * u;
      } else {
        pair[i] = -1;
        o1[i] = a.rd + 2 * V * (u - punits);
        o2[i] = o1[i] + V;
      }
      in1[i] = o1[i] < a.D;
      in2[i] = o2[i] < a.D;
    }
  }
};

// ---------------------------------------------------------------- angles
// An angle is a fraction of a turn: with f = inv_freq / (2 pi) as a 64-bit
// binary fraction of a turn, pos * f modulo 2^64 is the angle modulo a whole
// turn exactly, however far the position: an integer product in place of a
// range reduction.  (A product in 32 bits is off by 0.06 radians at position
// 2^20; in float64 it is exact enough, at 1/64 of the rate.)  f is rounded to
// 2^-54 of itself, the angle to 2^-32 of a turn and then to fp32.
__device__ __forceinline__ uint64_t rope_turns(double inv_freq) {
  double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  t -= rint(t);
  return static_cast<uint64_t>(__double2ll_rn(t * 18446744073709551616.0));  // 2^64
}

// Fills the table of turns per position in shared memory (the caller
// synchronises).
__device__ __forceinline__ void rope_table(const RopeArgs &a, uint64_t *turns) {
  for (int p = threadIdx.x; p < a.pairs; p += blockDim.x) turns[p] = rope_turns(a.inv_freq[p]);
}

__device__ __forceinline__ int64_t rope_pos(const RopeArgs &a, int axis, int64_t t) {
  const int64_t i = axis * a.pos_stride + t;
  return a.pos64 ? static_cast<const int64_t *>(a.pos)[i]
                 : static_cast<int64_t>(static_cast<const int32_t *>(a.pos)[i]);
}

// cos and sin of this lane's pairs at token t.
template <int V>
struct RopeAngles {
  static constexpr int NU = rope_units(V);
  float c[NU][V], s[NU][V];

  __device__ __forceinline__ void at(const RopeArgs &a, const RopeLane<V> &l,
                                     const uint64_t *turns, int64_t t) {
    int64_t pos[kRopeMaxAxes];
#pragma unroll
    for (int x = 0; x < kRopeMaxAxes; ++x) pos[x] = x < a.axes ? rope_pos(a, x, t) : 0;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (l.pair[i] < 0) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int p = l.pair[i] + e;
        const int ax = static_cast<int>(a.axis[p >> 5] >> ((p & 31) * 2)) & 3;
        const int64_t lo = ax & 1 ? pos[1] : pos[0], hi = ax & 1 ? pos[3] : pos[2];
        const uint64_t turn = static_cast<uint64_t>(ax & 2 ? hi : lo) * turns[p];
        const float half = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
        sincospif(half, &s[i][e], &c[i][e]);
        s[i][e] *= a.sign;
      }
    }
  }

  // Turns the 2V values of unit i.
  __device__ __forceinline__ void turn(int i, bool inter, float (&f)[2 * V]) const {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int p = inter ? 2 * e : e, q = inter ? 2 * e + 1 : V + e;
      const float u = f[p], v = f[q];
      f[p] = fmaf(u, c[i][e], -(v * s[i][e]));
      f[q] = fmaf(v, c[i][e], u * s[i][e]);
    }
  }
};

// Sum over the L lanes of a row, the same bits in each.
__device__ __forceinline__ float rope_sum(float v, int lanes_log2) {
#pragma unroll
  for (int o = 0; o < 5; ++o)
    if (o < lanes_log2) v += __shfl_xor_sync(0xffffffffu, v, 1 << o);
  return v;
}

// x - mean (LayerNorm) in f, zero where there is no element; returns rstd.
template <int MODE, int V>
__device__ __forceinline__ float rope_stats(const RopeArgs &a, const RopeLane<V> &l,
                                            float (&f)[rope_units(V)][2 * V]) {
  constexpr int NU = rope_units(V);
  if constexpr (MODE == kLayer) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) m += f[i][e];
    m = rope_sum(m, a.lanes_log2) * a.invD;
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e)
        f[i][e] = (e < V ? l.in1[i] : l.in2[i]) ? f[i][e] - m : 0.f;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) q = fmaf(f[i][e], f[i][e], q);
  return rsqrtf(fmaf(rope_sum(q, a.lanes_log2), a.invD, a.eps));
}

const void *rope_fwd_kernel_ptr(int dt, int V, int mode);
const void *rope_bwd_kernel_ptr(int dt, int V, int mode);
const void *rope_fold_kernel_ptr();
// Floats of shared memory that the backward's last fold takes.
__host__ __device__ inline int rope_fold_floats(int D, bool layer) {
  return (kRopeThreads / 32) * D * (layer ? 2 : 1);
}

}  // namespace gbn
