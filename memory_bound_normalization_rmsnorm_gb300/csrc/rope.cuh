// rope.cuh -- normalisation of query and key heads and their rotation by
// positions of up to four axes (norm_rope_fwd, norm_rope_bwd): arguments, lane
// layout, angles and the arithmetic that both directions share.
//
// A head row has D elements of one token and head.  Its first rd elements are
// rd / 2 pairs (p and p + rd / 2, or neighbours 2p and 2p + 1); pair p turns by
// the angle pos[axis(p)][token] * inv_freq[p], the others stay.
//
// Layout.  A unit is two chunks of V elements: the 2V elements of V pairs, or
// 2V elements behind rd.  The rows are short (D <= 256), so L = 1 to 32 lanes
// of a warp share one, a unit (or several, for the narrow V of odd sizes and where
// one each would leave lanes without) per lane: both elements of every pair lie in
// one thread, a row's statistics take log2 L shuffles, and the 32 / L groups of a
// warp read heads side by side.  V is the widest chunk (up to 16 bytes) that the
// pair count, the unturned rest, every stride and every address are whole
// multiples of.
#pragma once
#include <cstdint>

#include "elem.cuh"

namespace gbn {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxD = 256;
constexpr int kRopeMaxAxes = 4;
// CTAs per SM, by registers (LayerNorm holds two parameter rows; with eight
// elements per chunk it spills at 80 registers, and so does RMSNorm where pairs
// are neighbours: 16384 tokens of 16 + 16 heads of 128, bf16, 53 us with three
// CTAs, 47 with two).
__host__ __device__ constexpr int rope_fwd_ctas(int mode, int V, int NU, bool mixed) {
  return (V == 8 && (mode == 1 || (mode == 0 && mixed))) || NU == 3 ? 2 : 3;
}
constexpr int kRopeBwdCtas = 2;
__host__ __device__ constexpr int rope_fwd_stages(int NU) { return NU == 3 ? 3 : 5; }  // of the ring
constexpr int kRopeBwdStages = 4;
constexpr int kNoNorm = 2;  // mode beside kRMS and kLayer: rotation alone

struct RopeSide {
  const void *x;   // forward input
  const void *dy;  // backward: gradient of the output
  void *out;       // y, or dx
  const void *gamma, *beta;
  int64_t xt, xh, dt, dh, ot, oh;  // token and head strides, in elements
  int H;
};

// Division of n (0 <= n < 2^31) by d >= 1 known to the host, by a product
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", PLDI 1994).
struct RopeDiv {
  uint32_t m, l;
  void set(int d) {
    l = 0;
    while ((int64_t(1) << l) < d) ++l;
    m = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << l) - d)) / d + 1);
  }
  __device__ __forceinline__ int operator()(int n) const {
    const uint32_t u = static_cast<uint32_t>(n);
    return static_cast<int>((__umulhi(m, u) + u) >> l);
  }
};

struct RopeArgs {
  RopeSide side[2];  // q, k (H = 0: none)
  const void *pos;
  const double *inv_freq;
  int64_t pos_stride;   // between axes, in elements
  uint64_t axis[4];     // two bits per pair
  int64_t T;
  float *part;          // backward: partial rows of dgamma, then of dbeta
  int ctas[2];          // CTAs of each side
  int tile[2];          // tokens per tile of each side
  RopeDiv by_H[2];      // by the heads of each side
  int D, rd, pairs;
  int lanes_log2;       // log2 L
  int pairs_log2;       // log2 of the pairs, rounded up
  int axes;
  int pos64;
  int inter;            // pairs of neighbours
  float sign;           // -1: the inverse rotation
  float eps, invD;
};

__host__ __device__ constexpr int rope_units(int V) { return V >= 4 ? 1 : 4 / V; }

// --------------------------------------------------------------- chunks
// V elements at p (a whole multiple of V elements from an address aligned to
// V elements).
template <int DT, int V>
struct RopeVec {
  static constexpr int kBytes = V * elem_bytes(DT);
  static constexpr int kWords = (kBytes + 3) / 4;
  static constexpr int NP = V > 1 ? V / 2 : 1;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const char *p) {
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
  // Neighbours as fp32 pairs (V = 1: the element and 0).
  __device__ __forceinline__ void get(float2 (&f)[NP]) const {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if constexpr (DT == kFP32)
        f[i] = make_float2(__uint_as_float(w[V > 1 ? 2 * i : 0]),
                           V > 1 ? __uint_as_float(w[V > 1 ? 2 * i + 1 : 0]) : 0.f);
      else if constexpr (DT == kBF16)
        f[i] = bf2_to_f2(w[i]);
      else
        f[i] = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    }
  }
  // rounded to nearest even
  __device__ __forceinline__ void set(const float2 (&f)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if constexpr (DT == kFP32) {
        w[V > 1 ? 2 * i : 0] = __float_as_uint(f[i].x);
        if constexpr (V > 1) w[2 * i + 1] = __float_as_uint(f[i].y);
      } else if constexpr (DT == kBF16) {
        w[i] = f2_to_bf2(f[i]);
      } else {
        const __half2 h = __floats2half2_rn(f[i].x, f[i].y);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
  }
  __device__ __forceinline__ void store(char *p) const {
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

// A unit's 2V values: the first elements of its pairs in u and the second in w,
// packed two by two for the packed fp32 instructions, whichever way the pairs
// lie in memory.
// Pairs of neighbours: never, always, or as the unit says.  (A branch at run time
// costs copies of the row's registers: 16384 tokens backward 96 us with it, 81
// without; the narrow chunks of odd sizes have it to save kernels.)
constexpr int kApart = 0, kMixed = 1, kEither = 2;
__host__ __device__ constexpr bool rope_mixed(int mix, bool unit) {
  return mix == kMixed || (mix == kEither && unit);
}

template <int V>
struct RopeUnit {
  static constexpr int NP = V > 1 ? V / 2 : 1;
  float2 u[NP], w[NP];

  template <int MIX, int DT>
  __device__ __forceinline__ void get(const RopeVec<DT, V> (&v)[2], bool mix) {
    float2 a[NP], b[NP];
    v[0].get(a);
    v[1].get(b);
    if (V > 1 && rope_mixed(MIX, mix)) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        put(i, a[i]);
        put(NP + i, b[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) u[i] = a[i], w[i] = b[i];
    }
  }
  template <int MIX, int DT>
  __device__ __forceinline__ void set(RopeVec<DT, V> (&v)[2], bool mix) const {
    if (V > 1 && rope_mixed(MIX, mix)) {
      float2 a[NP], b[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        a[i] = pair(i);
        b[i] = pair(NP + i);
      }
      v[0].set(a);
      v[1].set(b);
    } else {
      v[0].set(u);
      v[1].set(w);
    }
  }

 private:
  __device__ __forceinline__ void put(int e, float2 p) {
    if (e & 1)
      u[e / 2].y = p.x, w[e / 2].y = p.y;
    else
      u[e / 2].x = p.x, w[e / 2].x = p.y;
  }
  __device__ __forceinline__ float2 pair(int e) const {
    return e & 1 ? make_float2(u[e / 2].y, w[e / 2].y) : make_float2(u[e / 2].x, w[e / 2].x);
  }
};

// ----------------------------------------------------------------- lanes
// Where the units of this lane lie in a row, and which chunks it moves between
// memory and the chip.  A unit of neighbours is 2V elements in a row: with 16-byte
// chunks a lane that moved its own would touch half of a 32-byte sector at a time,
// twice the traffic to L2, so its row's lanes move the chunks side by side and
// trade them in shared memory (16384 tokens of 16 + 16 heads of 128, forward: fp32
// 120 us where lanes moved their own, 93 now; bf16 61, 47).  The copies land in the
// lanes' order: permuted in shared memory they were split into three times the
// requests to L2, and no faster.
template <int DT, int V, int NU, int MIX>
struct RopeLane {
  int o1[NU], o2[NU];     // bytes from the row to the two chunks of the unit
  int m1[NU], m2[NU];     // and to those that are moved
  int pair[NU];           // first pair of the unit, or -1: not turned
  bool in1[NU], in2[NU];  // the chunk exists
  bool on1[NU], on2[NU];  // as in1, in2, of those that are moved
  bool mix[NU];           // kEither
  bool swap;              // kMixed: o1 is the unit's second chunk and o2 its first
  int group;              // this lane's row among the warp's

  __device__ __forceinline__ explicit RopeLane(const RopeArgs &a) {
    const int lane = threadIdx.x & 31;
    const int L = 1 << a.lanes_log2;
    group = lane >> a.lanes_log2;
    const int punits = a.pairs / V;
    // The lanes that read shared memory together find their first chunks in half
    // of the banks: every other group of them begins with the second chunk.
    constexpr int most = V * elem_bytes(DT) == 16 ? 2 : 3;
    const int bit = a.lanes_log2 - 1 < most ? a.lanes_log2 - 1 : most;
    swap = MIX == kMixed && bit >= 0 && (lane >> bit & 1);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int u = (lane & (L - 1)) + i * L;
      int e1, e2;
      if (u < punits) {
        pair[i] = u * V;
        e1 = a.inter ? 2 * V * u : V * u;
        e2 = a.inter ? e1 + V : a.pairs + V * u;
      } else {
        pair[i] = -1;
        e1 = a.rd + 2 * V * (u - punits);
        e2 = e1 + V;
      }
      if (swap) {
        const int e = e1;
        e1 = e2;
        e2 = e;
      }
      in1[i] = e1 < a.D;
      in2[i] = e2 < a.D;
      mix[i] = a.inter && pair[i] >= 0;
      o1[i] = e1 * elem_bytes(DT);
      o2[i] = e2 * elem_bytes(DT);
      if (MIX == kMixed) {
        e1 = V * (u + i * L);
        e2 = e1 + V * L;
      }
      on1[i] = e1 < a.D;
      on2[i] = e2 < a.D;
      m1[i] = e1 * elem_bytes(DT);
      m2[i] = e2 * elem_bytes(DT);
    }
  }

  // The lane's chunks of the row at p (zeros where there are none).
  __device__ __forceinline__ void load(RopeVec<DT, V> (&v)[NU][2], const char *p, bool row) const {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      v[i][0].zero();
      v[i][1].zero();
      if (row && in1[i]) v[i][0].load(p + o1[i]);
      if (row && in2[i]) v[i][1].load(p + o2[i]);
    }
  }
  // The chunks that the lane moves, to the row at p.
  __device__ __forceinline__ void store(const RopeVec<DT, V> (&v)[NU][2], char *p) const {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (on1[i]) v[i][0].store(p + m1[i]);
      if (on2[i]) v[i][1].store(p + m2[i]);
    }
  }
  __device__ __forceinline__ void get(RopeUnit<V> (&f)[NU], const RopeVec<DT, V> (&v)[NU][2]) const {
#pragma unroll
    for (int i = 0; i < NU; ++i) f[i].template get<MIX>(v[i], mix[i]);
  }
  // A parameter row (gamma or beta); zeros for null.
  __device__ __forceinline__ void param(RopeUnit<V> (&f)[NU], const void *p) const {
    RopeVec<DT, V> v[NU][2];
    load(v, static_cast<const char *>(p), p != nullptr);
    get(f, v);
  }
};

// ---------------------------------------------------------------- angles
// An angle is a fraction of a turn: with f = inv_freq / (2 pi) as a 64-bit
// binary fraction of a turn, pos * f modulo 2^64 is the angle modulo a whole
// turn: an integer product in place of a range reduction, which adds no error of
// its own.  (A product in 32 bits is off by 0.06 radians at position 2^20.)  f is
// formed from the bits of inv_freq in integers too (float64 products, at 1/64 of
// the fp32 rate, made 333 tokens take 5.1 us instead of 4.7).  It is truncated to
// 2^-64 of a turn, and 2^66 / (2 pi) to 64 bits is off by 0.0151: together at most
// 2^-64 + inv_freq 2^-72 turns per position, which for positions up to 2^35 and
// frequencies up to 256 is 2^-25 radians.
__device__ __forceinline__ uint64_t rope_turns(double inv_freq) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(inv_freq));
  const int e = static_cast<int>(bits >> 52) & 2047;
  if (e == 0) return 0;  // below 2^-1022
  const uint64_t m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
  const uint64_t r = 0xa2f9836e4e44152aull;  // 2^66 / (2 pi)
  const uint64_t hi = __umul64hi(m, r), lo = m * r;
  // inv_freq = m 2^(e - 1075): the turns are (hi, lo) 2^(e - 1141), the fraction
  // in units of 2^-64 (hi, lo) >> s
  const int s = 1077 - e;
  uint64_t f = 0;
  if (s >= 128)
    f = 0;
  else if (s >= 64)
    f = hi >> (s - 64);
  else if (s > 0)
    f = (hi << (64 - s)) | (lo >> s);
  return bits >> 63 ? 0 - f : f;
}

// cos and sin of a fraction of a turn given as a 32-bit binary fraction: the
// nearest quarter turn exactly, the Taylor polynomials of the rest (at most an
// eighth of a turn; the first terms left out are below 2e-9 and 2e-10), then a
// turn by the quarters.
__device__ __forceinline__ void rope_sincos(uint32_t turn, float &c, float &s) {
  const uint32_t q = (turn + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(turn - (q << 30))) * 0x1p-32f;
  const float a = x * 6.283185307f, z = a * a;  // radians
  float sp = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  sp = fmaf(z, sp, 8.3333333e-3f);
  sp = fmaf(z, sp, -1.6666667e-1f);
  sp = fmaf(a * z, sp, a);
  float cp = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  cp = fmaf(z, cp, -1.3888889e-3f);
  cp = fmaf(z, cp, 4.1666667e-2f);
  cp = fmaf(z, cp, -0.5f);
  cp = fmaf(z, cp, 1.f);
  const float u = q & 1 ? sp : cp, v = q & 1 ? cp : sp;
  c = (q + 1) & 2 ? -u : u;
  s = q & 2 ? -v : v;
}

// A CTA works on one side (queries or keys), tile after tile: `tile` tokens with
// all their heads, the rows side by side over the groups of its warps.  The
// angles of a tile's tokens are computed once, each by one thread (every lane of
// a row needs its V pairs, every head the same ones: computed where they are
// used they were half of the kernel's instructions), and read from shared
// memory.  The positions of the next tile are fetched meanwhile.
constexpr int kRopeMaxTile = 64;      // tokens
constexpr int kRopeMaxAngles = 2048;  // tokens x pairs
struct RopeShared {
  // [token][V / 2 rows of][unit] (cos, cos, sin, sin) of two pairs, so that the
  // lanes of a row read side by side
  alignas(16) float cs[2 * kRopeMaxAngles];
  int64_t pos[kRopeMaxAxes * kRopeMaxTile];  // [axis][token]
};
static_assert(sizeof(RopeShared) % 16 == 0, "the ring follows");

template <int V>
struct RopeTiles {
  int64_t t;     // first token of the tile
  int64_t step;  // tokens from one tile of this CTA to the next
  int64_t pos;   // this thread's position of the next tile
  uint64_t turns;  // per position, of this thread's pair
  int n;           // tokens of the tile
  int slot;        // where the pair's cos goes in a token's angles; -1: no pair
  int row;         // the pair's axis' positions

  __device__ __forceinline__ void start(const RopeArgs &a, int side, int cta) {
    const int tile = a.tile[side];
    step = static_cast<int64_t>(a.ctas[side]) * tile;
    t = static_cast<int64_t>(cta) * tile;
    fetch(a, tile, t);
    const int p = threadIdx.x & ((1 << a.pairs_log2) - 1);
    slot = -1;
    if (p < a.pairs) {
      turns = rope_turns(a.inv_freq[p]);
      row = (static_cast<int>(a.axis[p >> 5] >> ((p & 31) * 2)) & 3) * kRopeMaxTile;
      slot = V == 1 ? 2 * p : ((p % V) / 2 * (a.pairs / V) + p / V) * 4 + (p & 1);
    }
  }
  __device__ __forceinline__ bool any(const RopeArgs &a) const { return t < a.T; }
  // Before the tile's rows: its angles (every thread of the CTA).
  __device__ __forceinline__ void angles(const RopeArgs &a, int side, RopeShared &sh) {
    const int tile = a.tile[side];
    n = static_cast<int>(min(static_cast<int64_t>(tile), a.T - t));
    if (threadIdx.x < kRopeMaxAxes * kRopeMaxTile) sh.pos[threadIdx.x] = pos;
    __syncthreads();  // the last tile's angles have been read
    fetch(a, tile, t + step);
    if (slot >= 0) {
      for (int tok = threadIdx.x >> a.pairs_log2; tok < n; tok += kRopeThreads >> a.pairs_log2) {
        const uint64_t turn = static_cast<uint64_t>(sh.pos[row + tok]) * turns;
        float c, s;
        rope_sincos(static_cast<uint32_t>(turn >> 32), c, s);
        float *cs = sh.cs + tok * 2 * a.pairs + slot;
        cs[0] = c;
        cs[V == 1 ? 1 : 2] = s * a.sign;
      }
    }
    __syncthreads();
  }

 private:
  __device__ __forceinline__ void fetch(const RopeArgs &a, int tile, int64_t t0) {
    const int axis = threadIdx.x / kRopeMaxTile, token = threadIdx.x % kRopeMaxTile;
    if (axis < a.axes && token < tile && t0 + token < a.T) {
      const int64_t i = axis * a.pos_stride + t0 + token;
      pos = a.pos64 ? static_cast<const int64_t *>(a.pos)[i]
                    : static_cast<int64_t>(static_cast<const int32_t *>(a.pos)[i]);
    }
  }
};

// cos and sin of this lane's pairs.
template <int V, int NU>
struct RopeAngles {
  static constexpr int NP = V > 1 ? V / 2 : 1;
  float2 c[NU][NP], s[NU][NP];

  // cs: the token's angles
  template <int DT, int MIX>
  __device__ __forceinline__ void get(const RopeArgs &a, const RopeLane<DT, V, NU, MIX> &l,
                                      const float *cs) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        if (l.pair[i] < 0) continue;
        if constexpr (V == 1) {
          const float2 v = *reinterpret_cast<const float2 *>(cs + 2 * l.pair[i]);
          c[i][e] = make_float2(v.x, 0.f);
          s[i][e] = make_float2(v.y, 0.f);
        } else {
          const float4 v = *reinterpret_cast<const float4 *>(
              cs + ((l.swap ? e ^ (NP / 2) : e) * (a.pairs / V) + l.pair[i] / V) * 4);
          c[i][e] = make_float2(v.x, v.y);
          s[i][e] = make_float2(v.z, v.w);
        }
      }
    }
  }

  __device__ __forceinline__ void turn(int i, RopeUnit<V> &f) const {
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const float2 u = f.u[e], w = f.w[e], ns = mul2(s[i][e], splat2(-1.f));
      f.u[e] = fma2(u, c[i][e], mul2(w, ns));
      f.w[e] = fma2(w, c[i][e], mul2(u, s[i][e]));
    }
  }
};

// A thread's rows of a tile: one in every round, `per` rows apart, as addresses
// that move on by additions (a token's end adds another step).
template <int N>
struct RopeRow {
  const char *p[N];
  const char *base[N];             // token 0's row of the first round
  int64_t token[N], step[N], wrap[N];  // bytes: a token; a round; past the last head
  int h, h0, dh, H;
  int tok, t0, dt;                 // token within the tile; in the first round; its step

  template <int DT>
  __device__ __forceinline__ void start(const RopeArgs &a, int side, const void *const *bases,
                                        const int64_t *ts, const int64_t *hs, int first, int per) {
    constexpr int es = elem_bytes(DT);
    H = a.side[side].H;
    t0 = a.by_H[side](first);
    dt = a.by_H[side](per);
    h0 = first - t0 * H;
    dh = per - dt * H;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      base[k] = static_cast<const char *>(bases[k]) + (t0 * ts[k] + h0 * hs[k]) * es;
      token[k] = ts[k] * es;
      step[k] = (dt * ts[k] + dh * hs[k]) * es;
      wrap[k] = (ts[k] - H * hs[k]) * es;
    }
  }
  // The first round of the tile at token t.
  __device__ __forceinline__ void at(int64_t t) {
    h = h0;
    tok = t0;
#pragma unroll
    for (int k = 0; k < N; ++k) p[k] = base[k] + t * token[k];
  }
  __device__ __forceinline__ void next() {
    h += dh;
    const bool over = h >= H;
    if (over) h -= H;
    tok += over ? dt + 1 : dt;
#pragma unroll
    for (int k = 0; k < N; ++k) p[k] += over ? step[k] + wrap[k] : step[k];
  }
};

// ------------------------------------------------------------- row ring
// The rounds of a CTA's tiles in turn, a row per group and round, fetched S - 1
// rounds ahead by asynchronous copies that every thread makes for itself: the
// lane's chunks of N tensors (x, or x and dy) into its own slots of shared
// memory, zeros where there is no row.  No registers hold what is in flight and
// no barrier joins the threads.  A round is fetched into the slots of the one
// before the round that is being read, whose values have been used up.
// With pairs of neighbours (kMixed) a unit's chunks are read from the slots of the
// lanes that moved them, and the results go out the same way, through the slots of
// the round that was read: the warp waits for itself at both.
template <int DT, int V, int NU, int MIX, int N, int S>
struct RopeRing {
  static constexpr int kBytes = RopeVec<DT, V>::kBytes;
  static constexpr uint32_t kStage = kRopeThreads * N * 2 * NU * kBytes;
  static constexpr uint32_t kTotal = S * kStage;

  uint32_t slot;       // shared-memory address of this thread's first slot
  uint32_t unit[2];    // kMixed: of the slots of its first unit's chunks
  RopeRow<N> row;      // the row that is fetched next
  int64_t t;           // its tile
  int left;            // rows of the tile from the round's first on
  uint32_t stage, now; // byte offsets of the stages that are fetched into and read next

  __device__ __forceinline__ void start(const RopeArgs &a, int side,
                                        const RopeLane<DT, V, NU, MIX> &l, const void *ring,
                                        int64_t first_tile, int first, int per) {
    slot = smem_addr(ring) + threadIdx.x * kBytes;
    if constexpr (MIX == kMixed) {
      const int l2 = a.lanes_log2, L = 1 << l2, sub = threadIdx.x & (L - 1);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int chunk = 2 * sub + (c ^ int(l.swap));
        unit[c] = slot + static_cast<uint32_t>((chunk >> l2) * kRopeThreads - sub +
                                               (chunk & (L - 1))) * kBytes;
      }
    }
    t = first_tile;
    stage = now = 0;
    const RopeSide &s = a.side[side];
    const void *base[2] = {s.x, s.dy};
    const int64_t ts[2] = {s.xt, s.dt}, hs[2] = {s.xh, s.dh};
    row.template start<DT>(a, side, base, ts, hs, first, per);
    begin(a, side);
  }
  __device__ __forceinline__ void begin(const RopeArgs &a, int side) {
    left = 0;
    if (t >= a.T) return;
    left = static_cast<int>(min(static_cast<int64_t>(a.tile[side]), a.T - t)) * a.side[side].H;
    row.at(t);
  }
  static __device__ __forceinline__ uint32_t at(int k, int i, int c) {
    return static_cast<uint32_t>(((k * NU + i) * 2 + c) * kRopeThreads * kBytes);
  }
  // The chunk c of this lane's unit.
  __device__ __forceinline__ uint32_t own(int k, int i, int c) const {
    return MIX == kMixed ? unit[c] + at(k, i, 0) : slot + at(k, i, c);
  }
  static __device__ __forceinline__ void copy(uint32_t dst, const char *src, bool on) {
    if constexpr (kBytes == 16) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                   "r"(on ? 16 : 0)
                   : "memory");
    } else if constexpr (kBytes >= 4) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src),
                   "n"(kBytes), "r"(on ? kBytes : 0)
                   : "memory");
    } else {
      const uint16_t v = on ? *reinterpret_cast<const uint16_t *>(src) : uint16_t(0);
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst), "h"(v) : "memory");
    }
  }
  // Fetches the next round.
  __device__ __forceinline__ void fetch(const RopeArgs &a, int side, const RopeLane<DT, V, NU, MIX> &l,
                                        int first, int per) {
    if (left > 0) {
      const bool on = first < left;
#pragma unroll
      for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          copy(slot + stage + at(k, i, 0), row.p[k] + l.m1[i], on && l.on1[i]);
          copy(slot + stage + at(k, i, 1), row.p[k] + l.m2[i], on && l.on2[i]);
        }
      }
      left -= per;
      row.next();
      if (left <= 0) {
        t += static_cast<int64_t>(a.ctas[side]) * a.tile[side];
        begin(a, side);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    stage = stage + kStage == kTotal ? 0u : stage + kStage;
  }
  // Waits for the oldest round in flight.
  template <int LEFT>
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
    if constexpr (MIX == kMixed) __syncwarp();
  }
  // On to the next round.
  __device__ __forceinline__ void step() {
    now = now + kStage == kTotal ? 0u : now + kStage;
  }
  __device__ __forceinline__ void read(RopeVec<DT, V> (&v)[NU][2], int k) const {
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) get(v[i][c], own(k, i, c) + now);
  }
  // From the units' own chunks to those that the lane moves, through the slots of
  // the round that was read.
  __device__ __forceinline__ void trade(RopeVec<DT, V> (&v)[NU][2]) const {
    if constexpr (MIX == kMixed) {
#pragma unroll
      for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) put(v[i][c], own(0, i, c) + now);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) get(v[i][c], slot + now + at(0, i, c));
    }
  }

 private:
  static __device__ __forceinline__ void get(RopeVec<DT, V> &v, uint32_t p) {
    uint32_t *w = v.w;
    if constexpr (kBytes == 16) {
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(p)
                   : "memory");
    } else if constexpr (kBytes == 8) {
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(p) : "memory");
    } else if constexpr (kBytes == 4) {
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(p) : "memory");
    } else {
      uint16_t h;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(p) : "memory");
      w[0] = h;
    }
  }
  static __device__ __forceinline__ void put(const RopeVec<DT, V> &v, uint32_t p) {
    const uint32_t *w = v.w;
    if constexpr (kBytes == 16)
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(w[0]), "r"(w[1]),
                   "r"(w[2]), "r"(w[3])
                   : "memory");
    else
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(p), "r"(w[0]), "r"(w[1]) : "memory");
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
template <int MODE, int DT, int V, int NU, int MIX>
__device__ __forceinline__ float rope_stats(const RopeArgs &a, const RopeLane<DT, V, NU, MIX> &l,
                                            RopeUnit<V> (&f)[NU]) {
  constexpr int NP = RopeUnit<V>::NP;
  if constexpr (MODE == kLayer) {
    float2 m = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < NP; ++e) m = add2(m, add2(f[i].u[e], f[i].w[e]));
    const float mean = rope_sum(m.x + m.y, a.lanes_log2) * a.invD;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const float2 m1 = splat2(l.in1[i] ? -mean : 0.f), m2 = splat2(l.in2[i] ? -mean : 0.f);
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        // (mixed, the first half of u and w is the first chunk; with kEither a
        // unit that lacks its second chunk is not mixed)
        const bool one = MIX != kMixed || e < NP / 2;
        f[i].u[e] = add2(f[i].u[e], one ? m1 : m2);
        f[i].w[e] = add2(f[i].w[e], MIX == kMixed && one ? m1 : m2);
        if (V == 1) f[i].u[e].y = f[i].w[e].y = 0.f;
      }
    }
  }
  float2 q = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < NP; ++e) q = fma2(f[i].w[e], f[i].w[e], fma2(f[i].u[e], f[i].u[e], q));
  return rsqrtf(fmaf(rope_sum(q.x + q.y, a.lanes_log2), a.invD, a.eps));
}


// Kernels, and the shared memory of their rings.
const void *rope_fwd_kernel_ptr(int dt, int V, int NU, int mode, bool inter);
const void *rope_bwd_kernel_ptr(int dt, int V, int mode, bool inter);
inline uint32_t rope_ring_bytes(int dt, int V, int NU, int rounds) {
  return uint32_t(kRopeThreads * 2 * NU * V * elem_bytes(dt)) * rounds;
}
const void *rope_fold_kernel_ptr();
// Floats of shared memory that the backward's last fold takes.
__host__ __device__ inline int rope_fold_floats(int D, bool layer) {
  return (kRopeThreads / 32) * D * (layer ? 2 : 1);
}

}  // namespace gbn
