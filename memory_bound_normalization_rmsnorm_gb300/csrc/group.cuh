// group.cuh -- shared pieces of the group-normalisation kernels
// (group_fwd.cu, group_bwd.cu): arguments, the activation and its
// derivative, per-channel accumulators and their folds.
//
// x is [B, S, C], channels last: a sample is S rows of C contiguous
// channels, and group g of a sample owns the D = C / G channels [g D, (g+1)
// D) of every one of its rows.  A thread owns one 16-byte chunk column (V
// channels) and every R-th row of its CTA's row range, so its accumulators
// are per channel whatever D is; channels meet in groups only after the rows
// are folded.
//
// Two forms.  Resident: a cluster of k CTAs owns a slab of whole groups of
// one sample, each CTA a range of its rows, copied once into shared memory
// (each thread reads back only the chunks that it copied itself: the copy
// needs no barrier), so x (and dy) is read from HBM once.  Streamed: the
// sample is read twice, by a statistics kernel and an output kernel whose
// CTAs own the same row ranges and walk them in opposite directions, so the
// second read starts with what the first left in L2.
#pragma once
#include "dropout.cuh"

namespace gbn {

// Activations, with the values of norm_act_t: act(z) = z * sigmoid(k(z)).
constexpr int kActNone = 0;
constexpr int kActSilu = 1;  // k = z
constexpr int kActGelu = 2;  // k = 2 sqrt(2 / pi) (z + 0.044715 z^3): the tanh form

constexpr int kGroupThreads = 512;  // largest CTA of these kernels

struct GroupArgs {
  const void *x;      // [B, S, C]
  const void *dy;     // [B, S, C] (backward)
  const void *gamma;  // [C]
  const void *beta;   // [C] or null
  void *out;          // y or dx [B, S, C]
  float *mean;        // [B, G]: written by forward, read by backward
  float *rstd;        // [B, G]
  float *gpart;       // streamed: per-(sample, split, group) pairs [B, splits, G, 2]
  float *cpart;       // backward: per-channel partial rows [P, C] (dgamma), then [P, C] (dbeta)
  float *dbeta_part;  // backward: where the dbeta rows start, or null
  DropArgs drop;
  int B, S, C, G, D;
  int nc;      // 16-byte chunks per row
  int sg;      // groups per slab
  int ncs;     // chunk columns per (full) slab
  int nslab;   // slabs per sample
  int k;       // CTAs per cluster (row split of a unit)
  int R;       // row lanes per CTA
  int slots;   // resident: rows per thread (at most)
  int splits;  // streamed: row ranges per sample
  float eps;
};

// Shared memory after the resident data: the fold buffers (also the
// per-channel arrays, which are written after the folds), then two float2
// per group of the slab.
__host__ __device__ inline uint32_t group_fold_bytes(int R, int ncs, int V) {
  const uint32_t tree = static_cast<uint32_t>(R / 2) * static_cast<uint32_t>(ncs) *
                        (static_cast<uint32_t>(V) * 8u + 4u);
  const uint32_t chan = static_cast<uint32_t>(ncs) * static_cast<uint32_t>(V) * 8u;
  return ((tree > chan ? tree : chan) + 15u) & ~15u;
}
__host__ __device__ inline uint32_t group_smem_bytes(int slots, int ntensors, int R, int ncs, int V,
                                                     int sg) {
  return static_cast<uint32_t>(slots) * static_cast<uint32_t>(ncs * R) * 16u *
             static_cast<uint32_t>(ntensors) +
         group_fold_bytes(R, ncs, V) + static_cast<uint32_t>(sg) * 16u;
}

// ---------------------------------------------------------- activation
__device__ __forceinline__ float sigmoid_fast(float k) {
  // exp(-k) overflows to infinity for k below -88, and 1 / infinity is 0.
  return __fdividef(1.0f, 1.0f + __expf(-k));
}

constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == kActNone) return z;
  if constexpr (ACT == kActSilu) return z * sigmoid_fast(z);
  const float k = z * fmaf(kGeluC * kGeluA * z, z, kGeluC);
  return z * sigmoid_fast(k);
}

// act'(z) = s + z s (1 - s) k'(z), s = sigmoid(k(z)).  Where s (1 - s) has
// rounded to 0 the second term is 0, though z k'(z) may be infinite there.
template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if constexpr (ACT == kActNone) return 1.0f;
  if constexpr (ACT == kActSilu) {
    const float s = sigmoid_fast(z);
    return fmaf(z * s, 1.0f - s, s);
  }
  const float z2 = z * z;
  const float s = sigmoid_fast(z * fmaf(kGeluC * kGeluA, z2, kGeluC));
  const float t = s * (1.0f - s);
  const float zk = z * fmaf(3.0f * kGeluC * kGeluA, z2, kGeluC);
  return t == 0.0f ? s : fmaf(zk, t, s);
}

// ------------------------------------------------- asynchronous copies
__device__ __forceinline__ void cp_async_16(void *dst_smem, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst_smem)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Waits until at most `pending` of this thread's newest copy groups are
// outstanding (fewer when more than 7 are).
__device__ __forceinline__ void cp_async_wait_upto(int pending) {
  switch (pending) {
    case 0: cp_async_wait<0>(); break;
    case 1: cp_async_wait<1>(); break;
    case 2: cp_async_wait<2>(); break;
    case 3: cp_async_wait<3>(); break;
    case 4: cp_async_wait<4>(); break;
    case 5: cp_async_wait<5>(); break;
    case 6: cp_async_wait<6>(); break;
    default: cp_async_wait<7>(); break;
  }
}

// ------------------------------------------- per-channel accumulators
// Running (count, mean, M2) of a thread's V channels.  Rows enter in blocks
// of four whose own mean and squared deviations are formed first, then
// merged, so no sum of squares is ever taken about a distant origin: the
// statistics keep their accuracy whatever the ratio of mean to deviation.
template <int V>
struct ChannelStats {
  float2 m[V / 2], q[V / 2];
  float n;

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int p = 0; p < V / 2; ++p) m[p] = q[p] = splat2(0.f);
    n = 0.f;
  }
  __device__ __forceinline__ void add4(const float2 (&a)[V / 2], const float2 (&b)[V / 2],
                                       const float2 (&c)[V / 2], const float2 (&d)[V / 2]) {
    const float w = __fdividef(4.f, n + 4.f);
    const float2 w2 = splat2(w), nw = splat2(n * w), quarter = splat2(0.25f);
#pragma unroll
    for (int p = 0; p < V / 2; ++p) {
      const float2 mb = mul2(add2(add2(a[p], b[p]), add2(c[p], d[p])), quarter);
      const float2 nm = make_float2(-mb.x, -mb.y);
      const float2 da = add2(a[p], nm), db = add2(b[p], nm), dc = add2(c[p], nm),
                   dd = add2(d[p], nm);
      const float2 qb = fma2(da, da, fma2(db, db, fma2(dc, dc, mul2(dd, dd))));
      if (n == 0.f) {
        m[p] = mb;
        q[p] = qb;
      } else {
        const float2 e = add2(mb, make_float2(-m[p].x, -m[p].y));
        m[p] = fma2(e, w2, m[p]);
        q[p] = add2(q[p], fma2(mul2(e, e), nw, qb));
      }
    }
    n += 4.f;
  }
  __device__ __forceinline__ void add1(const float2 (&a)[V / 2]) {
    const float w = __fdividef(1.f, n + 1.f);
    const float2 w2 = splat2(w), nw = splat2(n * w);
#pragma unroll
    for (int p = 0; p < V / 2; ++p) {
      if (n == 0.f) {
        m[p] = a[p];
      } else {
        const float2 e = add2(a[p], make_float2(-m[p].x, -m[p].y));
        m[p] = fma2(e, w2, m[p]);
        q[p] = fma2(mul2(e, e), nw, q[p]);
      }
    }
    n += 1.f;
  }
  // Merge of another partial over nb rows.
  __device__ __forceinline__ void merge(const float2 (&mb)[V / 2], const float2 (&qb)[V / 2],
                                        float nb) {
    if (nb == 0.f) return;
    const bool none = n == 0.f;
    const float w = __fdividef(nb, n + nb);
    const float2 w2 = splat2(w), nw = splat2(n * w);
#pragma unroll
    for (int p = 0; p < V / 2; ++p) {
      if (none) {
        m[p] = mb[p];
        q[p] = qb[p];
      } else {
        const float2 e = add2(mb[p], make_float2(-m[p].x, -m[p].y));
        m[p] = fma2(e, w2, m[p]);
        q[p] = add2(q[p], fma2(mul2(e, e), nw, qb[p]));
      }
    }
    n += nb;
  }
};

template <int V>
__device__ __forceinline__ void put_pairs(float4 *buf, int cap, int slot, const float2 (&a)[V / 2],
                                          const float2 (&b)[V / 2]) {
#pragma unroll
  for (int j = 0; j < V / 4; ++j) {
    buf[j * cap + slot] = make_float4(a[2 * j].x, a[2 * j].y, a[2 * j + 1].x, a[2 * j + 1].y);
    buf[(V / 4 + j) * cap + slot] =
        make_float4(b[2 * j].x, b[2 * j].y, b[2 * j + 1].x, b[2 * j + 1].y);
  }
}
template <int V>
__device__ __forceinline__ void get_pairs(const float4 *buf, int cap, int slot, float2 (&a)[V / 2],
                                          float2 (&b)[V / 2]) {
#pragma unroll
  for (int j = 0; j < V / 4; ++j) {
    const float4 u = buf[j * cap + slot], w = buf[(V / 4 + j) * cap + slot];
    a[2 * j] = make_float2(u.x, u.y);
    a[2 * j + 1] = make_float2(u.z, u.w);
    b[2 * j] = make_float2(w.x, w.y);
    b[2 * j + 1] = make_float2(w.z, w.w);
  }
}

// Folds the R row lanes of each chunk column into lane 0, pairwise in a
// fixed order.  Called by every thread of the CTA; `on`: the thread owns a
// chunk column.  Ends with a barrier.
template <int V>
__device__ __forceinline__ void fold_stats(ChannelStats<V> &st, unsigned char *buf, int R, int rl,
                                           int cc, int ncs, bool on) {
  float4 *f4 = reinterpret_cast<float4 *>(buf);
  const int cap = (R / 2) * ncs;
  float *cnt = reinterpret_cast<float *>(f4 + (V / 2) * cap);
  for (int r = R; r > 1;) {
    const int h = (r + 1) >> 1;
    if (on && rl >= h && rl < r) {
      put_pairs<V>(f4, cap, (rl - h) * ncs + cc, st.m, st.q);
      cnt[(rl - h) * ncs + cc] = st.n;
    }
    __syncthreads();
    if (on && rl < r - h) {
      float2 mb[V / 2], qb[V / 2];
      get_pairs<V>(f4, cap, rl * ncs + cc, mb, qb);
      st.merge(mb, qb, cnt[rl * ncs + cc]);
    }
    __syncthreads();
    r = h;
  }
}
template <int V>
__device__ __forceinline__ void fold_sums(float2 (&a)[V / 2], float2 (&b)[V / 2],
                                          unsigned char *buf, int R, int rl, int cc, int ncs,
                                          bool on) {
  float4 *f4 = reinterpret_cast<float4 *>(buf);
  const int cap = (R / 2) * ncs;
  for (int r = R; r > 1;) {
    const int h = (r + 1) >> 1;
    if (on && rl >= h && rl < r) put_pairs<V>(f4, cap, (rl - h) * ncs + cc, a, b);
    __syncthreads();
    if (on && rl < r - h) {
      float2 ao[V / 2], bo[V / 2];
      get_pairs<V>(f4, cap, rl * ncs + cc, ao, bo);
#pragma unroll
      for (int p = 0; p < V / 2; ++p) {
        a[p] = add2(a[p], ao[p]);
        b[p] = add2(b[p], bo[p]);
      }
    }
    __syncthreads();
    r = h;
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// (mean, M2) of a group from the (mean, M2) of its D channels over n rows
// each, by one warp; every lane returns the result.
__device__ __forceinline__ float2 group_of_channels(const float *chm, const float *chq, int D,
                                                    float n) {
  const int lane = threadIdx.x & 31;
  float s = 0.f;
  for (int j = lane; j < D; j += 32) s += chm[j];
  const float gm = warp_sum(s) / static_cast<float>(D);
  float q = 0.f;
  for (int j = lane; j < D; j += 32) {
    const float e = chm[j] - gm;
    q += fmaf(n * e, e, chq[j]);
  }
  return make_float2(gm, warp_sum(q));
}

// Address of the V-element chunk column cc (within the tensor) of row s of
// sample b, in elements.
__device__ __forceinline__ int64_t group_elem(const GroupArgs &a, int b, int64_t s, int chunk,
                                              int V) {
  return (static_cast<int64_t>(b) * a.S + s) * a.C + static_cast<int64_t>(chunk) * V;
}

// First row of part i of n equal parts of S rows.
__host__ __device__ inline int64_t part_begin(int64_t S, int i, int n) { return S * i / n; }

// Parameters of a thread's V channels as fp32 pairs: gamma, beta (0 when
// absent).
template <int DT>
__device__ __forceinline__ void load_affine(const GroupArgs &a, int chunk,
                                            float2 (&gf)[chunk_elems(DT) / 2],
                                            float2 (&bf)[chunk_elems(DT) / 2]) {
  unpack<DT>(ld_global_nc_v4(static_cast<const uint4 *>(a.gamma) + chunk), gf);
  uint4 bv = make_uint4(0, 0, 0, 0);
  if (a.beta) bv = ld_global_nc_v4(static_cast<const uint4 *>(a.beta) + chunk);
  unpack<DT>(bv, bf);
}

const void *group_fwd_kernel_ptr(int dt, int act, bool drop);     // resident
const void *group_stats_kernel_ptr(int dt);                       // streamed, first pass
const void *group_apply_kernel_ptr(int dt, int act, bool drop);   // streamed, second pass
const void *group_bwd_kernel_ptr(int dt, int act, bool drop);     // resident
const void *group_sums_kernel_ptr(int dt, int act, bool drop);    // streamed, first pass
const void *group_dx_kernel_ptr(int dt, int act, bool drop);      // streamed, second pass

}  // namespace gbn
