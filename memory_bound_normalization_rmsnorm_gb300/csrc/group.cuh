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
// Three forms.  Resident, for small samples: a cluster of k CTAs owns a slab
// of whole groups of one sample, each CTA a range of its rows, copied once
// into shared memory (each thread reads back only the chunks that it copied
// itself: the copy needs no barrier), so x (and dy) is read from HBM once.
// Ring, for large samples: one cooperative kernel over the whole GPU whose
// CTAs keep what fits of their rows in shared memory between the statistics
// and the output pass and read the rest again, newest first, out of L2
// (group_ring.cu).  Streamed, for groups wider than a CTA: a statistics and
// an output kernel over the same row ranges, walked in opposite directions.
#pragma once
#include "dropout.cuh"

namespace gbn {

// Activations, with the values of norm_act_t: act(z) = z * sigmoid(k(z)).
constexpr int kActNone = 0;
constexpr int kActSilu = 1;  // k = z
constexpr int kActGelu = 2;  // k = 2 sqrt(2 / pi) (z + 0.044715 z^3): the tanh form

constexpr int kGroupThreads = 512;  // largest CTA of these kernels
constexpr int kMaxGroupCluster = 8;  // the portable size
// Ring: rows per thread and tile.
constexpr int kRingRowsFwd = 8;
constexpr int kRingRowsBwd = 4;
// Ring: tiles that tensor memory holds (a thread's chunks of a tile are 32
// 32-bit columns of its lane; four warps share the 512 columns of a lane).
constexpr int kRingTmemTiles = 4;

// Division of n (0 <= n < 2^31) by a divisor known to the host, d >= 1: with
// l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d = (hi(m n) + n)
// >> l (Granlund and Montgomery, "Division by invariant integers using
// multiplication", PLDI 1994; n + hi(m n) stays below 2^32 here).  A CTA starts
// with several divisions, one after the other, before its first copy.
struct FastDiv {
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

// Quotients by a divisor known to the host, with r = 1 / d rounded to nearest: a
// product and one correction give the correctly rounded quotient (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// IBM J. Res. Dev. 34, 1990) in three operations; a division in its place, three
// times in a row between the copies and the output, cost 1 x 64 x 1280 0.13 us of
// 3.3.  Infinities pass as they are (the correction would make them NaN).
struct FloatDiv {
  float d, r;
  void set(int64_t n) {
    d = static_cast<float>(n);
    r = 1.0f / d;
  }
  __device__ __forceinline__ float operator()(float a) const {
    const float q = a * r;
    return isinf(q) ? q : fmaf(fmaf(-q, d, a), r, q);
  }
};

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
  float *dgamma;      // ring backward: [C] outputs (dbeta may be null)
  float *dbeta;
  DropArgs drop;
  int B, S, C, G, D;
  int nc;      // 16-byte chunks per row
  int sg;      // groups per slab
  int ncs;     // chunk columns per (full) slab
  int nslab;   // slabs per sample
  int k;       // resident: CTAs that share a slab's rows
  int cb;      // resident backward: samples per cluster (1 or B)
  FastDiv by_ncs, by_k, by_csize, by_nslab, by_splits, by_R, by_D;  // csize = k cb
  int pq, prem;  // S rows in k (resident) or `splits` ranges: quotient, remainder
  FloatDiv f_S, f_D, f_SD;   // by the positions, the channels of a group, its values
  FloatDiv f_rows, f_rows1;  // by the rows of a range, pq and pq + 1
  int R;       // row lanes per CTA
  int slots;   // resident: rows per thread (at most)
  int splits;  // streamed and ring: row ranges per sample
  int lsh;     // log2 of the lanes that share a group in the folds
  int U;       // ring: rows per thread and tile
  int stages;  // ring: tiles in shared memory
  int nsamp;   // ring: samples per round
  int rounds;  // ring: ceil(B / nsamp)
  int tm;      // ring: tiles per CTA that tensor memory holds between the passes
  int keep;    // ring: tiles per CTA that L2 is asked to hold
  unsigned *err;  // device error word
  float eps;
};

// Shared memory after the resident data: the fold buffer (V pairs and a count
// per slot, half of R slots per column; a single row lane needs none), the
// two per-channel arrays, then two float2 per group of the slab.
__host__ __device__ inline uint32_t group_fold_bytes(int R, int ncs, int V) {
  if (R == 1) return 0;
  const uint32_t slots = static_cast<uint32_t>((R + 1) / 2) * static_cast<uint32_t>(ncs);
  return (slots * (static_cast<uint32_t>(V) * 8u + 4u) + 15u) & ~15u;
}
__host__ __device__ inline uint32_t group_chan_bytes(int ncs, int V) {
  return static_cast<uint32_t>(ncs * V) * 8u;
}
// The ring kernels: `stages` tiles of U * R rows (one per tensor), the fold
// buffer, the per-channel arrays, the backward's running per-channel totals,
// a float2 per group of the slab, the stages' full and free mbarriers, and
// the abort flag with the tensor-memory address.
constexpr int kGroupRingSplits = 192;  // row ranges of a sample, at most
struct GroupRingLayout {
  uint32_t tensor_bytes, stage_bytes, fold_off, chan_off, tot_off, gst_off, bar_off, flag_off,
      total;
};
__host__ __device__ inline GroupRingLayout group_ring_layout(int stages, int U, int R, int ncs,
                                                             int V, int sg, bool bwd) {
  GroupRingLayout L;
  L.tensor_bytes = static_cast<uint32_t>(U * R * ncs) * 16u;
  L.stage_bytes = L.tensor_bytes * (bwd ? 2u : 1u);
  L.fold_off = L.stage_bytes * static_cast<uint32_t>(stages);
  L.chan_off = L.fold_off + group_fold_bytes(R, ncs, V);
  // (the backward's column sums need a float per thread from fold_off on)
  if (bwd && L.chan_off < L.fold_off + 4u * kGroupThreads)
    L.chan_off = L.fold_off + 4u * kGroupThreads;
  L.tot_off = L.chan_off + group_chan_bytes(ncs, V);
  L.gst_off = L.tot_off + (bwd ? group_chan_bytes(ncs, V) : 0u);
  L.bar_off = L.gst_off + static_cast<uint32_t>(sg) * 8u;
  L.flag_off = L.bar_off + 16u * static_cast<uint32_t>(stages);
  L.total = align16(L.flag_off + 8u);  // abort flag, tensor-memory address
  return L;
}
__host__ __device__ inline uint32_t group_smem_bytes(int slots, int ntensors, int R, int ncs, int V,
                                                     int sg) {
  return static_cast<uint32_t>(slots) * static_cast<uint32_t>(ncs * R) * 16u *
             static_cast<uint32_t>(ntensors) +
         group_fold_bytes(R, ncs, V) + group_chan_bytes(ncs, V) + static_cast<uint32_t>(sg) * 16u;
}

// ---------------------------------------------------------- activation
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// s = sigmoid(k) and e = exp(-k) (so 1 - s = e s, without cancellation) of the
// same two channels in two rows, a and b: one reciprocal of (1 + e_a)(1 + e_b)
// serves both rows, six special-function operations instead of eight (their
// rate, 16 a cycle and SM, bounds the passes that take an activation).  Rows
// of one channel share a group, so a NaN that reaches the other row through
// the product finds it NaN already (the group's statistics are).  Needs k >=
// -43.6, which keeps the product finite.
// Accuracy, u = 2^-24: k log2(e) is rounded (2 u with its constant) and the
// exponential is off by two steps, so e is by (2 |k| + 4) u of itself; that
// reaches s times 1 - s, and the reciprocal with its products adds 5 u.  z s is off
// by 6 u of itself and, for SiLU, by at most |z| s (1 - s) (2 |z| + 4) u < 1.8 u
// beside: far below a rounding to 16 bits, and for fp32 results of size 1 a few
// steps, which is why the exponent is not carried in two parts.
__device__ __forceinline__ void sigmoid_rows(float2 ka, float2 kb, float2 &sa, float2 &sb,
                                             float2 &ea, float2 &eb) {
  const float2 ta = mul2(ka, splat2(-1.4426950408889634f));
  const float2 tb = mul2(kb, splat2(-1.4426950408889634f));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ea.x) : "f"(ta.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ea.y) : "f"(ta.y));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(eb.x) : "f"(tb.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(eb.y) : "f"(tb.y));
  const float2 da = add2(ea, splat2(1.f)), db = add2(eb, splat2(1.f));
  const float2 p = mul2(da, db);
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(p.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(p.y));
  sa = mul2(db, r);
  sb = mul2(da, r);
}

constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// Arguments are clamped below where act(z) has fallen to 5e-18 (there it
// stays: 18 orders below the argument), and for GELU's derivative above
// where it is 1, so that z^3 cannot overflow into it.
constexpr float kSiluMin = -43.6f;
constexpr float kGeluMin = -7.6f;  // k = -43.4
constexpr float kGeluMax = 12.0f;

template <int ACT>
__device__ __forceinline__ float2 clamp_low(float2 z) {
  constexpr float lo = ACT == kActSilu ? kSiluMin : kGeluMin;
  return make_float2(max_nan(z.x, lo), max_nan(z.y, lo));
}

// k(z) of a clamped argument.
template <int ACT>
__device__ __forceinline__ float2 act_arg(float2 z) {
  if constexpr (ACT == kActSilu) return z;
  return mul2(z, fma2(mul2(z, z), splat2(kGeluC * kGeluA), splat2(kGeluC)));
}

// a, b: z of the same two channels in two rows, replaced by act(z).
template <int ACT>
__device__ __forceinline__ void act_rows(float2 &a, float2 &b) {
  if constexpr (ACT != kActNone) {
    a = clamp_low<ACT>(a);
    b = clamp_low<ACT>(b);
    float2 sa, sb, ea, eb;
    sigmoid_rows(act_arg<ACT>(a), act_arg<ACT>(b), sa, sb, ea, eb);
    a = mul2(a, sa);
    b = mul2(b, sb);
  }
}

// a, b: z, replaced by act'(z) = s + z s (1 - s) k'(z), s = sigmoid(k(z)).
template <int ACT>
__device__ __forceinline__ void act_grad_rows(float2 &a, float2 &b) {
  a = clamp_low<ACT>(a);
  b = clamp_low<ACT>(b);
  float2 sa, sb, ea, eb;
  if constexpr (ACT == kActSilu) {
    sigmoid_rows(a, b, sa, sb, ea, eb);
    a = fma2(mul2(a, sa), mul2(ea, sa), sa);
    b = fma2(mul2(b, sb), mul2(eb, sb), sb);
  } else {
    a = make_float2(min_nan(a.x, kGeluMax), min_nan(a.y, kGeluMax));
    b = make_float2(min_nan(b.x, kGeluMax), min_nan(b.y, kGeluMax));
    const float2 c1 = splat2(kGeluC), c3 = splat2(kGeluC * kGeluA),
                 c9 = splat2(3.0f * kGeluC * kGeluA);
    const float2 a2 = mul2(a, a), b2 = mul2(b, b);
    sigmoid_rows(mul2(a, fma2(a2, c3, c1)), mul2(b, fma2(b2, c3, c1)), sa, sb, ea, eb);
    a = fma2(mul2(mul2(a, fma2(a2, c9, c1)), sa), mul2(ea, sa), sa);
    b = fma2(mul2(mul2(b, fma2(b2, c9, c1)), sb), mul2(eb, sb), sb);
  }
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

// Arrival at the barrier that keeps a cluster's CTAs from leaving while a peer
// may still read their shared memory.  It passes on no data, so it is relaxed: a
// releasing one waits for the thread's global stores.  The thread's reads of the
// peers have to be complete, so every value read has to have been used (shuffled
// or stored): a read whose value nothing waits for may still be on its way.  2 x
// 221 x 88 backward 5.3 -> 5.0 us, 3 x 1517 x 168 fp32 forward 5.8 -> 5.55.
__device__ __forceinline__ void cluster_arrive_leave() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

// ------------------------------------------- per-channel accumulators
// Running (count, mean, M2) of a thread's V channels.  Rows enter in blocks
// of four whose own mean and squared deviations are formed first, then
// merged, so no sum of squares is ever taken about a distant origin: the
// statistics keep their accuracy whatever the ratio of mean to deviation.  The
// merge weights are approximate quotients (2 steps): they multiply differences
// of means, which are of the deviation's size, and an error of the mean reaches
// the variance in the second order only.
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Row lanes that the pairwise folds leave: few enough for the loops over
// them that follow, at most half of R, rounded up (the slots per column that
// the buffer holds).
constexpr int kFoldLanes = 8;
__host__ __device__ inline int fold_lanes(int R) {
  if (R == 1) return 1;
  do R = (R + 1) / 2;
  while (R > kFoldLanes);
  return R;
}

// Folds the R > 1 row lanes of each chunk column pairwise, in a fixed order, to
// fold_lanes(R), and leaves those in the buffer: lane l of column cc in slot l
// * ncs + cc (see put_pairs; a partner's slot is the one its sum goes back
// to).  Called by every thread of the CTA; `on`: the thread owns a chunk
// column.  Ends with a barrier.  `merge(slot)` adds the partial in a slot to
// the thread's, `put(slot)` writes the thread's there.
template <typename Merge, typename Put>
__device__ __forceinline__ void fold_rows(int R, int rl, int cc, int ncs, bool on, Merge merge,
                                          Put put) {
  int r = R;
  const int left = fold_lanes(R);
  while (r > left) {
    const int h = (r + 1) >> 1;
    if (r < R) __syncthreads();  // the slots of the last level have been read
    if (on && rl >= h && rl < r) put((rl - h) * ncs + cc);
    __syncthreads();
    if (on && rl < r - h) merge(rl * ncs + cc);
    r = h;
  }
  // (an odd level's middle lane had no partner, so no slot was read there)
  if (on && rl < r) put(rl * ncs + cc);
  __syncthreads();
}

// Where value v of a slot lies in the buffer of put_pairs (first array: b =
// 0, second: 1).
template <int V>
__device__ __forceinline__ int pair_at(int cap, int slot, int v, int b) {
  return ((b * (V / 4) + (v >> 2)) * cap + slot) * 4 + (v & 3);
}
// Slots per column in the fold buffer.
__host__ __device__ inline int fold_slots(int R) { return (R + 1) / 2; }

template <int V>
__device__ __forceinline__ void fold_stats(ChannelStats<V> &st, unsigned char *buf, int R, int rl,
                                           int cc, int ncs, bool on) {
  float4 *f4 = reinterpret_cast<float4 *>(buf);
  const int cap = fold_slots(R) * ncs;
  float *cnt = reinterpret_cast<float *>(f4 + (V / 2) * cap);
  fold_rows(
      R, rl, cc, ncs, on,
      [&](int slot) {
        float2 mb[V / 2], qb[V / 2];
        get_pairs<V>(f4, cap, slot, mb, qb);
        st.merge(mb, qb, cnt[slot]);
      },
      [&](int slot) {
        put_pairs<V>(f4, cap, slot, st.m, st.q);
        cnt[slot] = st.n;
      });
}
template <int V>
__device__ __forceinline__ void fold_sums(float2 (&a)[V / 2], float2 (&b)[V / 2],
                                          unsigned char *buf, int R, int rl, int cc, int ncs,
                                          bool on) {
  float4 *f4 = reinterpret_cast<float4 *>(buf);
  const int cap = fold_slots(R) * ncs;
  fold_rows(
      R, rl, cc, ncs, on,
      [&](int slot) {
        float2 ao[V / 2], bo[V / 2];
        get_pairs<V>(f4, cap, slot, ao, bo);
#pragma unroll
        for (int p = 0; p < V / 2; ++p) {
          a[p] = add2(a[p], ao[p]);
          b[p] = add2(b[p], bo[p]);
        }
      },
      [&](int slot) { put_pairs<V>(f4, cap, slot, a, b); });
}

// Row statistics of a CTA's threads -> (mean, M2) of each channel of the slab
// over the CTA's rows (chm, chq; `nch` channels; f_rows divides by the rows).
// Called by all threads; the arrays are complete after the next barrier.
template <int V>
__device__ __forceinline__ void channel_stats(ChannelStats<V> &st, unsigned char *buf, float *chm,
                                              float *chq, int R, int rl, int cc, int ncs, bool on,
                                              int nch, const FloatDiv &f_rows) {
  if (R == 1) {
    if (on) {
#pragma unroll
      for (int p = 0; p < V / 2; ++p) {
        *reinterpret_cast<float2 *>(chm + cc * V + 2 * p) = st.m[p];
        *reinterpret_cast<float2 *>(chq + cc * V + 2 * p) = st.q[p];
      }
    }
    return;
  }
  fold_stats<V>(st, buf, R, rl, cc, ncs, on);
  const int cap = fold_slots(R) * ncs, rows = fold_lanes(R);
  const float *f = reinterpret_cast<const float *>(buf);
  const float *cnt = f + 2 * V * cap;
#pragma unroll 1
  for (int j = threadIdx.x; j < nch; j += blockDim.x) {
    const unsigned u = static_cast<unsigned>(j);
    const int col = static_cast<int>(u / V), v = static_cast<int>(u % V);
    const float *fm = f + pair_at<V>(cap, col, v, 0), *fq = f + pair_at<V>(cap, col, v, 1);
    // the mean first, then the deviations from it: no digit of the variance
    // is lost.  The quotient is the correctly rounded one, here and for the
    // groups: an error of a mean shifts all of its values one way.
    float n[kFoldLanes], m[kFoldLanes], mean = 0.f, q = 0.f;
#pragma unroll
    for (int r = 0; r < kFoldLanes; ++r) {
      const bool in = r < rows;
      n[r] = in ? cnt[r * ncs + col] : 0.f;
      m[r] = in ? fm[r * ncs * 4] : 0.f;
    }
#pragma unroll
    for (int r = 0; r < kFoldLanes; ++r)
      if (r < rows) mean = fmaf(n[r], m[r], mean);
    mean = f_rows(mean);
#pragma unroll
    for (int r = 0; r < kFoldLanes; ++r)
      if (r < rows) q += fmaf(n[r] * (m[r] - mean), m[r] - mean, fq[r * ncs * 4]);
    chm[j] = mean;
    chq[j] = q;
  }
}

// Sum of per-thread values over each channel j of the slab: s1 and s2 of the R
// row lanes, added up in a fixed order, times fa and fb(j).  Called by all
// threads; the arrays are complete after the next barrier.
template <int V, typename Factor>
__device__ __forceinline__ void channel_sums(float2 (&a)[V / 2], float2 (&b)[V / 2],
                                             unsigned char *buf, float *ca, float *cb, int R, int rl,
                                             int cc, int ncs, bool on, int nch, float fa,
                                             Factor fb) {
  if (R == 1) {
    if (on) {
#pragma unroll
      for (int p = 0; p < V / 2; ++p) {
        const int j = cc * V + 2 * p;
        *reinterpret_cast<float2 *>(ca + j) = mul2(a[p], splat2(fa));
        *reinterpret_cast<float2 *>(cb + j) = mul2(b[p], make_float2(fb(j), fb(j + 1)));
      }
    }
    return;
  }
  fold_sums<V>(a, b, buf, R, rl, cc, ncs, on);
  const int cap = fold_slots(R) * ncs, rows = fold_lanes(R);
  const float *at = reinterpret_cast<const float *>(buf);
#pragma unroll 1
  for (int j = threadIdx.x; j < nch; j += blockDim.x) {
    const unsigned u = static_cast<unsigned>(j);
    const int col = static_cast<int>(u / V), v = static_cast<int>(u % V);
    const float *pa = at + pair_at<V>(cap, col, v, 0), *pb = at + pair_at<V>(cap, col, v, 1);
    const float f = fb(j);
    float sa = pa[0], sb = pb[0];
#pragma unroll
    for (int r = 1; r < kFoldLanes; ++r)
      if (r < rows) {
        sa += pa[r * ncs * 4];
        sb += pb[r * ncs * 4];
      }
    ca[j] = sa * fa;
    cb[j] = sb * f;
  }
}

// rstd of a group: the quotient and the reciprocal root are correctly rounded (an
// rstd that is a step off scales a whole group).  An M2 that overflowed gives 0.
__device__ __forceinline__ float group_rstd(const GroupArgs &a, float m2) {
  return __frsqrt_rn(a.f_SD(m2) + a.eps);
}

// Sum over the 2^lsh lanes that share a group.
__device__ __forceinline__ float lanes_sum(float v, int lsh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < (1 << lsh)) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Runs fn(g, lane, valid) with 2^lsh lanes per group, as many groups at a
// time as the CTA has lanes for: all groups of a slab side by side, so that
// the latencies of their folds (shared memory, L2, shuffles) overlap.  Every
// lane of a warp takes part in every step.  (Loops with a stride known only
// at run time stay rolled here: unrolling them costs an integer division for
// the trip count, more than the few turns they take.)
template <typename Fn>
__device__ __forceinline__ void each_group(int ng, int lsh, Fn fn) {
  const int per = static_cast<int>(blockDim.x) >> lsh;
#pragma unroll 1
  for (int base = 0; base < ng; base += per) {
    const int g = base + (static_cast<int>(threadIdx.x) >> lsh);
    fn(g, static_cast<int>(threadIdx.x) & ((1 << lsh) - 1), g < ng);
  }
}

// (mean, M2) of every group from the (mean, M2) of its D channels over n rows
// each, handed to out(g, mean, M2) by one lane per group.
template <typename Out>
__device__ __forceinline__ void groups_of_channels(const GroupArgs &a, const float *chm,
                                                   const float *chq, int ng, float n, Out out) {
  const int D = a.D, lsh = a.lsh;
  each_group(ng, lsh, [&](int g, int l, bool in) {
    const float *m = chm + g * D, *q = chq + g * D;
    float s = 0.f, t = 0.f;
    if (in) {
#pragma unroll 1
      for (int j = l; j < D; j += 1 << lsh) s += m[j];
    }
    const float gm = a.f_D(lanes_sum(s, lsh));
    if (in) {
#pragma unroll 1
      for (int j = l; j < D; j += 1 << lsh) {
        const float e = m[j] - gm;
        t += fmaf(n * e, e, q[j]);
      }
    }
    t = lanes_sum(t, lsh);
    if (in && l == 0) out(g, gm, t);
  });
}

// Address of the V-element chunk column cc (within the tensor) of row s of
// sample b, in elements.
__device__ __forceinline__ int64_t group_elem(const GroupArgs &a, int b, int64_t s, int chunk,
                                              int V) {
  return (static_cast<int64_t>(b) * a.S + s) * a.C + static_cast<int64_t>(chunk) * V;
}

// S rows cut into ranges that differ by one row at most, the longer ones
// first.
struct Parts {
  const GroupArgs &a;
  int q, rem;
  __device__ __forceinline__ explicit Parts(const GroupArgs &args)
      : a(args), q(a.pq), rem(a.prem) {}
  __device__ __forceinline__ const FloatDiv &by_rows(int i) const {
    return i < rem ? a.f_rows1 : a.f_rows;
  }
  __device__ __forceinline__ int rows(int i) const { return q + (i < rem ? 1 : 0); }
  __device__ __forceinline__ int begin(int i) const { return i * q + (i < rem ? i : rem); }
};

// Parameters of a thread's V channels as fp32 pairs: gamma, beta (0 when
// absent).
struct AffineRaw {
  uint4 g, b;
};
__device__ __forceinline__ AffineRaw load_affine_raw(const GroupArgs &a, int chunk) {
  AffineRaw r;
  r.g = ld_global_nc_v4(static_cast<const uint4 *>(a.gamma) + chunk);
  r.b = make_uint4(0, 0, 0, 0);
  if (a.beta) r.b = ld_global_nc_v4(static_cast<const uint4 *>(a.beta) + chunk);
  return r;
}
template <int DT>
__device__ __forceinline__ void load_affine(const GroupArgs &a, int chunk,
                                            float2 (&gf)[chunk_elems(DT) / 2],
                                            float2 (&bf)[chunk_elems(DT) / 2]) {
  const AffineRaw r = load_affine_raw(a, chunk);
  unpack<DT>(r.g, gf);
  unpack<DT>(r.b, bf);
}

const void *group_ring_kernel_ptr(int dt, int act, bool drop, bool bwd);
const void *group_fwd_kernel_ptr(int dt, int act, bool drop);     // resident
const void *group_stats_kernel_ptr(int dt);                       // streamed, first pass
const void *group_apply_kernel_ptr(int dt, int act, bool drop);   // streamed, second pass
const void *group_bwd_kernel_ptr(int dt, int act, bool drop);     // resident
const void *group_sums_kernel_ptr(int dt, int act, bool drop);    // streamed, first pass
const void *group_dx_kernel_ptr(int dt, int act, bool drop);      // streamed, second pass

}  // namespace gbn
