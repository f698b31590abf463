// group_ring.cu -- group normalisation of large samples: one cooperative
// kernel, one CTA per SM, forward and backward.
//
// The samples are taken in rounds.  In a round every CTA owns one row range
// of one sample and walks it twice: a statistics pass (or, backward, the
// per-channel sums), a grid-wide barrier at which the CTAs of a sample see
// each other's partials, and an output pass.  A round holds as many samples
// as shared memory and L2 keep between the two passes (group.cu).
//
// Rows move as tiles (contiguous in memory) through a ring of shared-memory
// stages filled by bulk copies.  The first pass leaves the last `stages`
// tiles where they are and puts the up to four before those into tensor
// memory (each thread its own chunks, into columns of its own lane: 256 KB of
// an SM that this kernel has no other use for).  The output pass walks the
// tiles in the opposite order, so it starts with those, and as each stage is
// consumed it takes the tile that the first pass read latest among those
// dropped: the second read goes from the newest to the oldest line of L2.
// Once a round has no tile left to read again, freed stages take the next
// round's first tiles.
//
// What that does to the ring: a stage is always filled in the order in which
// stages are freed, so the walk through the stages turns round at the end of
// the first pass (where it stays on the last tile) and goes on in the new
// direction through the output pass and the next round's first pass.
//
// The bound is HBM: x (and dy) read once, y (dx) written once, plus whatever
// of the second read neither shared memory (29 MB over the GPU), nor tensor
// memory (39 MB), nor L2 still holds; and around it the cooperative launch
// (4 to 5 us) and the bubble at the grid barrier (folds, barrier, constants:
// about 6 us a round).  262144 x 256 fp16: 60 us, with SiLU 66 (268 MB, 60 % of
// the measured copy bandwidth).  The backward pass adds the instructions (see
// group_bwd.cu): 4 x 16384 x 512 bf16 51 us without activation, with SiLU 64 to
// 66 (201 MB, 45 %).
#include <cooperative_groups.h>

#include "common.cuh"
#include "group_rows.cuh"
#include "tcgen05.cuh"

namespace gbn {

namespace {

// One CTA's view of the ring: rows [row0, row0 + nrow) of one sample (in
// rounds: of sample b, b + nsamp, ...), chunk columns [chunk0, chunk0 + ncs).
//
// Every warp waits for a stage's copies on its `full` mbarrier and, where the
// stage is to be filled again, arrives on its `free` one when it has read it.
// Warp 0 fills a freed stage one item later (the others have then mostly
// finished with it), so no warp waits for another on the way through a pass.
template <int DT, int NT>
struct Ring {
  const GroupArgs &a;
  unsigned char *base;
  uint64_t *full, *empty;
  volatile int *abort_flag;
  GroupRingLayout L;
  int row0, nrow, TR, T, chunk0, ncs;
  int cur, dir;
  int tm;              // tiles of this CTA that stay in tensor memory
  uint32_t tq;         // this warp's columns there
  uint32_t par, epar;  // bit s: parity of stage s's next full / free phase
  int pstage, pb, ptile;  // the refill that warp 0 still owes (pstage < 0: none)
  bool pkeep;

  __device__ __forceinline__ Ring(const GroupArgs &args, unsigned char *smem, int split, int slab)
      : a(args), base(smem), cur(0), dir(1), par(0), epar(0), pstage(-1), pb(0), ptile(0),
        pkeep(false) {
    L = group_ring_layout(a.stages, a.U, a.R, a.ncs, chunk_elems(DT), a.sg, NT == 2);
    full = reinterpret_cast<uint64_t *>(smem + L.bar_off);
    empty = full + a.stages;
    abort_flag = reinterpret_cast<volatile int *>(smem + L.flag_off);
    const Parts parts(a);
    row0 = parts.begin(split);
    nrow = parts.rows(split);
    TR = a.U * a.R;
    T = (nrow + TR - 1) / TR;
    chunk0 = slab * a.ncs;
    ncs = min(a.ncs, a.nc - chunk0);
    tm = max(0, min(a.tm, T - a.stages));
    if (threadIdx.x == 0) {
      for (int s = 0; s < a.stages; ++s) {
        mbar_init(full + s, 1);
        mbar_init(empty + s, blockDim.x >> 5);
      }
      *abort_flag = 0;
      fence_mbar_init();
    }
    uint32_t *slot = reinterpret_cast<uint32_t *>(smem + L.flag_off) + 1;
    const int warp = threadIdx.x >> 5;
    if (a.tm && warp == 0) {
      tmem_alloc(slot, 512);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // warp w reaches lanes 32 (w % 4) ..; the four warps that share them take
    // 128 columns each
    tq = a.tm ? *slot + (static_cast<uint32_t>((warp & 3) * 32) << 16) +
                    static_cast<uint32_t>((warp >> 2) * 128)
              : 0u;
  }
  // Frees the tensor memory; every thread has read what it put there.
  __device__ __forceinline__ void finish() {
    tc_fence_before();
    __syncthreads();
    if (a.tm && threadIdx.x < 32) {
      tc_fence_after();
      tmem_dealloc(*(reinterpret_cast<uint32_t *>(base + L.flag_off) + 1), 512);
    }
  }

  // Half h of this thread's chunks of a tile: four rows of x (forward), or
  // all four of x (h = 0) or dy (h = 1).  `i`: the thread's chunk in row lane
  // 0 (negative: it owns none).
  __device__ __forceinline__ const uint4 *half(int h, int i) const {
    return stage(NT == 2 ? h : 0) + i + (NT == 2 ? 0 : 4 * h) * a.R * a.ncs;
  }
  // Puts the current stage's tile into tensor memory as tile m (whole warps).
  __device__ __forceinline__ void stash(int m, int i) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t r[16];
      const uint4 *t = half(h, i);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint4 v = i >= 0 ? t[u * a.R * a.ncs] : make_uint4(0, 0, 0, 0);
        r[4 * u] = v.x;
        r[4 * u + 1] = v.y;
        r[4 * u + 2] = v.z;
        r[4 * u + 3] = v.w;
      }
      __syncwarp();
      tmem_st_n<16>(tq + m * 32 + h * 16, r);
    }
  }
  // Takes two neighbouring chunks, c and c + 1 of half h, of tile m back
  // (whole warps).
  __device__ __forceinline__ void unstash(int m, int h, int c, uint4 &v, uint4 &w) const {
    uint32_t r[8];
    __syncwarp();
    tmem_ld_n<8>(tq + m * 32 + h * 16 + c * 4, r);
    tmem_wait_ld_n<8>(r);
    v = make_uint4(r[0], r[1], r[2], r[3]);
    w = make_uint4(r[4], r[5], r[6], r[7]);
  }

  __device__ __forceinline__ int rows_of(int tile) const { return min(TR, nrow - tile * TR); }

  // First-pass lines that the output pass reads again out of L2: the tiles
  // read last before those that stay in shared memory.
  __device__ __forceinline__ bool kept(int tile) const {
    return tile < T - a.stages - tm && tile >= T - a.stages - tm - a.keep;
  }

  // Fills stage s with tile `tile` of sample b (all lanes of one warp).
  __device__ __forceinline__ void issue(int b, int tile, int s, bool keep) {
    const int lane = threadIdx.x & 31;
    const int rows = rows_of(tile);
    const int64_t c = (static_cast<int64_t>(b) * a.S + row0 + static_cast<int64_t>(tile) * TR) *
                          a.nc + chunk0;
    const uint4 *srcs[2] = {static_cast<const uint4 *>(a.x) + c,
                            static_cast<const uint4 *>(a.dy) + c};
    unsigned char *dst = base + static_cast<size_t>(s) * L.stage_bytes;
    const uint32_t rb = static_cast<uint32_t>(ncs) * 16u;
    const uint64_t pol = keep ? l2_evict_last_policy() : l2_evict_first_policy();
    if (lane == 0) mbar_arrive_expect_tx(full + s, NT * rb * rows);
    __syncwarp();
    if (ncs == a.nc) {
      if (lane < NT) bulk_g2s(dst + lane * L.tensor_bytes, srcs[lane], rb * rows, full + s, pol);
    } else {
      // stage rows are a.ncs chunks apart, whatever this slab's width
      for (int r = lane; r < rows; r += 32)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          bulk_g2s(dst + t * L.tensor_bytes + static_cast<size_t>(r) * a.ncs * 16,
                   srcs[t] + static_cast<int64_t>(r) * a.nc, rb, full + s, pol);
    }
  }
  // The first tiles of sample b, by warp 0.
  __device__ __forceinline__ void start(int b) {
    if (threadIdx.x < 32)
      for (int j = 0; j < min(a.stages, T); ++j) issue(b, j, j, kept(j));
  }

  // Warp 0 fills the stage that was freed one item ago.
  __device__ __forceinline__ void flush() {
    if (threadIdx.x < 32 && pstage >= 0) {
      mbar_wait(empty + pstage, (epar >> pstage) & 1u, a.err, abort_flag);
      epar ^= 1u << pstage;
      fence_proxy_async_smem();
      __syncwarp();
      issue(pb, ptile, pstage, pkeep);
      pstage = -1;
    }
  }
  __device__ __forceinline__ void wait() {
    mbar_wait(full + cur, (par >> cur) & 1u, a.err, abort_flag);
    par ^= 1u << cur;
  }
  __device__ __forceinline__ void step() {
    cur += dir;
    if (cur == a.stages) cur = 0;
    if (cur < 0) cur = a.stages - 1;
  }
  // This warp has read the current stage, which takes `tile` of b next.
  __device__ __forceinline__ void refill(int b, int tile, bool keep) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(empty + cur);
    pstage = cur;
    pb = b;
    ptile = tile;
    pkeep = keep;
  }
  __device__ __forceinline__ uint4 *stage(int tensor) const {
    return reinterpret_cast<uint4 *>(base + static_cast<size_t>(cur) * L.stage_bytes +
                                           tensor * L.tensor_bytes);
  }

  // First pass over sample b: body(tile, its rows).  `i`: see half().
  template <typename Body>
  __device__ __forceinline__ void first_pass(int b, int i, Body body) {
#pragma unroll 1
    for (int j = 0; j < T; ++j) {
      flush();
      wait();
      body(j, rows_of(j));
      const int m = j - (T - a.stages - tm);
      if (m >= 0 && m < tm) stash(m, i);
      if (j + a.stages < T) refill(b, j + a.stages, kept(j + a.stages));
      if (j + 1 < T) step();
    }
    dir = -dir;
  }
  // Output pass over sample b, last tile first: body(tile, its rows) on the
  // current stage, far(m, tile, its rows) for the tiles in tensor memory.
  // `next`: the sample of this CTA's next round, or -1.
  template <typename Body, typename Far>
  __device__ __forceinline__ void output_pass(int b, int next, Body body, Far far) {
    const int n = T - tm;  // tiles of this pass that come by way of a stage
    auto far_tiles = [&]() {
#pragma unroll 1
      for (int m = tm - 1; m >= 0; --m) {
        const int tile = T - a.stages - tm + m;
        far(m, tile, rows_of(tile));
      }
    };
    if (tm) {
      __syncwarp();
      tmem_wait_st();
    }
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      flush();
      if (i == a.stages) far_tiles();
      if (i >= a.stages) wait();
      const int tile = T - 1 - i - (i < a.stages ? 0 : tm);
      body(tile, rows_of(tile));
      // the freed stage takes this pass's tile i + stages, or else the next
      // round's first ones
      const int k = i + a.stages;
      if (k < n) refill(b, T - 1 - tm - k, false);
      else if (next >= 0 && k - n < T) refill(next, k - n, kept(k - n));
      step();
    }
    if (n <= a.stages) far_tiles();
  }
};

// Roles of a CTA: sample within the round, slab, row range.
struct Role {
  int sj, slab, sp;
  __device__ __forceinline__ explicit Role(const GroupArgs &a) {
    const int u = static_cast<int>(blockIdx.x);
    const int v = a.by_splits(u);
    sp = u - v * a.splits;
    sj = a.by_nslab(v);
    slab = v - sj * a.nslab;
  }
};

template <int DT, int ACT, bool DROP>
__global__ void __launch_bounds__(kGroupThreads, 1) group_ring_fwd_kernel(const GroupArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int V = chunk_elems(DT);
  constexpr int U = kRingRowsFwd;
  static_assert(U == 8, "a thread's part of a tile is two halves of four rows");
  const Role role(a);
  Ring<DT, 1> ring(a, smem, role.sp, role.slab);
  const int tid = threadIdx.x;
  const int rl = a.by_ncs(tid);
  const int cc = tid - rl * a.ncs;
  const bool on = rl < a.R && cc < ring.ncs;
  const int own = on ? rl * a.ncs + cc : -1;  // this thread's chunk in a tile
  const int g0 = role.slab * a.sg;
  const int ng = min(a.sg, a.G - g0);
  unsigned char *fold = smem + ring.L.fold_off;
  float *chm = reinterpret_cast<float *>(smem + ring.L.chan_off);
  float *chq = chm + a.ncs * V;
  float2 *gfin = reinterpret_cast<float2 *>(smem + ring.L.gst_off);
  float2 *gpart = reinterpret_cast<float2 *>(a.gpart);
  const int pstride = (a.splits + 1) & ~1;  // (rows of partials start on 16 bytes)
  const Parts parts(a);
  const float fD = static_cast<float>(a.D);
  DropGen gen(a.drop);
  if (DROP) gen.start();
  auto grid = cooperative_groups::this_grid();

  if (role.sj < a.B) ring.start(role.sj);

  for (int round = 0; round < a.rounds; ++round) {
    const int b = round * a.nsamp + role.sj;
    const int next = (round + 1 < a.rounds && b + a.nsamp < a.B) ? b + a.nsamp : -1;
    if (b < a.B) {
      ChannelStats<V> st;
      st.clear();
      ring.first_pass(b, own, [&](int, int rows) {
        if (!on) return;
        const uint4 *t = ring.stage(0) + own;
        const int step = a.R * a.ncs;
        if (rl + (U - 1) * a.R < rows) {
#pragma unroll
          for (int h = 0; h < U; h += 4) {
            float2 f[4][V / 2];
#pragma unroll
            for (int u = 0; u < 4; ++u) unpack<DT>(t[(h + u) * step], f[u]);
            st.add4(f[0], f[1], f[2], f[3]);
          }
        } else {
          for (int u = 0; rl + u * a.R < rows; ++u) {
            float2 f[V / 2];
            unpack<DT>(t[u * step], f);
            st.add1(f);
          }
        }
      });
      channel_stats<V>(st, fold, chm, chq, a.R, rl, cc, a.ncs, on, ring.ncs * V,
                       parts.by_rows(role.sp));
      __syncthreads();
      // partials laid out [b][group][split]: the fold below reads a group's
      // splits side by side
      groups_of_channels(a, chm, chq, ng, static_cast<float>(ring.nrow),
                         [&](int g, float m, float m2) {
                           gpart[(static_cast<int64_t>(b) * a.G + g0 + g) * pstride + role.sp] =
                               make_float2(m, m2);
                         });
    }
    grid.sync();
    if (b < a.B) {
      each_group(ng, a.lsh, [&](int g, int l, bool in) {
        const float2 *part = gpart + (static_cast<int64_t>(b) * a.G + g0 + g) * pstride;
        // two splits per load; the mean first, then the deviations from it,
        // a lane's first kNear pairs staying in registers in between
        constexpr int kNear = 6;
        float4 v[kNear];
        float m = 0.f, m2 = 0.f;
#pragma unroll
        for (int i = 0; i < kNear; ++i) {
          const int r = 2 * (l + (i << a.lsh));
          v[i] = in && r < a.splits ? __ldcg(reinterpret_cast<const float4 *>(part + r))
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        auto mean_of = [&](int r, float4 u) {
          m = fmaf(static_cast<float>(parts.rows(r)), u.x, m);
          if (r + 1 < a.splits) m = fmaf(static_cast<float>(parts.rows(r + 1)), u.z, m);
        };
        auto deviation = [&](int r, float4 u) {
          const float e = u.x - m;
          m2 += fmaf(static_cast<float>(parts.rows(r)) * fD * e, e, u.y);
          if (r + 1 < a.splits) {
            const float f = u.z - m;
            m2 += fmaf(static_cast<float>(parts.rows(r + 1)) * fD * f, f, u.w);
          }
        };
#pragma unroll
        for (int i = 0; i < kNear; ++i) {
          const int r = 2 * (l + (i << a.lsh));
          if (r < a.splits) mean_of(r, v[i]);
        }
        const int far = in ? 2 * (l + (kNear << a.lsh)) : a.splits;
#pragma unroll 1
        for (int r = far; r < a.splits; r += 2 << a.lsh)
          mean_of(r, __ldcg(reinterpret_cast<const float4 *>(part + r)));
        m = a.f_S(lanes_sum(m, a.lsh));
#pragma unroll
        for (int i = 0; i < kNear; ++i) {
          const int r = 2 * (l + (i << a.lsh));
          if (r < a.splits) deviation(r, v[i]);
        }
#pragma unroll 1
        for (int r = far; r < a.splits; r += 2 << a.lsh)
          deviation(r, __ldcg(reinterpret_cast<const float4 *>(part + r)));
        m2 = lanes_sum(m2, a.lsh);
        if (in && l == 0) {
          const float rs = group_rstd(a, m2);
          gfin[g] = make_float2(m, rs);
          if (role.sp == 0) {
            a.mean[static_cast<int64_t>(b) * a.G + g0 + g] = m;
            a.rstd[static_cast<int64_t>(b) * a.G + g0 + g] = rs;
          }
        }
      });
      __syncthreads();
      float2 nmu[V / 2], sc[V / 2], bf[V / 2];
      if (on) {
        const int chunk = ring.chunk0 + cc;
        out_constants<DT>(a, load_affine_raw(a, chunk), gfin, g0, chunk, nmu, sc, bf);
      }
      const int64_t e0 = group_elem(a, b, ring.row0 + rl, ring.chunk0 + cc, V);
      const int64_t estep = static_cast<int64_t>(a.R) * a.C;
      unsigned char *out = static_cast<unsigned char *>(a.out);
      // rows u and u + 1 of this thread in a tile of `rows` rows
      auto emit = [&](int64_t e, int u, int rows, uint4 va, uint4 vb) {
        if (rl + u * a.R >= rows) return;
        const bool two = rl + (u + 1) * a.R < rows;
        if (!two) vb = va;
        out_rows<DT, ACT, DROP>(va, vb, nmu, sc, bf, gen, e, e + estep);
        st_global_cs_v4(out + e * elem_bytes(DT), va);
        if (two) st_global_cs_v4(out + (e + estep) * elem_bytes(DT), vb);
      };
      ring.output_pass(
          b, next,
          [&](int tile, int rows) {
            if (!on) return;
            const uint4 *t = ring.stage(0) + own;
            const int step = a.R * a.ncs;
            int64_t e = e0 + static_cast<int64_t>(tile) * ring.TR * a.C;
#pragma unroll
            for (int u = 0; u < U; u += 2) {
              emit(e, u, rows, t[u * step], t[(u + 1) * step]);
              e += 2 * estep;
            }
          },
          [&](int m, int tile, int rows) {
            int64_t e = e0 + static_cast<int64_t>(tile) * ring.TR * a.C;
#pragma unroll 1
            for (int u = 0; u < U; u += 2) {
              uint4 va, vb;
              ring.unstash(m, u >> 2, u & 3, va, vb);
              if (on) emit(e, u, rows, va, vb);
              e += 2 * estep;
            }
          });
    }
  }
  ring.finish();
}

template <int DT, int ACT, bool DROP>
__global__ void __launch_bounds__(kGroupThreads, 1) group_ring_bwd_kernel(const GroupArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int V = chunk_elems(DT);
  constexpr int U = kRingRowsBwd;
  static_assert(U == 4, "a thread's part of a tile is four rows of x and of dy");
  const Role role(a);
  Ring<DT, 2> ring(a, smem, role.sp, role.slab);
  const int tid = threadIdx.x;
  const int lane = tid & 31;
  const int rl = a.by_ncs(tid);
  const int cc = tid - rl * a.ncs;
  const bool on = rl < a.R && cc < ring.ncs;
  const int own = on ? rl * a.ncs + cc : -1;  // this thread's chunk in a tile
  const int g0 = role.slab * a.sg;
  const int ng = min(a.sg, a.G - g0);
  const int ch0 = ring.chunk0 * V;
  unsigned char *fold = smem + ring.L.fold_off;
  float *cb = reinterpret_cast<float *>(smem + ring.L.chan_off);  // sum dz per channel
  float *cg = cb + a.ncs * V;                                     // sum dz xhat per channel
  float *tb = reinterpret_cast<float *>(smem + ring.L.tot_off);  // their totals over rounds
  float *tg = tb + a.ncs * V;
  float2 *gfin = reinterpret_cast<float2 *>(smem + ring.L.gst_off);
  float2 *gpart = reinterpret_cast<float2 *>(a.gpart);
  const int pstride = (a.splits + 1) & ~1;  // (rows of partials start on 16 bytes)
  DropGen gen(a.drop);
  if (DROP) gen.start();
  auto grid = cooperative_groups::this_grid();

  if (role.sj < a.B) ring.start(role.sj);

  for (int round = 0; round < a.rounds; ++round) {
    const int b = round * a.nsamp + role.sj;
    const int next = (round + 1 < a.rounds && b + a.nsamp < a.B) ? b + a.nsamp : -1;
    const int64_t estep = static_cast<int64_t>(a.R) * a.C;
    int64_t e0 = 0;
    BwdConst<V> k;
    if (b < a.B) {
      e0 = group_elem(a, b, ring.row0 + rl, ring.chunk0 + cc, V);
      if (on) load_const<DT>(a, b, ring.chunk0 + cc, k);
      float2 s1[V / 2], s2[V / 2];
#pragma unroll
      for (int p = 0; p < V / 2; ++p) s1[p] = s2[p] = splat2(0.f);
      ring.first_pass(b, own, [&](int tile, int rows) {
        if (!on) return;
        const int step = a.R * a.ncs;
        const uint4 *tx = ring.stage(0) + own;
        uint4 *td = ring.stage(1) + own;
        int64_t e = e0 + static_cast<int64_t>(tile) * ring.TR * a.C;
        // dropped elements of dy are zeroed; in a tile that stays on the SM,
        // in the stage too, so that the dx pass need not ask the generator
        // again
        const bool stays = tile >= ring.T - a.stages - ring.tm;
#pragma unroll
        for (int u = 0; u < U; u += 2) {
          if (rl + u * a.R < rows) {
            const bool two = rl + (u + 1) * a.R < rows;
            const int o = (u + (two ? 1 : 0)) * step;
            uint4 da = td[u * step], db = td[o];
            if (DROP) {
              gen.template mask<DT>(da, static_cast<uint64_t>(e));
              gen.template mask<DT>(db, static_cast<uint64_t>(e + estep));
              if (stays) {
                td[u * step] = da;
                if (two) td[o] = db;
              }
            }
            sum_rows<DT, ACT>(tx[u * step], da, tx[o], db, two, k, s1, s2);
          }
          e += 2 * estep;
        }
      });
      channel_sums<V>(s1, s2, fold, cb, cg, a.R, rl, cc, a.ncs, on, ring.ncs * V,
                      sum_factor<DROP>(a),
                      [&](int j) { return xhat_factor<DROP>(a, b, ch0 + j); });
      __syncthreads();
      group_sums<DT>(a, cb, cg, ch0, ng, [&](int g, float2 v) {
        gpart[(static_cast<int64_t>(b) * a.G + g0 + g) * pstride + role.sp] = v;
      });
      // running dgamma / dbeta of this CTA's rows over the rounds; after the
      // last one they are its partial row
      float *rg = a.cpart + static_cast<int64_t>(role.sj * a.splits + role.sp) * a.C + ch0;
      float *rb = a.dbeta_part
                      ? a.dbeta_part + static_cast<int64_t>(role.sj * a.splits + role.sp) * a.C + ch0
                      : nullptr;
#pragma unroll 1
      for (int j = tid; j < ring.ncs * V; j += blockDim.x) {
        float vg = cg[j], vb = cb[j];
        if (round > 0) {
          vg += tg[j];
          vb += tb[j];
        }
        if (next < 0) {
          rg[j] = vg;
          if (rb) rb[j] = vb;
        } else {
          tg[j] = vg;
          tb[j] = vb;
        }
      }
    }
    grid.sync();
    if (b < a.B) {
      each_group(ng, a.lsh, [&](int g, int l, bool in) {
        const float2 *part = gpart + (static_cast<int64_t>(b) * a.G + g0 + g) * pstride;
        float2 t = splat2(0.f);
        if (in) {
#pragma unroll 4
          for (int r = 2 * l; r < a.splits; r += 2 << a.lsh) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(part + r));
            t = add2(t, make_float2(v.x, v.y));
            if (r + 1 < a.splits) t = add2(t, make_float2(v.z, v.w));
          }
        }
        t.x = lanes_sum(t.x, a.lsh);
        t.y = lanes_sum(t.y, a.lsh);
        if (in && l == 0) {
          const float rs = __ldg(a.rstd + static_cast<int64_t>(b) * a.G + g0 + g);
          gfin[g] = make_float2(-rs * a.f_SD(t.x), -rs * rs * a.f_SD(t.y));
        }
      });
      __syncthreads();
      float2 ra[V / 2], rc[V / 2];
      if (on) dx_constants<DT>(a, gfin, g0, ring.chunk0 + cc, ra, rc);
      unsigned char *out = static_cast<unsigned char *>(a.out);
      // rows u and u + 1 of this thread in a tile of `rows` rows; `ask`: the
      // dropped elements of dy are not zeroed yet
      auto emit = [&](int64_t e, int u, int rows, bool ask, uint4 xa, uint4 da, uint4 xb,
                      uint4 db) {
        if (rl + u * a.R >= rows) return;
        const bool two = rl + (u + 1) * a.R < rows;
        if (DROP && ask) {
          gen.template mask<DT>(da, static_cast<uint64_t>(e));
          gen.template mask<DT>(db, static_cast<uint64_t>(e + estep));
        }
        if (!two) {
          xb = xa;
          db = da;
        }
        dx_rows<DT, ACT, DROP>(a, xa, da, xb, db, k, ra, rc);
        st_global_cs_v4(out + e * elem_bytes(DT), xa);
        if (two) st_global_cs_v4(out + (e + estep) * elem_bytes(DT), xb);
      };
      ring.output_pass(
          b, next,
          [&](int tile, int rows) {
            if (!on) return;
            const int step = a.R * a.ncs;
            const uint4 *tx = ring.stage(0) + own;
            const uint4 *td = ring.stage(1) + own;
            int64_t e = e0 + static_cast<int64_t>(tile) * ring.TR * a.C;
            const bool ask = tile < ring.T - a.stages;
#pragma unroll
            for (int u = 0; u < U; u += 2) {
              emit(e, u, rows, ask, tx[u * step], td[u * step], tx[(u + 1) * step],
                   td[(u + 1) * step]);
              e += 2 * estep;
            }
          },
          [&](int m, int tile, int rows) {
            int64_t e = e0 + static_cast<int64_t>(tile) * ring.TR * a.C;
#pragma unroll 1
            for (int u = 0; u < U; u += 2) {
              uint4 xa, xb, da, db;
              ring.unstash(m, 0, u, xa, xb);
              ring.unstash(m, 1, u, da, db);
              if (on) emit(e, u, rows, false, xa, da, xb, db);
              e += 2 * estep;
            }
          });
    }
  }

  ring.finish();

  // dgamma / dbeta: column sums of the partial rows, which every CTA wrote
  // before the last barrier (samples of earlier rounds only, where the last
  // round has none for it).  A CTA takes 32 columns at a time, its warps
  // every 16th row; the warps' sums are added in warp order.
  const int P = min(a.nsamp, a.B) * a.splits;
  const int cols = (a.C + 31) / 32;
  float *part = reinterpret_cast<float *>(fold);  // [16][32]
  for (int t = blockIdx.x; t < cols * (a.dbeta ? 2 : 1); t += gridDim.x) {
    const bool beta = t >= cols;
    const int c = (beta ? t - cols : t) * 32 + lane;
    const float *rows = beta ? a.dbeta_part : a.cpart;
    float acc = 0.f;
    if (c < a.C) {
#pragma unroll 4
      for (int r = tid >> 5; r < P; r += (static_cast<int>(blockDim.x) >> 5))
        acc += __ldcg(rows + static_cast<int64_t>(r) * a.C + c);
    }
    part[tid] = acc;
    __syncthreads();
    if (tid < 32 && c < a.C) {
      for (int w = 1; w < (static_cast<int>(blockDim.x) >> 5); ++w) acc += part[w * 32 + lane];
      (beta ? a.dbeta : a.dgamma)[c] = acc;
    }
    __syncthreads();
  }
}

template <int DT, int ACT, bool DROP>
const void *pick_dir(bool bwd) {
  return bwd ? reinterpret_cast<const void *>(&group_ring_bwd_kernel<DT, ACT, DROP>)
             : reinterpret_cast<const void *>(&group_ring_fwd_kernel<DT, ACT, DROP>);
}

template <int DT>
const void *pick_act(int act, bool drop, bool bwd) {
  switch (act) {
    case kActSilu: return drop ? pick_dir<DT, kActSilu, true>(bwd) : pick_dir<DT, kActSilu, false>(bwd);
    case kActGelu: return drop ? pick_dir<DT, kActGelu, true>(bwd) : pick_dir<DT, kActGelu, false>(bwd);
    default: return drop ? pick_dir<DT, kActNone, true>(bwd) : pick_dir<DT, kActNone, false>(bwd);
  }
}

}  // namespace

const void *group_ring_kernel_ptr(int dt, int act, bool drop, bool bwd) {
  switch (dt) {
    case kBF16: return pick_act<kBF16>(act, drop, bwd);
    case kFP16: return pick_act<kFP16>(act, drop, bwd);
    default: return pick_act<kFP32>(act, drop, bwd);
  }
}

}  // namespace gbn
