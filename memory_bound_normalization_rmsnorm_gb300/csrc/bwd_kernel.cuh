// bwd_kernel.cuh -- the backward RMSNorm / LayerNorm kernel template (one
// fused row pass: dx, and per-CTA partial column sums for dgamma and dbeta),
// included by the translation units that instantiate it: bwd.cu (plain and
// fused residual add) and drop_add.cu (dropout + residual add).  The
// rationale and the page paragraphs it follows are in bwd.cu.
#pragma once

#include "common.cuh"
#include "dropout.cuh"
#include "ptx.cuh"
#include "rowops.cuh"
#include "tiles.cuh"

namespace gbn {

// EXACT: every CTA's slice is exactly K * tpr chunks and tpr >= 32, so no
// chunk needs an ownership test and the warp butterfly is full width.
// RESID: fused residual add -- x is h, and the stage also holds dh, added to
// dx (in fp32, before rounding): dx = norm backward + dh.
// DROP: (with RESID) that sum is dr, the gradient of the residual stream, and
// dx = drop(dr) that of the branch that the forward dropped out.
template <int MODE, int K, bool CLUSTER, bool EXACT, bool RESID, bool DROP = false>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_bwd_kernel(const NormArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  const SmemLayout L = make_layout(a.RT, a.NS, a.S, a.G, a.tpr, RESID ? 3 : 2, true, a.C);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L.bar_off);
  float *red = reinterpret_cast<float *>(smem + L.red_off);
  const float *stats_all = reinterpret_cast<const float *>(smem + L.stats_off);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L.flag_off);
  int *done_cnt = reinterpret_cast<int *>(smem + L.flag_off) + 1;

  const int tid = threadIdx.x;
  const int g = tid / a.tpr;
  const int t = tid - g * a.tpr;
  const int nwarps = blockDim.x >> 5;
  const int crank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t cid = CLUSTER ? static_cast<int64_t>(cluster_id_x()) : blockIdx.x;
  const int64_t ncl = CLUSTER ? static_cast<int64_t>(ncluster_x()) : gridDim.x;
  const int col0 = crank * a.NS;
  // Chunks this CTA owns (the last CTA of a cluster may own fewer).
  const int nsc_me = min(a.nsc, a.N / 8 - crank * a.nsc);

  if (tid == 0) {
    for (int s = 0; s < a.S; ++s) {
      mbar_init(full + s, 1);
      done_cnt[s] = 0;
    }
    if (CLUSTER) {
      uint64_t *xb = xch_bars(smem, L, a.RT, a.C);
      for (int b = 0; b < kXchBuffers; ++b) mbar_init(xb + b, 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  // Programmatic dependent launch: let the next kernel in the stream start
  // its prologue as our CTAs retire, and touch no global memory before the
  // previous kernel's writes are complete and visible.
  grid_launch_dependents();
  grid_dependency_wait();

  // The first S tiles are requested before anything else, so that their
  // DRAM round trip overlaps the parameter loads below (warp 0, whose lane 0
  // initialised the barriers, issues them after a warp sync).
  const uint64_t pol = l2_evict_first_policy();
  if (tid < 32) {
    __syncwarp();
    for (int j = 0; j < a.S; ++j) {
      const int64_t tile = cid + j * ncl;
      if (tile < a.ntiles) issue_bwd_tile<MODE, CLUSTER, RESID>(a, L, smem, tile, j, col0, nsc_me, pol);
    }
  }

  // gamma (fp32 pairs) and the column accumulators of this thread's chunks
  // live in registers for the whole kernel.
  float2 gf[K][4], accg[K][4], accb[K][4];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = t + k * a.tpr;
    const uint4 gv = (c < nsc_me) ? ld_global_nc_v4(a.gamma + col0 + c * 8) : make_uint4(0, 0, 0, 0);
    chunk_to_f2(gv, gf[k]);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      accg[k][p] = splat2(0.f);
      accb[k][p] = splat2(0.f);
    }
  }

  if (CLUSTER) cluster_sync(); else __syncthreads();

  DropGen gen(a.drop);
  if (DROP) gen.start();
  const float invN = a.invN;
  int rpar = 0;
  ClusterXch xch = make_xch(smem, L, a.RT, CLUSTER ? a.C : 1, crank);
  // Stage s and its phase parity advance with the tile count (no division).
  int s = 0;
  uint32_t par = 0;
  for (int64_t tile = cid; tile < a.ntiles; tile += ncl) {
    mbar_wait(full + s, par, a.err, abort_flag);
    const int64_t row0 = tile * a.RT;
    const int nrows = static_cast<int>(min64(a.RT, a.M - row0));
    const unsigned char *stx = smem + static_cast<size_t>(s) * L.stage_bytes;
    const float *stats = stats_all + static_cast<size_t>(s) * a.RT * 2;

    for (int q = 0; q < a.rpg; ++q) {
      const int r = g + q * a.G;
      const bool active = r < nrows;
      float rs = 0.f, mu = 0.f;
      if (active) {
        rs = stats[2 * r];
        if (MODE == kLayer) mu = stats[2 * r + 1];
      }
      const float2 rs2 = splat2(rs);
      const float2 nmu = splat2(-mu);
      const unsigned char *xrow = stx + static_cast<size_t>(r) * a.NS * 2 + t * 16;
      // xhat and g = dy * gamma stay in registers between the two passes.
      float2 xh[K][4], gg[K][4];
      float2 s1 = splat2(0.f), s2 = splat2(0.f), s1b = splat2(0.f), s2b = splat2(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const bool ok = active && (EXACT || t + k * a.tpr < nsc_me);
        uint4 xv = make_uint4(0, 0, 0, 0), dv = make_uint4(0, 0, 0, 0);
        if (ok) {
          xv = *reinterpret_cast<const uint4 *>(xrow + k * a.tpr * 16);
          dv = *reinterpret_cast<const uint4 *>(xrow + L.tensor_bytes + k * a.tpr * 16);
        }
        float2 xf[4], df[4];
        chunk_to_f2(xv, xf);
        chunk_to_f2(dv, df);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          xh[k][p] = mul2(MODE == kLayer ? add2(xf[p], nmu) : xf[p], rs2);
          gg[k][p] = mul2(df[p], gf[k][p]);
          // two independent accumulator pairs shorten the dependency chains
          if (p & 1) {
            s2b = fma2(gg[k][p], xh[k][p], s2b);
            if (MODE == kLayer) s1b = add2(s1b, gg[k][p]);
          } else {
            s2 = fma2(gg[k][p], xh[k][p], s2);
            if (MODE == kLayer) s1 = add2(s1, gg[k][p]);
          }
          accg[k][p] = fma2(df[p], xh[k][p], accg[k][p]);
          if (MODE == kLayer) accb[k][p] = add2(accb[k][p], df[p]);
        }
      }
      s1 = add2(s1, s1b);
      s2 = add2(s2, s2b);
      float v[2] = {s1.x + s1.y, s2.x + s2.y};
      if (MODE == kLayer) {
        group_sum<2, EXACT>(v, a.tpr, g, a.G, t, red, rpar);
        if (CLUSTER) cluster_sum<2>(v, r, t, xch, a.err, abort_flag);
      } else {
        float w1[1] = {v[1]};
        group_sum<1, EXACT>(w1, a.tpr, g, a.G, t, red, rpar);
        if (CLUSTER) cluster_sum<1>(w1, r, t, xch, a.err, abort_flag);
        v[1] = w1[0];
      }
      // dx = rstd (g - a - xhat c) = rstd g - rstd a - (rstd c) xhat
      const float2 nra = splat2((MODE == kLayer) ? -rs * (v[0] * invN) : 0.f);
      const float2 nrc = splat2(-rs * (v[1] * invN));

      if (active) {
        uint16_t *dxrow = a.out + (row0 + r) * a.N + col0 + t * 8;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (EXACT || t + k * a.tpr < nsc_me) {
            float2 o[4];
#pragma unroll
            for (int p = 0; p < 4; ++p)
              o[p] = fma2(xh[k][p], nrc,
                          MODE == kLayer ? fma2(gg[k][p], rs2, nra) : mul2(gg[k][p], rs2));
            if (RESID) {
              float2 dh[4];
              chunk_to_f2(*reinterpret_cast<const uint4 *>(stx + 2 * L.tensor_bytes +
                                                           static_cast<size_t>(r) * a.NS * 2 +
                                                           (t + k * a.tpr) * 16),
                          dh);
#pragma unroll
              for (int p = 0; p < 4; ++p) o[p] = add2(o[p], dh[p]);
            }
            if (DROP) {
              const int64_t at = (row0 + r) * a.N + col0 + (t + k * a.tpr) * 8;
              st_global_cs_v4(a.out2 + at, f2_to_chunk(o));
              gen.template chunk<8>(o, static_cast<uint64_t>(at));
            }
            st_global_cs_v4(dxrow + k * a.tpr * 8, f2_to_chunk(o));
          }
        }
      }
    }

    if (last_warp_done(done_cnt, s, nwarps)) {
      const int64_t next = tile + static_cast<int64_t>(a.S) * ncl;
      if (next < a.ntiles) {
        if ((tid & 31) == 0) fence_proxy_async_smem();
        __syncwarp();
        issue_bwd_tile<MODE, CLUSTER, RESID>(a, L, smem, next, s, col0, nsc_me, pol);
      }
    }
    if (++s == a.S) {
      s = 0;
      par ^= 1u;
    }
  }

  write_column_partials<MODE, K, EXACT>(a, smem, accg, accb, g, t, nsc_me, cid, col0);
  if (CLUSTER) cluster_sync();
}

}  // namespace gbn
