// linear_pair.cu -- large products of norm_linear_fwd / norm_linear_bwd:
// 256 x bn output tiles by CTA pairs (bn a multiple of 32 up to 256), with the
// epilogue of linear.cuh.
//
// Bound by the tensor cores (one 256 x 256 x 64 block takes a pair about 512
// clocks; its 64 KB of operands come from L2 mostly).  A persistent grid of
// 2-CTA clusters walks the tiles; per CTA:
//   warp 0   TMA loads of 128 A rows and bn / 2 B rows per stage (5 to 9
//            stages), counted on rank 0's barrier;
//   warp 1   (rank 0) four cta_group::2 MMAs per K block into one of two
//            accumulators in tensor memory;
//   warps 2-9  drain the other accumulator: 64 columns at a time, two warps per
//            32 rows taking them in turn, each through its own swizzled output
//            buffers and TMA stores, so that no barrier joins the eight.  A
//            residual tile is loaded into the buffer that its output leaves
//            from, a slice of the warp earlier where there are two buffers.
// Rows of outputs or residuals that tensor copies cannot address (an odd row
// length, for example), and the last 32 columns of a tile that is no multiple of
// 64 wide, are moved by the warps, two elements per lane.
#include <cuda.h>
#include <cuda_runtime.h>

#include "linear.cuh"

namespace gbn {

namespace {

constexpr uint32_t kTile = 16384;  // 128 x 64 elements
constexpr int kMaxStages = kPairMaxStages;
constexpr int kMaxSets = 2;  // output buffers (pairs with z) of a warp
constexpr int kSliceCols = 64;

__device__ __forceinline__ void wait_read(int left) {
  if (left == 0)
    bulk_wait_read_all();
  else
    bulk_wait_read_but_one();
}

// Tiles in groups of gm row blocks, column by column within a group, so that
// those in flight share operands in L2.
struct Walk {
  int m_tiles, n_tiles, gm, first, step;
  __device__ __forceinline__ bool at(int j, int &mb, int &nb) const {
    const int tile = first + j * step;
    if (tile >= m_tiles * n_tiles) return false;
    const int per_group = gm * n_tiles;
    const int group = tile / per_group;
    const int row0 = group * gm;
    const int rows = min(gm, m_tiles - row0);
    const int idx = tile - group * per_group;
    mb = row0 + idx % rows;
    nb = idx / rows;
    return true;
  }
};

template <int DT, int ACT>
__device__ __forceinline__ void finish(float (&v)[2], const float *bias, uint32_t rw, bool has_r,
                                       uint32_t &zw, uint32_t &yw) {
  if (bias) {
    v[0] += bias[0];
    v[1] += bias[1];
  }
  zw = lin_pack<DT>(v[0], v[1]);
  v[0] = lin_act<ACT>(v[0]);
  v[1] = lin_act<ACT>(v[1]);
  if (has_r) {
    const float2 r = lin_unpack<DT>(rw);
    v[0] += r.x;
    v[1] += r.y;
  }
  yw = lin_pack<DT>(v[0], v[1]);
}

// 32 accumulator columns of one row: bias, z, activation, residual; the 16-byte
// chunks q0 .. q0 + 3 of the row's 128-byte lines in the buffers.
template <int DT, int ACT>
__device__ __forceinline__ void finish32(const uint32_t (&acc)[32], const float *bias, int q0,
                                         int row, uint8_t *ybuf, uint8_t *zbuf, bool has_r) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t at = uint32_t(row) * 128u + uint32_t(((q0 + q) ^ (row & 7)) << 4);
    uint4 rv = make_uint4(0u, 0u, 0u, 0u), zv, yv;
    if (has_r) rv = *reinterpret_cast<const uint4 *>(ybuf + at);
    const uint32_t rw[4] = {rv.x, rv.y, rv.z, rv.w};
    uint32_t zw[4], yw[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float v[2] = {__uint_as_float(acc[q * 8 + 2 * p]), __uint_as_float(acc[q * 8 + 2 * p + 1])};
      finish<DT, ACT>(v, bias ? bias + q * 8 + 2 * p : nullptr, rw[p], has_r, zw[p], yw[p]);
    }
    if (zbuf) {
      zv = make_uint4(zw[0], zw[1], zw[2], zw[3]);
      *reinterpret_cast<uint4 *>(zbuf + at) = zv;
    }
    yv = make_uint4(yw[0], yw[1], yw[2], yw[3]);
    *reinterpret_cast<uint4 *>(ybuf + at) = yv;
  }
}

// The warp's 32 rows x 64 columns between a swizzled buffer and rows that no
// tensor copy addresses: lane l takes columns l and l + 32, eight rows at a time
// (777 x 1234 x 999 with r and z, tiles of 64: 15.9 us with four at a time and
// their loads behind each other's stores, 15.3 now).
template <bool LOAD>
__device__ __forceinline__ void copy_rows(uint8_t *buf, int t0, void *base, int64_t ld, int row0,
                                          int m, int col0, int n) {
  const int lane = threadIdx.x & 31;
  uint16_t *g = static_cast<uint16_t *>(base);
  const auto at = [&](int r, int c) {
    const int t = t0 + r;
    return reinterpret_cast<uint16_t *>(buf + t * 128 + (((c >> 3) ^ (t & 7)) << 4)) + (c & 7);
  };
#pragma unroll 1
  for (int r0 = 0; r0 < 32 && row0 + r0 < m; r0 += 8) {
    uint16_t v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = r0 + i / 2, c = lane + 32 * (i & 1);
      const bool in = row0 + r < m && col0 + c < n;
      if (!LOAD)
        v[i] = *at(r, c);
      else if (in)
        v[i] = g[static_cast<int64_t>(row0 + r) * ld + col0 + c];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = r0 + i / 2, c = lane + 32 * (i & 1);
      const bool in = row0 + r < m && col0 + c < n;
      if (LOAD && in) *at(r, c) = v[i];
      if (!LOAD && in) g[static_cast<int64_t>(row0 + r) * ld + col0 + c] = v[i];
    }
  }
}

template <bool AMN, bool BMN, int DT>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tm_a,
                       const __grid_constant__ CUtensorMap tm_b,
                       const __grid_constant__ CUtensorMap tm_y,
                       const __grid_constant__ CUtensorMap tm_z,
                       const __grid_constant__ CUtensorMap tm_r, const PairArgs p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t *ring = smem_raw + pad;
  uint8_t *staging = ring + kPairTiles - p.bufs * kTile;  // behind the stages
  float *bias_s = reinterpret_cast<float *>(ring + kPairTiles);
  uint64_t *full = reinterpret_cast<uint64_t *>(bias_s + 256);
  uint64_t *empty = full + kMaxStages;
  uint64_t *acc_full = empty + kMaxStages;  // [2]
  uint64_t *acc_empty = acc_full + 2;       // [2]
  uint64_t *done = acc_empty + 2;
  uint64_t *rfull = done + 1;               // [8 warps][kMaxSets]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(rfull + 8 * kMaxSets);
  volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = warp_index();
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int stages = p.stages;
  const uint32_t kstage = pair_stage(p.bn, BMN);  // A tile, then B tile
  Walk walk;
  walk.m_tiles = (p.m + 255) / 256;
  walk.n_tiles = (p.n + p.bn - 1) / p.bn;
  walk.gm = p.gm;
  walk.first = blockIdx.x / 2;
  walk.step = gridDim.x / 2;

  grid_dependency_wait();  // before tensor memory is taken: never held while waiting
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 16);  // eight warps of each CTA
    }
    mbar_init(done, 1);
    for (int i = 0; i < 8 * kMaxSets; ++i) mbar_init(&rfull[i], 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  grid_launch_dependents();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (elect_one()) {
      int s = 0, issued = 0;
      uint32_t ph = 0;
      bool ok = true;
      const uint32_t full_rank0 = mapa_shared(full, 0);
      int mb, nb;
      for (int j = 0; ok && walk.at(j, mb, nb); ++j) {
        const int m0 = mb * 256 + int(rank) * 128;
        const int n0 = nb * p.bn + int(rank) * (p.bn / 2);
        for (int kb = 0; kb < p.nk; ++kb) {
          if (issued >= stages && !mbar_wait(&empty[s], ph ^ 1u, p.err, abort)) {
            ok = false;
            break;
          }
          const uint32_t bar = full_rank0 + uint32_t(s * 8);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kstage);
          uint8_t *a = ring + s * kstage, *b = a + kTile;
          const int k0 = kb * kLinBK;
          if (AMN) {
            tma_load_2d_pair(a, &tm_a, m0, k0, bar);
            tma_load_2d_pair(a + 8192, &tm_a, m0 + 64, k0, bar);
          } else {
            tma_load_2d_pair(a, &tm_a, k0, m0, bar);
          }
          if (BMN) {
            tma_load_2d_pair(b, &tm_b, n0, k0, bar);
            tma_load_2d_pair(b + 8192, &tm_b, n0 + 64, k0, bar);
          } else {
            tma_load_2d_pair(b, &tm_b, k0, n0, bar);
          }
          ++issued;
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // No copy may still be landing in either CTA when the pair exits: rank 0
      // sees the bytes of both.
      if (rank == 0) {
        volatile int never = 0;
        for (int i = 0; i < stages && i < issued; ++i) {
          const int loads = (issued - i + stages - 1) / stages;
          mbar_wait(&full[i], (loads - 1) & 1, p.err, &never);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = lin_idesc(256, p.bn, DT == kBF16, AMN, BMN);
      constexpr uint32_t astep = lin_kstep(AMN), bstep = lin_kstep(BMN);
      const uint64_t adesc0 = lin_desc(smem_addr(ring), AMN);
      const uint64_t bdesc0 = lin_desc(smem_addr(ring + kTile), BMN);
      const uint32_t full0 = smem_addr(full), empty0 = smem_addr(empty);
      bool ok = true;
      int s = 0, mb, nb;
      uint32_t ph = 0;
      for (int j = 0; ok && walk.at(j, mb, nb); ++j) {
        const int b = j & 1;
        if (j >= 2 && !mbar_wait_cluster(&acc_empty[b], ((j >> 1) - 1) & 1, p.err, abort)) break;
        tc_fence_after();
        const uint32_t d = tmem + uint32_t(b * 256);
        for (int kb = 0; kb < p.nk; ++kb) {
          const uint32_t fb = full0 + 8u * uint32_t(s);
          if (!mbar_try_wait_sa(fb, ph) && !mbar_wait_sa(fb, ph, p.err, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = adesc0 + uint32_t(s) * (kstage >> 4);
          const uint64_t bd = bdesc0 + uint32_t(s) * (kstage >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16_ss_pair(d, ad + k * astep, bd + k * bstep, idesc, (kb | k) != 0);
          mma_commit_pair_sa(empty0 + 8u * uint32_t(s), 0x3);
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (ok) mma_commit_pair(&acc_full[b], 0x3);
      }
      mma_commit_pair(done, 0x3);
    }
    __syncwarp();
  } else {
    // Warp w reaches tensor-memory lanes 32 (w % 4) .. + 31.
    const int quarter = warp & 3, half = (warp - 2) / 4;
    const int t0 = quarter * 32, t = t0 + lane;
    const LinEpilogue &e = p.e;
    const bool has_r = e.r != nullptr, pre = has_r && p.tma_r;
    const int sets = p.sets, ahead = sets - 1;
    uint8_t *const bufs = staging + half * (p.bufs / 2) * int(kTile);  // this half's
    const int zset = sets * int(kTile);
    const uint32_t acc_empty0 = mapa_shared(acc_empty, 0);
    uint64_t *rbar = rfull + (warp - 2) * kMaxSets;
    // A slice is whole (64 columns, moved by tensor copies) or the last 32 of a
    // tile; the warp takes every other one.
    const auto whole = [&](int h) { return (h + 1) * kSliceCols <= p.bn; };
    const auto in_tile = [&](int h, int nb) {
      return h * kSliceCols < p.bn && nb * p.bn + h * kSliceCols < p.n;
    };
    int lj = 0, lh = half, lset = 0;  // next residual slice to load: tile, slice, set
    auto load_next = [&]() {          // one lane
      int mb, nb;
      for (;; ++lj, lh = half) {
        if (!walk.at(lj, mb, nb)) return;
        if (in_tile(lh, nb)) break;
      }
      if (whole(lh)) {
        mbar_arrive_expect_tx(rbar + lset, 4096);
        tma_load_2d(bufs + lset * kTile + t0 * 128, &tm_r, nb * p.bn + lh * kSliceCols,
                    mb * 256 + int(rank) * 128 + t0, rbar + lset);
      }
      lset = lset + 1 == sets ? 0 : lset + 1;
      lh += 2;
    };
    if (pre && elect_one())
      for (int i = 0; i < ahead; ++i) load_next();
    uint32_t rphase = 0;  // per set: parity of its next load
    int set = 0;
    int mb, nb;
    for (int j = 0; walk.at(j, mb, nb); ++j) {
      const int b = j & 1;
      const int row0 = mb * 256 + int(rank) * 128 + t0;
      const int n0 = nb * p.bn;
      mbar_wait(&acc_full[b], (j >> 1) & 1, p.err, abort);
      if (e.bias) {
        named_bar_sync(1, 256);  // the last tile's values have been read
        const int c = threadIdx.x - 64;
        bias_s[c] = c < p.bn && n0 + c < p.n ? load_elem<DT>(e.bias, n0 + c) : 0.f;
        named_bar_sync(1, 256);
      }
      __syncwarp();
      tc_fence_after();
      const uint32_t t_lane = tmem + (uint32_t(t0) << 16) + uint32_t(b * 256);
      const auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (elect_one()) {
          if (rank == 0)
            mbar_arrive(&acc_empty[b]);
          else
            mbar_arrive_remote(acc_empty0 + uint32_t(b * 8));
        }
      };
      if (!in_tile(half, nb)) release();
#pragma unroll 1
      for (int h = half; in_tile(h, nb); h += 2) {
        const int col = n0 + h * kSliceCols;
        const int cols_end = min(p.n, n0 + p.bn);
        const bool by_tma = whole(h);
        uint8_t *ybuf = bufs + set * kTile;
        uint8_t *zbuf = e.z ? ybuf + zset : nullptr;
        __syncwarp();
        if (elect_one()) {
          if (pre) {
            wait_read(0);
            load_next();
          } else {
            wait_read(sets - 1);
          }
        }
        __syncwarp();
        uint32_t acc[2][32];
        tmem_ld32(t_lane + h * kSliceCols, acc[0]);
        tmem_ld32(t_lane + h * kSliceCols + 32, acc[1]);
        if (pre && by_tma) {
          mbar_wait(&rbar[set], (rphase >> set) & 1, p.err, abort);
          rphase ^= 1u << set;
        } else if (has_r) {
          copy_rows<true>(ybuf, t0, const_cast<void *>(e.r), e.ldr, row0, p.m, col, cols_end);
        }
        __syncwarp();
        tmem_wait_ld(acc[0]);
        tmem_wait_ld(acc[1]);
        if (!in_tile(h + 2, nb)) release();  // this warp has read its slices
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float *bs = e.bias ? bias_s + h * kSliceCols + q * 32 : nullptr;
          if (e.act == kLinNone)
            finish32<DT, kLinNone>(acc[q], bs, q * 4, t, ybuf, zbuf, has_r);
          else if (e.act == kLinSilu)
            finish32<DT, kLinSilu>(acc[q], bs, q * 4, t, ybuf, zbuf, has_r);
          else
            finish32<DT, kLinGelu>(acc[q], bs, q * 4, t, ybuf, zbuf, has_r);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (elect_one()) {
          if (row0 < p.m && by_tma) {
            if (p.tma_y) tma_store_2d(&tm_y, col, row0, ybuf + t0 * 128);
            if (zbuf && p.tma_z) tma_store_2d(&tm_z, col, row0, zbuf + t0 * 128);
          }
          bulk_commit();
        }
        if (!p.tma_y || !by_tma) copy_rows<false>(ybuf, t0, e.y, e.ldy, row0, p.m, col, cols_end);
        if (zbuf && !(p.tma_z && by_tma))
          copy_rows<false>(zbuf, t0, e.z, e.ldz, row0, p.m, col, cols_end);
        set = set + 1 == sets ? 0 : set + 1;
      }
    }
    if (elect_one()) bulk_wait_all();
    __syncwarp();
  }

  // Every MMA has finished before tensor memory is freed, and neither CTA exits
  // while the other may still signal it or load into it.
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) {
      volatile int never = 0;
      mbar_wait(done, 0, p.err, &never);
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  cluster_sync();
}

template <bool AMN, bool BMN>
const void *pick(bool bf16) {
  return bf16 ? reinterpret_cast<const void *>(&linear_pair_kernel<AMN, BMN, kBF16>)
              : reinterpret_cast<const void *>(&linear_pair_kernel<AMN, BMN, kFP16>);
}

}  // namespace

const void *linear_pair_kernel_ptr(bool a_mn, bool b_mn, bool bf16) {
  if (a_mn) return b_mn ? pick<true, true>(bf16) : nullptr;
  return b_mn ? pick<false, true>(bf16) : pick<false, false>(bf16);
}

}  // namespace gbn
