// linear_split.cu -- products of norm_linear_fwd / norm_linear_bwd with few or
// middling rows (tokens): 128 output features x `bn` tokens per cluster, whose
// CTAs share the contraction.
//
// Few tokens: bound by reading the weights once, and for one layer alone by the
// way from launch to first byte and from last byte to result.  The weights are the
// MMA's 128-row operand and the tokens its columns (16 at least), so a tile of W
// feeds the tensor core whatever the number of tokens, and a layer of 4096
// features has 32 tiles: the contraction is cut into up to 8 parts to keep
// every SM's copies in flight.  Each CTA streams its part of W and x by TMA (the
// first stages before anything else is set up).  The tile's tokens are shared out
// among the CTAs, which add the fp32 partial sums of theirs in rank order (no
// atomics) and write them with the epilogue, whole 256-byte rows per warp.  Up to
// 16 tokens go from tensor memory straight to their owners over distributed
// shared memory, behind one cluster barrier; more go through the CTA's own shared
// memory (the ring's) and are fetched in 16-byte pieces, behind two (64 tokens by
// single words: 17 us where this takes 12).  A CTA holds no tensor memory while it
// waits for a peer that might wait for some, so clusters of different streams
// cannot block each other.
#include <cuda.h>
#include <cuda_runtime.h>

#include "linear.cuh"

namespace gbn {

namespace {

__device__ __forceinline__ float4 ld_peer(uint32_t local, int rank) {
  uint32_t remote;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(remote)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_peer(uint32_t remote, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(v) : "memory");
}

// Four consecutive elements (fewer at the end of a row).
template <int DT>
__device__ __forceinline__ void load4(const void *base, int64_t at, int count, bool vec, float (&f)[4]) {
  if (vec && count == 4) {
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + at);
    const float2 a = lin_unpack<DT>(w.x), b = lin_unpack<DT>(w.y);
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < count ? load_elem<DT>(base, at + i) : 0.f;
  }
}
template <int DT>
__device__ __forceinline__ void store4(void *base, int64_t at, int count, bool vec, const float (&f)[4]) {
  if (vec && count == 4) {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + at) =
        make_uint2(lin_pack<DT>(f[0], f[1]), lin_pack<DT>(f[2], f[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < count) store_elem<DT>(base, at + i, f[i]);
  }
}

// sums[c] = part[0][c] + part[1][c] + ..., a column per thread, in order.
__device__ __forceinline__ void add_rows(const SplitArgs &a, int first) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int c = first + static_cast<int>(threadIdx.x);
  if (c >= a.cols) return;
  float v = 0.f;
#pragma unroll 8
  for (int r = 0; r < a.rows; ++r) v += __ldcg(a.part + int64_t(r) * a.cols + c);
  a.sums[c] = v;
}

// FWD: one product of two K-major operands (what a decoding step runs; with the
// choices at run time 48 x 4096 x 16384 takes 28.6 us, compiled in 27.4).
template <int DT, bool FWD>
__global__ void __launch_bounds__(kSplitThreads)
    linear_split_kernel(const __grid_constant__ SplitMaps maps, const __grid_constant__ SplitArgs args) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t *ring = smem_raw + pad;
  const int splits = args.splits;
  const int cluster = blockIdx.x / splits;
  const int which = FWD ? 0 : cluster >= args.q[0].clusters;
  const SplitProblem &p = args.q[which];
  if (!FWD && which && cluster >= args.q[0].clusters + p.clusters) {  // whole clusters
    add_rows(args, (blockIdx.x - (args.q[0].clusters + p.clusters) * splits) * kSplitThreads);
    return;
  }
  const CUtensorMap &tm_a = maps.a[which], &tm_b = maps.b[which];
  const bool a_mn = !FWD && p.a_mn, b_mn = !FWD && p.b_mn;
  const uint32_t stage_bytes = split_stage_bytes(p.bn);
  const int share = split_share(p.bn, splits);
  const bool push = split_push(p.bn, splits);
  uint64_t *full = reinterpret_cast<uint64_t *>(ring + p.stages * stage_bytes);
  // received: [rank][share][128 features]; or this CTA's: [token][128], in the ring
  float *part = reinterpret_cast<float *>(push ? reinterpret_cast<uint8_t *>(full) + 256 : ring);
  uint64_t *empty = full + kSplitMaxStages;
  uint64_t *acc = empty + kSplitMaxStages;  // every MMA of the CTA finished
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc + 1);
  volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = warp_index();
  const int lane = threadIdx.x % 32;
  const int rank = splits > 1 ? int(cluster_ctarank()) : 0;
  const int tile = cluster - (which ? args.q[0].clusters : 0);
  const int j0 = (tile % p.tiles_j) * p.bn;  // first token
  const int i0 = (tile / p.tiles_j) * 128;   // first feature
  const int kb0 = int(int64_t(p.nk) * rank / splits), kb1 = int(int64_t(p.nk) * (rank + 1) / splits);
  const int nkb = kb1 - kb0;
  const int stages = p.stages;
  const int tokens = min(p.bn, p.m - j0);

  // Fetches K block kb0 + n into stage s.
  const auto fetch = [&](int n, int s) {
    mbar_arrive_expect_tx(&full[s], stage_bytes);
    uint8_t *b = ring + s * stage_bytes, *a = b + 16384;
    const int k0 = (kb0 + n) * kLinBK;
    if (b_mn) {
      tma_load_2d(b, &tm_b, i0, k0, &full[s]);
      tma_load_2d(b + 8192, &tm_b, i0 + 64, k0, &full[s]);
    } else {
      tma_load_2d(b, &tm_b, k0, i0, &full[s]);
    }
    if (a_mn) {
      for (int c = 0; c < p.bn; c += 64) tma_load_2d(a + c * 128, &tm_a, j0 + c, k0, &full[s]);
    } else {
      tma_load_2d(a, &tm_a, k0, j0, &full[s]);
    }
  };

  if (warp == 0 && elect_one()) {
    prefetch_tensor_map(&tm_a);
    prefetch_tensor_map(&tm_b);
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc, 1);
    *abort = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncwarp();
  if (splits > 1) cluster_arrive_release();  // this CTA runs: peers may write to it
  grid_dependency_wait();  // before tensor memory is taken: never held while waiting
  if (warp == 0) {
    if (elect_one())
      for (int n = 0; n < stages && n < nkb; ++n) fetch(n, n);
    __syncwarp();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, args.tmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();
  const uint32_t tmem = *tmem_slot;

  // The epilogue's first operands, fetched while the products run: this CTA owns
  // tokens ja .. jb - 1 of the tile, a warp per token, four features per lane.
  const LinEpilogue &e = p.e;
  const bool vec = p.vec;
  const int ja = min(tokens, rank * share), jb = min(tokens, ja + share);
  const int i = i0 + lane * 4;
  const int count = min(4, p.n - i);
  float bias[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f};
  const auto load_r = [&](int j) {
    if (e.r && count > 0 && j < jb) load4<DT>(e.r, int64_t(j0 + j) * e.ldr + i, count, vec, r);
  };

  if (warp == 0) {
    if (elect_one()) {
      int issued = min(stages, nkb);
      for (; issued < nkb; ++issued) {
        const int s = issued % stages;
        if (!mbar_wait(&empty[s], (issued / stages - 1) & 1, args.err, abort)) break;
        fetch(issued, s);
      }
      // No copy may still be landing when the CTA exits.
      volatile int never = 0;
      for (int s = 0; s < stages && s < issued; ++s) {
        const int loads = (issued - s + stages - 1) / stages;
        mbar_wait(&full[s], (loads - 1) & 1, args.err, &never);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      // rows of the accumulator: features; columns: tokens
      const uint32_t idesc = lin_idesc(128, p.bn, DT == kBF16, b_mn, a_mn);
      const uint32_t astep = lin_kstep(a_mn), bstep = lin_kstep(b_mn);
      int s = 0;
      uint32_t ph = 0;
      for (int kb = 0; kb < nkb; ++kb) {
        if (!mbar_wait(&full[s], ph, args.err, abort)) break;
        tc_fence_after();
        const uint32_t base = smem_addr(ring + s * stage_bytes);
        const uint64_t bd = lin_desc(base, b_mn), ad = lin_desc(base + 16384, a_mn);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_bf16_ss(tmem, bd + k * bstep, ad + k * astep, idesc, (kb | k) != 0);
        mma_commit(&empty[s]);
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
      }
      mma_commit(acc);
    }
    __syncwarp();
  }
  if (e.bias && count > 0) load4<DT>(e.bias, i, count, vec, bias);
  load_r(ja + warp);
  __syncwarp();
  if (splits > 1) cluster_wait_acquire();  // every CTA of the cluster runs
  if (warp >= 2) {
    mbar_wait(acc, 0, args.err, abort);
    __syncwarp();
    tc_fence_after();
    const int t0 = (warp & 3) * 32;
    const uint32_t t_lane = tmem + (uint32_t(t0) << 16);
    if (push) {
      uint32_t v[16];
      tmem_ld_n<16>(t_lane, v);
      tmem_wait_ld_n<16>(v);
      float *const mine = part + rank * share * 128 + t0 + lane;
      int owner = 0, at = 0;  // of token q: its CTA, and its row there
      uint32_t to = mapa_shared(mine, 0);
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        if (q < tokens) {
          st_peer(to + uint32_t(at) * 512u, v[q]);
          if (++at == share && ++owner < splits) {
            at = 0;
            to = mapa_shared(mine, owner);
          }
        }
      }
    } else {
      for (int c = 0; c < tokens; c += 16) {
        uint32_t v[16];
        tmem_ld_n<16>(t_lane + c, v);
        tmem_wait_ld_n<16>(v);
#pragma unroll
        for (int q = 0; q < 16; ++q) part[(c + q) * 128 + t0 + lane] = __uint_as_float(v[q]);
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  if (splits > 1) cluster_arrive_release();
  __syncthreads();
  if (warp == 1) {  // every read of it is done; freed before the peers are waited for
    tc_fence_after();
    tmem_dealloc(tmem, args.tmem);
  }
  if (splits > 1) cluster_wait_acquire();

  if (count > 0) {
    for (int j = ja + warp; j < jb; j += kSplitThreads / 32) {
      const int64_t row = j0 + j;
      float4 v[8];
      if (push || splits == 1) {
        const float *src = part + (j - ja) * 128 + lane * 4;  // (one CTA owns all: ja = 0)
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s < splits) v[s] = *reinterpret_cast<const float4 *>(src + s * share * 128);
      } else {
        const uint32_t src = smem_addr(part + j * 128 + lane * 4);
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s < splits) v[s] = ld_peer(src, s);
      }
      float f[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int s = 1; s < 8; ++s)
        if (s < splits) f[0] += v[s].x, f[1] += v[s].y, f[2] += v[s].z, f[3] += v[s].w;
#pragma unroll
      for (int q = 0; q < 4; ++q) f[q] += bias[q];
      if (e.z) store4<DT>(e.z, row * e.ldz + i, count, vec, f);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float z = f[q];
        f[q] = (e.act == kLinNone ? z : e.act == kLinSilu ? lin_act<kLinSilu>(z)
                                                          : lin_act<kLinGelu>(z)) +
               r[q];
      }
      store4<DT>(e.y, row * e.ldy + i, count, vec, f);
      load_r(j + kSplitThreads / 32);
    }
  }
  if (splits > 1 && !push) {  // peers may still read this CTA's partials
    __syncwarp();
    cluster_sync();
  }
}

}  // namespace

const void *linear_split_kernel_ptr(bool fwd, bool bf16) {
  if (fwd)
    return bf16 ? reinterpret_cast<const void *>(&linear_split_kernel<kBF16, true>)
                : reinterpret_cast<const void *>(&linear_split_kernel<kFP16, true>);
  return bf16 ? reinterpret_cast<const void *>(&linear_split_kernel<kBF16, false>)
              : reinterpret_cast<const void *>(&linear_split_kernel<kFP16, false>);
}

}  // namespace gbn
