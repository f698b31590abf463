// linear.cuh -- the linear layer with bias, activation and residual in its
// epilogue (norm_linear_fwd) and its gradients (norm_linear_bwd): arguments of
// the kernels, operand descriptors and the arithmetic of the epilogue.
//
// Every product is out[j, i] = sum_k A[j, k] B[i, k] over two 16-bit matrices,
// fp32 accumulation in tensor memory, i the contiguous dimension of the output:
//   forward  A = x   [M, K]            B = W   [N, K]            j token, i feature
//   dx       A = dz  [M, N]            B = W^T (W read along its rows)
//   dW       A = dz^T                  B = x^T (both read along their rows)
// An operand stored with k contiguous is K-major, else MN-major; the tensor
// cores take either from shared memory, so no transpose is ever written.
#pragma once
#include <cuda.h>

#include <cstdint>

#include "elem.cuh"
#include "tcgen05.cuh"

namespace gbn {

constexpr int kLinBK = 64;  // K block: one 128-byte swizzle row of 16-bit elements

// Activations, with the values of norm_act_t.
constexpr int kLinNone = 0;
constexpr int kLinSilu = 1;
constexpr int kLinGelu = 2;

struct LinEpilogue {
  const void *bias;  // [n] or null
  const void *r;     // [m, n], row stride ldr, or null
  void *z;           // [m, n], row stride ldz, or null
  void *y;           // [m, n], row stride ldy
  int64_t ldr, ldz, ldy;
  int act;
};

// ---------------------------------------------------- single-thread roles
// One lane of a converged warp.  A branch on this tells the compiler that one
// thread takes it, and warp_index() that all of a warp do, so that what they form
// there (descriptors, addresses) is uniform to it, as the tensor instructions'
// operands have to be: with `lane == 0` in its place a K block of the MMA loop took
// 440 clocks, twice that of its 256 x 128 x 64 MMAs.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ int warp_index() {
  return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
}

// Fetches a tensor map (a kernel parameter) ahead of its first copy.
__device__ __forceinline__ void prefetch_tensor_map(const void *tmap) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tmap)) : "memory");
}

// --------------------------------------------------------- descriptors
// kind::f16 with fp32 D: A and B both bf16 or both fp16, K- or MN-major.
__host__ __device__ constexpr uint32_t lin_idesc(int M, int N, bool bf16, bool a_mn, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) |
         (b_mn ? 1u << 16 : 0u) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// Shared-memory descriptor of an operand tile with the 128-byte swizzle.
// K-major: rows of 64 k (128 bytes), 8-row groups 1024 bytes apart.  MN-major:
// 64 x 64 boxes (64 rows of k, each 64 mn = 128 bytes) one after the other along
// mn: 8192 bytes from box to box (the leading offset), 1024 bytes from one
// group of 8 k to the next (the stride offset).
__device__ __forceinline__ uint64_t lin_desc(uint32_t saddr, bool mn) {
  return desc_sw128(saddr) - (uint64_t(1) << 16) + (uint64_t(mn ? 8192 >> 4 : 1) << 16);
}
// Start-address step (16-byte units) of 16 k: 32 bytes along a K-major row, 16
// rows of an MN-major box.
__host__ __device__ constexpr uint32_t lin_kstep(bool mn) { return mn ? 2048 >> 4 : 32 >> 4; }

// ---------------------------------------------------------- arithmetic
__device__ __forceinline__ float lin_ex2(float v) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
  return e;
}
constexpr float kLinLog2e = 1.4426950408889634f;
constexpr float kLinGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// act(z) = z / (1 + exp(-k(z))), k = z (SiLU) or c (z + 0.044715 z^3) (GELU).
template <int ACT>
__device__ __forceinline__ float lin_act(float z) {
  if constexpr (ACT == kLinNone) return z;
  float t;
  if constexpr (ACT == kLinSilu)
    t = -kLinLog2e * z;
  else
    t = z * fmaf(z * z, -kLinLog2e * kLinGeluC * 0.044715f, -kLinLog2e * kLinGeluC);
  return __fdividef(z, 1.f + lin_ex2(t));  // exp = inf where z is far below 0: -0
}

// act'(z) = s + z s (1 - s) k'(z) with s = sigmoid(k) and 1 - s = exp(-k) s.  z
// is clamped where act' has reached 0 or 1 (s below 2e-35 or equal to 1), so
// that no infinity meets a zero; NaN passes.
__device__ __forceinline__ float lin_act_grad(float z, int act) {
  if (act == kLinNone) return 1.f;
  const float lim = act == kLinSilu ? 80.f : 16.f;
  z = z > lim ? lim : z < -lim ? -lim : z;
  float k = z, dk = 1.f;
  if (act == kLinGelu) {
    const float q = z * z;
    k = z * fmaf(q, kLinGeluC * 0.044715f, kLinGeluC);
    k = k < -80.f ? -80.f : k;
    dk = fmaf(q, 3.f * kLinGeluC * 0.044715f, kLinGeluC);
  }
  const float e = lin_ex2(-kLinLog2e * k);
  const float s = __fdividef(1.f, 1.f + e);
  return fmaf(z * s * dk, e * s, s);
}

template <int DT>
__device__ __forceinline__ float2 lin_unpack(uint32_t w) {
  if constexpr (DT == kBF16) return bf2_to_f2(w);
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <int DT>
__device__ __forceinline__ uint32_t lin_pack(float a, float b) {
  if constexpr (DT == kBF16) return f2_to_bf2(make_float2(a, b));
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// ------------------------------------------------------------- kernels
// Output tiles of 256 x bn by CTA pairs, persistent (linear_pair.cu).
constexpr int kPairThreads = 320;
struct PairArgs {
  LinEpilogue e;
  int m, n, nk;
  int bn;       // tile columns: a multiple of 32, up to 256
  int stages;   // operand stages
  int bufs;     // 16 KB output buffers: 2 or 4
  int sets;     // of them a warp's slices use in turn (pairs where z is written): 1 or 2
  int tma_y, tma_z, tma_r;  // moved by tensor copies (else by the warps)
  int gm;       // row blocks per group of the tile walk
  unsigned *err;
};
constexpr int kPairMaxStages = 9;
// Operand ring (A and B tiles of a stage), output buffers, bias row, barriers.
constexpr uint32_t kPairTiles = 6 * 32768 + 2 * 16384;  // ring and buffers
__host__ __device__ constexpr uint32_t pair_stage(int bn, bool b_mn) {
  return 16384u + (b_mn ? 16384u : uint32_t(bn) * 64u);
}
__host__ __device__ constexpr int pair_stages(int bn, bool b_mn, int bufs) {
  const uint32_t n = (kPairTiles - uint32_t(bufs) * 16384u) / pair_stage(bn, b_mn);
  return n < uint32_t(kPairMaxStages) ? int(n) : kPairMaxStages;
}
__host__ __device__ constexpr uint32_t pair_smem() { return 1024 + kPairTiles + 1024 + 512; }
// (A MN-major, B MN-major, bf16); nullptr for A MN-major with B K-major.
const void *linear_pair_kernel_ptr(bool a_mn, bool b_mn, bool bf16);

// One 128-feature x bn-token tile per cluster of `splits` CTAs that share its k
// (linear_split.cu).
constexpr int kSplitThreads = 192;
constexpr int kSplitMaxStages = 12;
struct SplitProblem {
  LinEpilogue e;
  int m, n, nk;    // tokens, features, K blocks
  int bn;          // tokens per tile: a multiple of 16 (64 where A is MN-major), up to 256
  int stages;
  int tiles_j;     // token tiles
  int clusters;    // tiles of the problem
  int a_mn, b_mn;  // storage of the token operand (A) and of the feature operand (B)
  int vec;         // y, z, r and bias take 8-byte accesses
};
// One or two products in one launch, clusters of one after those of the other, and
// behind them CTAs that add rows of partial sums (dbias).
struct SplitArgs {
  SplitProblem q[2];
  const float *part;  // [rows, cols] or null
  float *sums;        // [cols]
  int rows, cols;
  int splits;      // CTAs per cluster
  uint32_t tmem;   // tensor-memory columns
  unsigned *err;
};
struct SplitMaps {
  CUtensorMap a[2], b[2];
};
__host__ __device__ constexpr uint32_t split_stage_bytes(int bn) { return 16384u + uint32_t(bn) * 128u; }
// Each CTA of a cluster owns a share of the tile's tokens.
__host__ __device__ constexpr int split_share(int bn, int splits) { return (bn + splits - 1) / splits; }
// Few tokens: the partial sums go straight to their owners, into a region beside
// the ring.  More: they go through the ring's memory.
__host__ __device__ constexpr bool split_push(int bn, int splits) { return bn == 16 && splits > 1; }
__host__ __device__ constexpr uint32_t split_smem(int bn, int splits, int stages) {
  return 1024u + uint32_t(stages) * split_stage_bytes(bn) + 256u +
         (split_push(bn, splits) ? uint32_t(splits * split_share(bn, splits)) * 512u : 0u);
}
// fwd: for a single product of K-major operands, without sums behind it.
const void *linear_split_kernel_ptr(bool fwd, bool bf16);

// linear_grad.cu
constexpr int kGradThreads = 256;
struct GradArgs {
  const void *dy, *z;
  void *dz;            // [M, N], row stride lddz, or null
  float *part;         // [chunks, N] column sums, or null
  int64_t lddy, ldz, lddz;
  int M, N, chunks, act;
};
// (fp16 / bf16, eight columns per thread or one)
const void *linear_grad_kernel_ptr(bool bf16, bool vec);
// (two elements at a time, where rows are even and start on four bytes)
const void *linear_pack_kernel_ptr(bool two);
struct PackArgs {  // up to two matrices
  const uint16_t *src[2];
  uint16_t *dst[2];
  int64_t ld[2], ldd[2];
  int rows[2], cols[2];
  int strips[2];  // of 256 columns (pairs of columns)
};
const void *linear_fold_kernel_ptr();

}  // namespace gbn
