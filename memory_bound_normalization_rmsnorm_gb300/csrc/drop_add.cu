// drop_add.cu -- instantiations of the row kernels with dropout of the
// residual branch in front of the residual add: the forward reads x and r,
// writes h = bf16(r + drop(x)) and y = norm(h); the backward writes dr (the
// fused residual backward's dx) and dx = drop(dr).  The generator runs on
// each 16-byte chunk where the fused residual kernels add it, about 8 issue
// slots per element on passes that move 8 and 10 bytes per element, so HBM
// stays the bound of large calls: LayerNorm 32768 x 4096 forward in 171 us
// (1.07 GB, 92 % of the measured copy bandwidth; 62 % of the issue slots),
// backward with the partial reduction in 211 us (1.34 GB, 94 %).  RMSNorm 256
// x 1024 forward takes 4.0 us, most of it launch and one row's latency.
// Splitting the dropout off into its own pass would add 4 bytes per element,
// 80 us at that size.
//
// The streaming kernels of very long rows have no form with dropout, so the
// resident long-row kernels take those.  Of the measured copy bandwidth, 4096
// rows, RMSNorm / LayerNorm: forward 93 / 79 % at 16384 columns, 89 / 75 at 32768,
// 72 / 60 at 131072; backward 91 / 52, 74 / 53, 63 / 42.  There the streaming
// norm_add_bwd and a dropout of its result are faster than the fused backward,
// although they move 12 bytes per element and not 10: 32768 columns 254 / 261 us
// against 266 / 372, 131072 960 / 1029 against 1248 / 1897.
#include "bwd_kernel.cuh"
#include "fwd_kernel.cuh"
#include "long_kernel.cuh"

namespace gbn {

namespace {

template <int MODE, int K, bool EXACT>
const void *fwd_ptr() {
  return reinterpret_cast<const void *>(
      &norm_fwd_kernel<MODE, K, false, EXACT, true, kOutBf16, false, false, true>);
}
template <int MODE, int K, bool EXACT>
const void *bwd_ptr() {
  return reinterpret_cast<const void *>(&norm_bwd_kernel<MODE, K, false, EXACT, true, true>);
}
template <int MODE, int K, bool CLUSTER, bool EXACT>
const void *long_fwd_ptr() {
  return reinterpret_cast<const void *>(
      &norm_fwd_long_kernel<MODE, K, CLUSTER, EXACT, true, kOutBf16, true>);
}
template <int MODE, int K, bool CLUSTER, bool EXACT>
const void *long_bwd_ptr() {
  return reinterpret_cast<const void *>(
      &norm_bwd_long_kernel<MODE, K, CLUSTER, EXACT, true, true>);
}

// Chunks per thread as the planner gives them: 1 to 6 and 8 in the forward,
// 1 to 4 in the backward.
template <int MODE, bool EXACT>
const void *pick_short(int K, bool bwd) {
  switch (K) {
    case 1: return bwd ? bwd_ptr<MODE, 1, EXACT>() : fwd_ptr<MODE, 1, EXACT>();
    case 2: return bwd ? bwd_ptr<MODE, 2, EXACT>() : fwd_ptr<MODE, 2, EXACT>();
    case 3: return bwd ? bwd_ptr<MODE, 3, EXACT>() : fwd_ptr<MODE, 3, EXACT>();
    case 4: return bwd ? bwd_ptr<MODE, 4, EXACT>() : fwd_ptr<MODE, 4, EXACT>();
    case 5: return bwd ? nullptr : fwd_ptr<MODE, 5, EXACT>();
    case 6: return bwd ? nullptr : fwd_ptr<MODE, 6, EXACT>();
    case 8: return bwd ? nullptr : fwd_ptr<MODE, 8, EXACT>();
    default: return nullptr;
  }
}

// Long rows: 8 chunks per thread in the forward (4 by the shape override), 4 in
// the backward.
template <int MODE, bool CLUSTER, bool EXACT>
const void *pick_long(int K, bool bwd) {
  switch (K) {
    case 4: return bwd ? long_bwd_ptr<MODE, 4, CLUSTER, EXACT>()
                       : long_fwd_ptr<MODE, 4, CLUSTER, EXACT>();
    case 8: return bwd ? nullptr : long_fwd_ptr<MODE, 8, CLUSTER, EXACT>();
    default: return nullptr;
  }
}

template <int MODE, bool EXACT>
const void *pick(int K, bool cluster, bool bwd, bool long_rows) {
  if (!long_rows) return cluster ? nullptr : pick_short<MODE, EXACT>(K, bwd);
  return cluster ? pick_long<MODE, true, EXACT>(K, bwd) : pick_long<MODE, false, EXACT>(K, bwd);
}

}  // namespace

const void *drop_add_kernel_ptr(int mode, int K, bool cluster, bool exact, bool bwd,
                                bool long_rows) {
  if (mode == kRMS)
    return exact ? pick<kRMS, true>(K, cluster, bwd, long_rows)
                 : pick<kRMS, false>(K, cluster, bwd, long_rows);
  return exact ? pick<kLayer, true>(K, cluster, bwd, long_rows)
               : pick<kLayer, false>(K, cluster, bwd, long_rows);
}

}  // namespace gbn
