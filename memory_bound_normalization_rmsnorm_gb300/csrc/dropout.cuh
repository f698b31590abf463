// dropout.cuh -- the counter-based dropout mask shared by every kernel that
// drops elements.  Nothing of the mask is stored: it is a function of (seed,
// offset, element index), so a backward pass recomputes the forward's.
//
// Block i of eight consecutive elements of the (flattened, row-major) tensor
// takes the four 32-bit outputs of Philox4x32-10 (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011) at the
// 128-bit counter (i, offset) under the 64-bit key `seed`; element e of the
// block reads 16-bit half e (the low half of word e / 2 first) and is kept
// when half >= T, T = p * 2^16 to the nearest integer.  Kept elements are
// multiplied by 2^16 / (2^16 - T), the exact inverse of the probability that
// the comparison keeps, so the expectation is the input's whatever p.
//
// Sixteen bits per element, so one generator call serves one 16-byte chunk
// of bf16: the call is about 45 issue slots, 6 per element instead of 11
// with 32 bits, which is what keeps plain dropout (4 bytes per element, 21
// issue slots per element at the measured copy bandwidth) memory-bound.
// The price is that p is held to the nearest multiple of 2^-16.
#pragma once
#include "elem.cuh"

namespace gbn {

// The generator of one kernel argument.
struct DropGen {
  const DropArgs &a;
  uint32_t o0, o1;

  __device__ __forceinline__ explicit DropGen(const DropArgs &args) : a(args), o0(0), o1(0) {}
  // Reads the offset word (after the previous kernel's writes are visible).
  __device__ __forceinline__ void start() {
    uint64_t o = a.offset;
    if (a.offset_dev) o += *a.offset_dev;
    o0 = static_cast<uint32_t>(o);
    o1 = static_cast<uint32_t>(o >> 32);
  }

  // The four words of block `i`.
  __device__ __forceinline__ uint4 words(uint64_t i) const {
    uint32_t c0 = static_cast<uint32_t>(i), c1 = static_cast<uint32_t>(i >> 32), c2 = o0, c3 = o1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t m0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
      const uint64_t m1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
      c0 = static_cast<uint32_t>(m1 >> 32) ^ c1 ^ a.key[r][0];
      c1 = static_cast<uint32_t>(m1);
      c2 = static_cast<uint32_t>(m0 >> 32) ^ c3 ^ a.key[r][1];
      c3 = static_cast<uint32_t>(m0);
    }
    return make_uint4(c0, c1, c2, c3);
  }

  // Dropout of the pair whose halves are word w.  A dropped element is 0
  // whatever its value (infinities and NaN included), so this selects.
  __device__ __forceinline__ float2 pair(float2 v, uint32_t w) const {
    const float2 s = mul2(v, splat2(a.scale));
    return make_float2((w << 16) >= a.thr ? s.x : 0.f, w >= a.thr ? s.y : 0.f);
  }

  // Dropout of the 16-byte chunk of V elements that starts at element
  // index e (a multiple of V).
  template <int V>
  __device__ __forceinline__ void chunk(float2 (&v)[V / 2], uint64_t e) const {
    const uint4 w = words(e >> 3);
    if constexpr (V == 8) {
      v[0] = pair(v[0], w.x);
      v[1] = pair(v[1], w.y);
      v[2] = pair(v[2], w.z);
      v[3] = pair(v[3], w.w);
    } else {
      const bool hi = (e & 4) != 0;
      v[0] = pair(v[0], hi ? w.z : w.x);
      v[1] = pair(v[1], hi ? w.w : w.y);
    }
  }

  // Zeroes the dropped elements of a 16-byte chunk as it lies in memory (the
  // kept ones still want the factor).
  template <int DT>
  __device__ __forceinline__ void mask(uint4 &c, uint64_t e) const {
    const uint4 w = words(e >> 3);
    if constexpr (DT == kFP32) {
      const bool hi = (e & 4) != 0;
      const uint32_t u = hi ? w.z : w.x, v = hi ? w.w : w.y;
      c.x = (u << 16) >= a.thr ? c.x : 0u;
      c.y = u >= a.thr ? c.y : 0u;
      c.z = (v << 16) >= a.thr ? c.z : 0u;
      c.w = v >= a.thr ? c.w : 0u;
    } else {
      auto kept = [&](uint32_t u) {
        return ((u << 16) >= a.thr ? 0xffffu : 0u) | (u >= a.thr ? 0xffff0000u : 0u);
      };
      c.x &= kept(w.x);
      c.y &= kept(w.y);
      c.z &= kept(w.z);
      c.w &= kept(w.w);
    }
  }
};

}  // namespace gbn
