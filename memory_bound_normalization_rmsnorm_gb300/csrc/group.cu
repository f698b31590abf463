// group.cu -- the group-normalisation entry points of include/gbnorm.h:
// argument validation, the choice between the resident and the streamed form
// (group.cuh) with their launch shapes, and the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <numeric>
#include <tuple>

#include "../../include/gbnorm.h"
#include "common.cuh"
#include "group.cuh"
#include "host_util.h"

namespace gbn {
namespace {

constexpr int kResident = 0, kStreamed = 1, kRing = 2;

struct GroupPlan {
  int form = kResident;
  int sg = 0, ncs = 0, nslab = 1, k = 1, cb = 1, R = 1, slots = 0, splits = 1;
  int stages = 0, nsamp = 0, rounds = 0, keep = 0, tm = 0;  // ring
  int threads = 0;
  int64_t grid = 0;
  uint32_t smem = 0;  // resident or ring kernel, or the streamed form's first pass
  uint32_t smem2 = 0; // streamed form's second pass
};

// Shape override for sweeps and tests: GBNORM_GROUP="form=1,sg=4,k=2,R=8,
// splits=3" (any subset; form 0 resident, 1 streamed, 2 ring; for the ring
// also stages=, nsamp=, tm= and keep=; cb=1 one sample per cluster).  Bypasses the cache.
struct GroupOverride {
  int form = -1, sg = 0, k = 0, R = 0, splits = 0, stages = 0, nsamp = 0, keep = -1, cb = 0, tm = -1;
  bool any = false;
};

GroupOverride read_group_override() {
  GroupOverride o;
  const char *s = std::getenv("GBNORM_GROUP");
  while (s && *s) {
    char key[16];
    int val = 0;
    if (std::sscanf(s, "%15[^=]=%d", key, &val) == 2 && val >= 0) {
      if (!std::strcmp(key, "form")) o.form = val;
      else if (!std::strcmp(key, "sg")) o.sg = val;
      else if (!std::strcmp(key, "k")) o.k = val;
      else if (!std::strcmp(key, "R")) o.R = val;
      else if (!std::strcmp(key, "splits")) o.splits = val;
      else if (!std::strcmp(key, "stages")) o.stages = val;
      else if (!std::strcmp(key, "nsamp")) o.nsamp = val;
      else if (!std::strcmp(key, "keep")) o.keep = val;
      else if (!std::strcmp(key, "cb")) o.cb = val;
      else if (!std::strcmp(key, "tm")) o.tm = val;
      o.any = true;
    }
    s = std::strchr(s, ',');
    if (s) ++s;
  }
  return o;
}

int round32(int v) { return (v + 31) & ~31; }
int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// CTAs of `threads` threads and `smem` bytes that one SM holds, at 128 registers
// per thread, the most that these kernels use (some need 64 to 104: for those
// this is too few, and the estimate was fitted with it).
int ctas_per_sm(int threads, int64_t smem, int smem_optin) {
  const int64_t by_smem = (static_cast<int64_t>(smem_optin) + 1024) / (smem + 1024);
  const int64_t by_regs = 65536 / (128 * threads);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min(by_smem, by_regs), 16)));
}

// Estimated times (us), for choosing among the plans of a shape.  Form of the
// estimate: memory time at the measured bandwidth (less for slabs narrower
// than 128 bytes of a row and where few SMs work), issue time per element and
// per thread, both stretched where the last wave of single CTAs, or the SMs'
// shares of one wave, are uneven or slabs and row lanes reach past the sample,
// and fixed times per launch, cluster and its CTAs, fold level, row of a thread
// and wave.  Large clusters leave part of the SMs unused, less so the more CTAs
// an SM takes.  The constants were fitted to 8400 measured plans of 156 shapes
// (1 to 5000 samples, 1 to 65536 positions, 32 to 2560 channels, both
// directions, 16 and 32 bits).  For the kernels and candidates of that time, and
// on the shapes of the fit, the plan of least estimate was 1.5 % slower than the
// fastest measured one in the geometric mean, 16 % at worst (a fit that knew no
// unevenness: 5.5 %, 61 % at worst; one wave of widest CTAs: 8 %).  The folds, the
// cluster exchange and the number of row lanes changed afterwards without a new
// fit, and no shape was held back from this one, so how far the choice is off on
// the present kernels and on other shapes is not known.
double resident_cost(const GroupPlan &p, double elems, double bytes, bool bwd, bool reduce,
                     int nc, int S, int sms, int smem_optin) {
  const int occ = ctas_per_sm(p.threads, p.smem, smem_optin);
  const int cluster = p.k * p.cb, seg_bytes = p.ncs * 16;
  const double grid = static_cast<double>(p.grid);
  const double usable =
      sms * (1.0 - (cluster > 4 ? 0.16 : cluster > 2 ? 0.095 : 0.0) / occ);
  const double share = grid / usable, fill = share / occ, waves = std::ceil(fill);
  const double conc = fill > 1 ? occ : std::max(1.0, std::ceil(share));
  double uneven = 1.0;
  if (fill > 1) {
    if (occ == 1) uneven += 0.70 * (waves - fill) / fill;
  } else if (share > 1) {
    uneven += 0.225 * (std::ceil(share) - share) / share;
  }
  const double past_slabs = static_cast<double>(p.ncs) * p.nslab / nc;
  const double past_rows = static_cast<double>(p.slots) * p.R * p.k / S;
  const double used = std::min(usable, grid);
  const double seg = seg_bytes >= 128 ? 1.0 : seg_bytes >= 64 ? 0.9 : seg_bytes >= 32 ? 0.8 : 0.7;
  const double mem = bytes * std::pow(past_slabs, 0.24) /
                     (6.6e6 * seg * std::min(1.0, used / (0.43 * sms)));
  const double warps = conc * p.threads / 32;
  const double issue =
      (elems * (bwd ? 0.378e-6 : 0.238e-6) * std::pow(past_slabs, 0.58) * past_rows +
       grid * p.threads * (bwd ? 4.1e-6 : 0.12e-6)) *
      sms / used / std::min(1.0, std::pow(warps / 16.0, 0.4));
  const double level = p.R > 8 ? std::log2(p.R / 8.0) : p.R > 1 ? 1.0 : 0.0;
  return 2.86 + (reduce ? 1.4 : 0.0) + (cluster > 1 ? 0.82 : 0.0) + (cluster > 4 ? 0.16 : 0.0) +
         (bwd ? 0.072 * (cluster - 1) : 0.031 * (p.k - 1)) + 0.29 * level +
         (bwd ? 0.14 : 0.07) * p.slots +
         (mem + issue) * uneven * (1.0 + 0.083 * (fill > 1 ? 1.0 / conc : 1.0)) +
         4.1 * (waves - 1);
}

// Bytes of a round's first pass that cost nothing to read again in the output
// pass (the rest of those that are still near, in shared memory, tensor memory
// and L2, come at L2's price).
constexpr double kNearBytes = 47e6;

double ring_cost(const GroupPlan &p, double elems, double bytes, double read_bytes, bool bwd,
                 int sms) {
  const double again = std::max(0.0, read_bytes / p.rounds - kNearBytes) * p.rounds;
  const double issue = elems * (bwd ? 0.38e-6 : 0.24e-6) * sms / static_cast<double>(p.grid);
  return 1.0 + (bwd ? 3.5 : 0.0) + 9.0 * p.rounds + (bytes + again) / 6.6e6 + issue;
}

// What L2 is asked to hold of it.
constexpr int64_t kL2KeepBytes = 64 << 20;

// Ring plan (group_ring.cu): slabs as wide as a CTA has threads for (whole
// rows where they fit), as many stages as shared memory holds, and rounds of
// at most n samples.
norm_status_t make_ring_plan(int B, int S, int C, int G, int dt, bool bwd, int sms, int smem_optin,
                             const GroupOverride &ov, int64_t n, GroupPlan *out) {
  const int V = chunk_elems(dt), nt = bwd ? 2 : 1;
  const int D = C / G, nc = C / V;
  const int sgu = 8 / std::gcd(D, 8);
  const int64_t unit = static_cast<int64_t>(sgu) * D / V;  // chunks of the narrowest slab
  GroupPlan p;
  p.form = kRing;
  if (nc <= kGroupThreads && !ov.sg) {
    p.sg = G;
  } else {
    if (unit > kGroupThreads) return NORM_ERR_UNSUPPORTED;
    p.sg = ov.sg ? ov.sg : static_cast<int>(std::min<int64_t>(G, kGroupThreads / unit * sgu));
    if (p.sg < 1 || p.sg > G || p.sg % sgu || static_cast<int64_t>(p.sg) * D / V > kGroupThreads)
      return NORM_ERR_UNSUPPORTED;
  }
  p.ncs = p.sg * D / V;
  p.nslab = (G + p.sg - 1) / p.sg;
  const int U = nt == 1 ? kRingRowsFwd : kRingRowsBwd;
  p.R = std::max(1, std::min(kGroupThreads / p.ncs, (S + U - 1) / U));
  if (ov.R) p.R = std::min(p.R, ov.R);
  p.threads = round32(p.ncs * p.R);
  const int TR = U * p.R;
  n = std::min<int64_t>(n, std::min(B, sms / p.nslab));
  if (n < 1) return NORM_ERR_UNSUPPORTED;
  p.rounds = static_cast<int>((B + n - 1) / n);
  p.nsamp = (B + p.rounds - 1) / p.rounds;
  const int tiles = (S + TR - 1) / TR;
  p.splits = std::max(1, std::min({sms / (p.nsamp * p.nslab), tiles, kGroupRingSplits}));
  if (ov.splits) p.splits = std::max(1, std::min({ov.splits, S, p.splits}));
  int stages = 31;
  while (stages >= 2 &&
         static_cast<int64_t>(group_ring_layout(stages, U, p.R, p.ncs, V, p.sg, bwd).total) >
             smem_optin)
    --stages;
  if (ov.stages) stages = std::min(stages, ov.stages);
  // The stages turn over in full between rounds: no CTA may have fewer tiles
  // than stages.
  if (p.rounds > 1) stages = std::min(stages, (S / p.splits + TR - 1) / TR);
  stages = std::min(stages, (static_cast<int>(ceil_div64(S, p.splits)) + TR - 1) / TR);
  if (stages < 1) return NORM_ERR_UNSUPPORTED;
  p.stages = stages;
  p.smem = group_ring_layout(stages, U, p.R, p.ncs, V, p.sg, bwd).total;
  if (static_cast<int64_t>(p.smem) > smem_optin) return NORM_ERR_UNSUPPORTED;
  p.grid = static_cast<int64_t>(p.nsamp) * p.nslab * p.splits;
  // tensor memory for what the stages do not hold
  const int most = (static_cast<int>(ceil_div64(S, p.splits)) + TR - 1) / TR;
  p.tm = std::max(0, std::min(ov.tm >= 0 ? std::min(ov.tm, kRingTmemTiles) : kRingTmemTiles,
                              most - p.stages));
  // A CTA takes all of its SM's tensor memory, and its peers wait for it at
  // the grid barrier: beside another CTA that holds some (of this kernel or of
  // one on another stream whose CTAs wait for each other too) the two could
  // wait for each other.  So it takes all of the shared memory as well, which
  // every kernel that feeds tensor memory needs.
  if (p.tm) p.smem = static_cast<uint32_t>(smem_optin);
  const int64_t tile_bytes = static_cast<int64_t>(TR) * p.ncs * 16 * nt;
  p.keep = ov.keep >= 0 ? ov.keep : static_cast<int>(kL2KeepBytes / (tile_bytes * p.grid));
  *out = p;
  return NORM_OK;
}

norm_status_t make_group_plan(int B, int S, int C, int G, int dt, bool bwd, int sms,
                              int smem_optin, const GroupOverride &ov, GroupPlan *out) {
  const int V = chunk_elems(dt), es = elem_bytes(dt), nt = bwd ? 2 : 1;
  const int D = C / G;
  const int nc = C / V;
  const double elems = static_cast<double>(B) * S * C;
  const double bytes = elems * es * (nt + 1);
  GroupPlan best;
  double best_cost = -1.0;
  // Resident: slabs of `sg` groups whose channels are a multiple of 8 (so a
  // slab starts on a 16-byte boundary in every type), clusters of 1 to 8.
  const int sgu = 8 / std::gcd(D, 8);
  const int nu = G / sgu;
  if (ov.form < 1) {
    int last = 0;
    for (int t = 1; t <= nu; ++t) {
      const int sg = ((nu + t - 1) / t) * sgu;
      if (sg == last) continue;
      last = sg;
      if (ov.sg && sg != ov.sg) continue;
      const int ncs = static_cast<int>(static_cast<int64_t>(sg) * D / V);
      if (ncs > kGroupThreads) continue;
      for (int k = 1; k <= kMaxGroupCluster && k <= S; k *= 2) {
        if (ov.k && k != ov.k) continue;
        const int rows = static_cast<int>(ceil_div64(S, k));
        const int rmax = std::min(kGroupThreads / ncs, std::max(1, S / k));
        // row lanes: all that a CTA has threads for, then fewer (several
        // smaller CTAs per SM overlap their loads, folds and stores)
        for (int R = ov.R ? std::min(rmax, ov.R) : rmax; R >= 1; R = R / 2) {
          GroupPlan p;
          p.sg = sg;
          p.ncs = ncs;
          p.nslab = (G + sg - 1) / sg;
          p.k = k;
          // a small batch in one cluster: dgamma and dbeta come out of it
          // whole, without a second launch
          if (bwd && static_cast<int64_t>(B) * k <= kMaxGroupCluster && ov.cb != 1) p.cb = B;
          // (no more lanes than that many rows per thread need: idle ones cost
          // folds and shared memory; 2 x 221 x 88 backward 5.9 -> 5.35 us)
          p.slots = (rows + R - 1) / R;
          p.R = ov.R ? R : (rows + p.slots - 1) / p.slots;
          p.threads = round32(ncs * p.R);
          const int64_t data = static_cast<int64_t>(p.slots) * ncs * p.R * 16 * nt;
          p.grid = static_cast<int64_t>(B) * p.nslab * k;
          if (data <= smem_optin && p.grid <= 0x7fffffff) {
            p.smem = group_smem_bytes(p.slots, nt, p.R, ncs, V, sg);
            if (static_cast<int64_t>(p.smem) <= smem_optin) {
              const double c =
                  resident_cost(p, elems, bytes, bwd, bwd && B > p.cb, nc, S, sms, smem_optin);
              if (best_cost < 0 || c < best_cost) {
                best_cost = c;
                best = p;
              }
            }
          }
          if (ov.R) break;
        }
      }
    }
    if (ov.form == 0 && best_cost < 0) return NORM_ERR_UNSUPPORTED;
  }
  if (ov.form < 0 || ov.form == 2) {
    // rounds of all samples, a half of them, a quarter, ...
    norm_status_t st = NORM_OK;
    for (int64_t n = ov.nsamp ? ov.nsamp : B; n >= 1; n /= 2) {
      GroupPlan p;
      st = make_ring_plan(B, S, C, G, dt, bwd, sms, smem_optin, ov, n, &p);
      if (st != NORM_OK) break;
      const double c = ring_cost(p, elems, bytes, elems * es * nt, bwd, sms);
      if (best_cost < 0 || c < best_cost) {
        best_cost = c;
        best = p;
      }
      if (ov.nsamp) break;
    }
    if (best_cost < 0 && ov.form == 2) return st;
  }
  // Streamed: groups too wide for the others.
  if (best_cost < 0) {
    GroupPlan p;
    p.form = kStreamed;
    p.sg = G;
    p.ncs = std::min(nc, kGroupThreads);
    const int rmax = std::max(1, std::min(kGroupThreads / p.ncs, S));
    p.R = ov.R ? std::min(rmax, ov.R) : rmax;
    p.threads = round32(p.ncs * p.R);
    // Row ranges: enough to fill the SMs once (with few samples) or in
    // nearly full waves, each of at least eight rows per thread.
    const int64_t resident =
        static_cast<int64_t>(sms) * std::max(1, std::min(2, 1024 / p.threads / 2));
    const int64_t most = std::max<int64_t>(1, S / (static_cast<int64_t>(p.R) * 8));
    int64_t sp = std::max<int64_t>(1, resident / B);
    for (; sp < most; ++sp) {
      const int64_t total = sp * B;
      if (total * 10 >= ceil_div64(total, resident) * resident * 9) break;
    }
    sp = std::min(sp, most);
    if (ov.splits) sp = std::min<int64_t>(ov.splits, S);
    p.splits = static_cast<int>(std::max<int64_t>(1, sp));
    p.smem = static_cast<uint32_t>(C) * 8u + group_fold_bytes(p.R, p.ncs, V);
    p.smem2 = static_cast<uint32_t>(G) * 8u;
    p.grid = static_cast<int64_t>(B) * p.splits;
    if (static_cast<int64_t>(p.smem) > smem_optin || p.grid > 0x7fffffff)
      return NORM_ERR_UNSUPPORTED;
    best = p;
  }
  *out = best;
  return NORM_OK;
}

std::mutex g_group_mu;
std::map<std::tuple<int, int64_t, int64_t, int64_t, int64_t, int>, GroupPlan> g_group_plans;

norm_status_t group_plan(int dev, int sms, int optin, int64_t B, int64_t S, int64_t C, int64_t G,
                         int dt, bool bwd, GroupPlan *out) {
  const GroupOverride ov = read_group_override();
  const auto key = std::make_tuple(dev, B, S, C, G, dt * 2 + (bwd ? 1 : 0));
  if (!ov.any) {
    std::lock_guard<std::mutex> lk(g_group_mu);
    auto it = g_group_plans.find(key);
    if (it != g_group_plans.end()) {
      *out = it->second;
      return NORM_OK;
    }
  }
  norm_status_t st = make_group_plan(static_cast<int>(B), static_cast<int>(S), static_cast<int>(C),
                                     static_cast<int>(G), dt, bwd, sms, optin, ov, out);
  if (st == NORM_OK && !ov.any) {
    std::lock_guard<std::mutex> lk(g_group_mu);
    try {
      g_group_plans[key] = *out;
    } catch (...) {  // out of host memory: the plan is made again next time
    }
  }
  return st;
}

norm_status_t check_group(int64_t B, int64_t S, int64_t C, int64_t G, norm_dtype_t dtype) {
  if (dtype != NORM_BF16 && dtype != NORM_FP16 && dtype != NORM_FP32) return NORM_ERR_ARG;
  if (B < 1 || S < 1 || C < 8 || C % 8 || C > NORM_MAX_GROUP_C) return NORM_ERR_SHAPE;
  if (G < 1 || G > C || C % G) return NORM_ERR_SHAPE;
  if (B > (int64_t(1) << 24) || S > (int64_t(1) << 30) || B * S > (int64_t(1) << 40))
    return NORM_ERR_SHAPE;
  return NORM_OK;
}

// Workspace regions (bytes from its start): the group pairs of the streamed
// and ring forms,
// then the backward's partial rows (dgamma, dbeta).
struct GroupWs {
  size_t cpart = 0, total = 0;
  int P = 0;  // partial rows of dgamma (and of dbeta)
};
GroupWs group_ws(const GroupPlan &p, int64_t B, int64_t C, int64_t G, bool bwd) {
  GroupWs w;
  if (p.form == kStreamed) w.cpart = static_cast<size_t>(p.grid) * G * 8;
  if (p.form == kRing) w.cpart = static_cast<size_t>(B) * G * ((p.splits + 1) & ~1) * 8;
  w.cpart = (w.cpart + 15) & ~size_t(15);
  w.total = w.cpart;
  if (bwd) {
    w.P = static_cast<int>(p.form == kStreamed ? p.grid
                           : p.form == kRing   ? static_cast<int64_t>(p.nsamp) * p.splits
                                               : B / p.cb);
    if (w.P > 1 || p.form == kRing) w.total += static_cast<size_t>(w.P) * C * 8;
  }
  return w;
}

GroupArgs group_args(const GroupPlan &p, int64_t B, int64_t S, int64_t C, int64_t G, int dt) {
  GroupArgs a;
  std::memset(&a, 0, sizeof a);
  a.B = static_cast<int>(B);
  a.S = static_cast<int>(S);
  a.C = static_cast<int>(C);
  a.G = static_cast<int>(G);
  a.D = static_cast<int>(C / G);
  a.nc = static_cast<int>(C / chunk_elems(dt));
  a.sg = p.sg;
  a.ncs = p.ncs;
  a.nslab = p.nslab;
  a.k = p.k;
  a.cb = p.cb;
  a.R = p.R;
  a.slots = p.slots;
  a.splits = p.splits;
  a.stages = p.stages;
  a.nsamp = p.nsamp;
  a.rounds = p.rounds;
  a.keep = p.keep;
  a.tm = p.tm;
  a.by_ncs.set(p.ncs);
  a.by_k.set(p.k);
  a.by_csize.set(p.k * p.cb);
  a.by_nslab.set(p.nslab);
  a.by_splits.set(p.splits);
  a.by_R.set(p.R);
  a.by_D.set(a.D);
  a.f_S.set(S);
  a.f_D.set(a.D);
  a.f_SD.set(S * a.D);
  const int ranges = p.form == kResident ? p.k : p.splits;
  a.pq = a.S / ranges;
  a.prem = a.S % ranges;
  a.f_rows.set(std::max(a.pq, 1));
  a.f_rows1.set(a.pq + 1);
  while ((p.sg << (a.lsh + 1)) <= p.threads && a.lsh < 5) ++a.lsh;
  return a;
}

norm_status_t run(int dev, int optin, const void *fn, const GroupPlan &p, uint32_t smem, int cluster,
                  GroupArgs &a, cudaStream_t s) {
  norm_status_t st = function_ready(dev, fn, optin);
  if (st != NORM_OK) return st;
  void *args[] = {&a};
  return launch_serial(fn, dim3(static_cast<unsigned>(p.grid)), dim3(p.threads), smem, cluster,
                       args, s);
}

norm_status_t run_ring(int dev, int optin, const GroupPlan &p, int dt, int act, bool drop, bool bwd,
                       unsigned *err, GroupArgs &a, cudaStream_t s) {
  const void *fn = group_ring_kernel_ptr(dt, act, drop, bwd);
  norm_status_t st = function_ready(dev, fn, optin);
  if (st != NORM_OK) return st;
  a.U = bwd ? kRingRowsBwd : kRingRowsFwd;
  a.err = err;
  void *args[] = {&a};
  return launch_cooperative(fn, dim3(static_cast<unsigned>(p.grid)), dim3(p.threads), p.smem, args,
                            s);
}

norm_status_t group_workspace(int64_t B, int64_t S, int64_t C, int64_t G, norm_dtype_t dtype,
                              bool bwd, size_t *bytes) {
  if (!bytes) return NORM_ERR_NULL;
  norm_status_t st = check_group(B, S, C, G, dtype);
  if (st != NORM_OK) return st;
  int dev = 0, sms = 0, optin = 0;
  unsigned *err = nullptr;
  if ((st = device_context(&dev, &sms, &optin, &err, nullptr)) != NORM_OK) return st;
  GroupPlan p;
  if ((st = group_plan(dev, sms, optin, B, S, C, G, dtype, bwd, &p)) != NORM_OK) return st;
  *bytes = group_ws(p, B, C, G, bwd).total;
  return NORM_OK;
}

}  // namespace
}  // namespace gbn

using namespace gbn;

extern "C" {

norm_status_t norm_group_fwd_workspace_bytes(int64_t B, int64_t S, int64_t C, int64_t groups,
                                             norm_dtype_t dtype, size_t *bytes) {
  return group_workspace(B, S, C, groups, dtype, false, bytes);
}

norm_status_t norm_group_bwd_workspace_bytes(int64_t B, int64_t S, int64_t C, int64_t groups,
                                             norm_dtype_t dtype, size_t *bytes) {
  return group_workspace(B, S, C, groups, dtype, true, bytes);
}

norm_status_t norm_group_fwd(const void *x, const void *gamma, const void *beta, int64_t B,
                             int64_t S, int64_t C, int64_t groups, float eps, norm_act_t act,
                             norm_dtype_t dtype, float p, uint64_t seed, uint64_t offset,
                             const void *offset_dev, void *y, float *rstd, float *mean,
                             void *workspace, size_t workspace_bytes, norm_stream_t stream) {
  if (!x || !gamma || !y || !rstd || !mean) return NORM_ERR_NULL;
  norm_status_t st = check_group(B, S, C, groups, dtype);
  if (st != NORM_OK) return st;
  if (act != NORM_ACT_NONE && act != NORM_ACT_SILU && act != NORM_ACT_GELU) return NORM_ERR_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return NORM_ERR_ARG;
  DropArgs drop;
  if ((st = make_drop(p, seed, offset, offset_dev, &drop)) != NORM_OK) return st;
  const void *ptrs[] = {x, gamma, beta, y, rstd, mean, workspace};
  for (const void *q : ptrs)
    if (q && !aligned_to_16(q)) return NORM_ERR_ALIGN;
  int dev = 0, sms = 0, optin = 0;
  unsigned *err = nullptr;
  if ((st = device_context(&dev, &sms, &optin, &err, nullptr)) != NORM_OK) return st;
  GroupPlan pl;
  if ((st = group_plan(dev, sms, optin, B, S, C, groups, dtype, false, &pl)) != NORM_OK) return st;
  const GroupWs w = group_ws(pl, B, C, groups, false);
  if (w.total && (!workspace || workspace_bytes < w.total)) return NORM_ERR_WORKSPACE;
  GroupArgs a = group_args(pl, B, S, C, groups, dtype);
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.out = y;
  a.mean = mean;
  a.rstd = rstd;
  a.gpart = static_cast<float *>(workspace);
  a.drop = drop;
  a.eps = eps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool dropping = drop.thr != 0;
  if (pl.form == kRing) return run_ring(dev, optin, pl, dtype, act, dropping, false, err, a, s);
  if (pl.form == kResident)
    return run(dev, optin, group_fwd_kernel_ptr(dtype, act, dropping), pl, pl.smem, pl.k, a, s);
  if ((st = run(dev, optin, group_stats_kernel_ptr(dtype), pl, pl.smem, 1, a, s)) != NORM_OK)
    return st;
  return run(dev, optin, group_apply_kernel_ptr(dtype, act, dropping), pl, pl.smem2, 1, a, s);
}

norm_status_t norm_group_bwd(const void *dy, const void *x, const void *gamma, const void *beta,
                             const float *rstd, const float *mean, int64_t B, int64_t S, int64_t C,
                             int64_t groups, norm_act_t act, norm_dtype_t dtype, float p,
                             uint64_t seed, uint64_t offset, const void *offset_dev, void *dx,
                             float *dgamma, float *dbeta, void *workspace, size_t workspace_bytes,
                             norm_stream_t stream) {
  if (!dy || !x || !gamma || !rstd || !mean || !dx || !dgamma) return NORM_ERR_NULL;
  norm_status_t st = check_group(B, S, C, groups, dtype);
  if (st != NORM_OK) return st;
  if (act != NORM_ACT_NONE && act != NORM_ACT_SILU && act != NORM_ACT_GELU) return NORM_ERR_ARG;
  DropArgs drop;
  if ((st = make_drop(p, seed, offset, offset_dev, &drop)) != NORM_OK) return st;
  const void *ptrs[] = {dy, x, gamma, beta, rstd, mean, dx, dgamma, dbeta, workspace};
  for (const void *q : ptrs)
    if (q && !aligned_to_16(q)) return NORM_ERR_ALIGN;
  int dev = 0, sms = 0, optin = 0;
  unsigned *err = nullptr;
  if ((st = device_context(&dev, &sms, &optin, &err, nullptr)) != NORM_OK) return st;
  GroupPlan pl;
  if ((st = group_plan(dev, sms, optin, B, S, C, groups, dtype, true, &pl)) != NORM_OK) return st;
  const GroupWs w = group_ws(pl, B, C, groups, true);
  if (w.total && (!workspace || workspace_bytes < w.total)) return NORM_ERR_WORKSPACE;
  GroupArgs a = group_args(pl, B, S, C, groups, dtype);
  a.x = x;
  a.dy = dy;
  a.gamma = gamma;
  a.beta = beta;
  a.out = dx;
  a.mean = const_cast<float *>(mean);
  a.rstd = const_cast<float *>(rstd);
  a.gpart = static_cast<float *>(workspace);
  a.drop = drop;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  float *rows = w.P > 1 || pl.form == kRing ? reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + w.cpart)
                        : nullptr;
  a.cpart = rows ? rows : dgamma;
  a.dbeta_part = !dbeta ? nullptr : rows ? rows + static_cast<size_t>(w.P) * C : dbeta;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool dropping = drop.thr != 0;
  if (pl.form == kRing) return run_ring(dev, optin, pl, dtype, act, dropping, true, err, a, s);
  if (pl.form == kResident) {
    st = run(dev, optin, group_bwd_kernel_ptr(dtype, act, dropping), pl, pl.smem, pl.k * pl.cb, a, s);
  } else {
    st = run(dev, optin, group_sums_kernel_ptr(dtype, act, dropping), pl, pl.smem, 1, a, s);
    if (st == NORM_OK)
      st = run(dev, optin, group_dx_kernel_ptr(dtype, act, dropping), pl, pl.smem2, 1, a, s);
  }
  if (st != NORM_OK || !rows) return st;
  return reduce_rows(rows, w.P, static_cast<int>(C), dgamma, dbeta, s);
}

norm_status_t norm_group_plan(int64_t B, int64_t S, int64_t C, int64_t groups, norm_dtype_t dtype,
                              int backward, int sm_count, int smem_optin_bytes,
                              norm_group_plan_t *out) {
  if (!out) return NORM_ERR_NULL;
  norm_status_t st = check_group(B, S, C, groups, dtype);
  if (st != NORM_OK) return st;
  if (backward & ~1) return NORM_ERR_ARG;
  GroupPlan p;
  if (sm_count > 0) {
    if (smem_optin_bytes <= 0) return NORM_ERR_ARG;
    st = make_group_plan(static_cast<int>(B), static_cast<int>(S), static_cast<int>(C),
                         static_cast<int>(groups), dtype, backward != 0, sm_count,
                         smem_optin_bytes, read_group_override(), &p);
  } else {
    int dev = 0, sms = 0, optin = 0;
    unsigned *err = nullptr;
    if ((st = device_context(&dev, &sms, &optin, &err, nullptr)) != NORM_OK) return st;
    st = group_plan(dev, sms, optin, B, S, C, groups, dtype, backward != 0, &p);
  }
  if (st != NORM_OK) return st;
  out->form = p.form;
  out->groups_per_slab = p.sg;
  out->slabs = p.nslab;
  out->chunk_columns = p.ncs;
  out->cluster = p.k;
  out->cluster_samples = p.cb;
  out->row_lanes = p.R;
  out->rows_per_thread = p.slots;
  out->row_splits = p.splits;
  out->stages = p.stages;
  out->tensor_memory_tiles = p.tm;
  out->samples_per_round = p.nsamp;
  out->rounds = p.rounds;
  out->threads = p.threads;
  out->smem_bytes = static_cast<int32_t>(p.smem);
  out->grid = static_cast<int32_t>(p.grid);
  out->workspace_bytes = static_cast<int64_t>(group_ws(p, B, C, groups, backward != 0).total);
  return NORM_OK;
}

}  // extern "C"
