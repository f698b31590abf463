// linear.cu -- entry points norm_linear_fwd / norm_linear_bwd: which kernels run
// a product, its tensor maps, workspaces and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdlib>
#include <cstring>
#include <tuple>
#include <utility>

#include "../../include/gbnorm.h"
#include "common.cuh"
#include "host_util.h"
#include "linear.cuh"
#include "plan_cache.h"
#include "tensor_map.h"

namespace gbn {

namespace {

// A 16-bit matrix of `rows` rows of `cols` elements, `ld` elements apart.
struct Matrix {
  const void *p;
  int64_t ld;
  int64_t rows, cols;
};

// Tensor copies take addresses and row strides that are multiples of 16 bytes.
bool tma_ready(const Matrix &t) {
  return aligned_to_16(t.p) && (t.rows == 1 || t.ld % 8 == 0);
}

norm_status_t map_of(CUtensorMap *m, const Matrix &t, bool bf16, uint32_t box_rows) {
  MapEncoder enc = nullptr;
  const norm_status_t st = map_encoder(&enc);
  if (st != NORM_OK) return st;
  const int64_t ld = t.rows == 1 ? (t.cols + 7) / 8 * 8 : t.ld;
  cuuint64_t dims[2] = {cuuint64_t(t.cols), cuuint64_t(t.rows)};
  cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
  cuuint32_t box[2] = {kLinBK, box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r =
      enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
          const_cast<void *>(t.p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? NORM_OK : NORM_ERR_CUDA;
}

struct Device {
  int dev = 0, sms = 0, optin = 0;
  unsigned *err = nullptr;
};

// How a product runs.
struct ProductPlan {
  bool pair = false;
  int bn = 0;      // tile columns (pair), or tokens per tile (split)
  int splits = 1;  // the split form
  int stages = 0;
  double time = 1e30;  // estimate, us
};

int round_up(int64_t v, int to) { return static_cast<int>((v + to - 1) / to * to); }

// As many stages as there are K blocks, or as leave room for two CTAs per SM
// where that makes four; the ring also takes the partial sums of all tokens.
int split_stages(int nk, int bn, int splits, int optin) {
  const int nkb = (nk + splits - 1) / splits;
  const uint32_t sb = split_stage_bytes(bn), fixed = split_smem(bn, splits, 0);
  int most = static_cast<int>((uint32_t(optin) / 2 - 1024 - fixed) / sb);
  if (most < 4) most = static_cast<int>((uint32_t(optin) - fixed) / sb);
  if (most > kSplitMaxStages) most = kSplitMaxStages;
  int stages = nkb < most ? nkb : most;
  const int least = static_cast<int>((uint32_t(bn) * 512u + sb - 1) / sb);
  if (!split_push(bn, splits) && stages < least) stages = least;
  return stages;
}

uint32_t tmem_columns(int bn) {
  uint32_t c = 32;
  while (c < uint32_t(bn)) c *= 2;
  return c;
}

constexpr size_t kMaxPlans = 4096;

// clusters resident at once, by kernel, cluster size and device, shared memory
PlanCache<std::tuple<const void *, int, uint32_t>, int> g_resident(kMaxPlans);

// Clusters of `cluster` CTAs of kernel fn that are resident at once.
norm_status_t resident(const Device &d, const void *fn, int threads, int cluster, uint32_t smem,
                       int *out) {
  const auto key = std::make_tuple(fn, cluster * 64 + d.dev, smem);
  if (!g_resident.find(key, out)) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = unsigned(cluster);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(unsigned(cluster) * 1024u);
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return NORM_ERR_CUDA;
    }
    g_resident.keep(key, n);
    *out = n;
  }
  return *out < 1 ? NORM_ERR_UNSUPPORTED : NORM_OK;
}

// Estimated microseconds of the two forms.  The constants were fitted to 830
// measured (form, size) pairs of 52 sizes (1 to 16384 rows, forward and both
// gradients, operands not in L2); on these sizes the form of least estimate is
// 3 % slower than the fastest measured one in the geometric mean, 28 % at worst.
// No size was held back; with best_form's limits it is 1.6 % and 10 % on 47 more,
// and 13 % for 512 x 4096 x 16384 (50.0 us, with tiles of 256 44.4).
double pair_time(int64_t m, int64_t n, int nk, int bn, bool b_mn, int pairs) {
  const int64_t tiles = ((m + 255) / 256) * ((n + bn - 1) / bn);
  const double waves = double((tiles + pairs - 1) / pairs);
  double kb = 0.0289 + 0.001076 * bn;         // per K block: the MMAs
  if (b_mn && kb < 0.2157) kb = 0.2157;       // whole 128-column boxes to load
  const double epi = 1.2 + 0.0033 * bn;  // per tile, beside the next tile's MMAs
  const double main = nk * kb;
  const double mem = 2.0 * (double(m + n) * nk * kLinBK + double(m) * n) / 3.54e6;
  const double work = waves * (main > epi ? main : epi);
  return 3.2 + epi + (work > mem ? work : mem);
}

double split_time(int64_t m, int64_t n, int nk, int bn, int splits, int stages, int clusters,
                  int sms) {
  const int64_t tiles = ((m + bn - 1) / bn) * ((n + 127) / 128);
  const int nkb = (nk + splits - 1) / splits;
  const double stage = split_stage_bytes(bn);
  const double rate = stage / 134600.0 > 0.00196 * bn ? stage / 134600.0 : 0.00196 * bn;
  const auto wave = [&](int64_t c) {  // c clusters side by side
    if (c == 0) return 0.0;
    const double per_sm = double(c) * splits > sms ? double(c) * splits / sms : 1.0;
    double kb = per_sm * rate;              // an SM's bytes or MMAs
    if (kb < 0.053 / stages) kb = 0.053 / stages;
    if (kb < 0.2) kb = 0.2;  // one CTA's turn
    return nkb * kb + 0.0251 * bn / splits * per_sm + 3.51;
  };
  const double work = double(tiles / clusters) * wave(clusters) + wave(tiles % clusters);
  const double mem = 2.0 * (double(m + n) * nk * kLinBK + double(m) * n) / 5.13e6;
  const double join = splits == 1 ? 0.0 : split_push(bn, splits) ? 0.016 : 2.56;
  const double odd = splits == 8 ? 0.5 : splits == 6 ? 0.4 : splits == 3 ? 0.2 : 0.1 * (splits == 2);
  return (work > mem ? work : mem) + join + odd;
}

// The split form with clusters of s CTAs (s <= nk): its tile width and estimate.
norm_status_t split_form(const Device &d, const void *fn, int64_t m, int64_t n, int nk, bool a_mn,
                         int s, int want_bn, ProductPlan *best) {
  const int unit = a_mn ? 64 : 16;
  const int whole = m <= 128 ? round_up(m, unit) : 128;
  *best = ProductPlan{};
  for (int bn : {whole, 64}) {
    if (want_bn >= unit && want_bn <= 256 && want_bn % unit == 0) bn = want_bn;
    const int stages = split_stages(nk, bn, s, d.optin);
    int clusters = 0;
    const norm_status_t st =
        resident(d, fn, kSplitThreads, s, split_smem(bn, s, stages), &clusters);
    if (st != NORM_OK) return st;
    const int tm = d.sms * (512 / int(tmem_columns(bn))) / s;  // tensor memory's limit
    const double t = split_time(m, n, nk, bn, s, stages, clusters < tm ? clusters : tm, d.sms);
    if (t < best->time) *best = ProductPlan{false, bn, s, stages, t};
  }
  return NORM_OK;
}

// The split form is for few rows, and as long as its tiles are two waves or so.
bool split_size(int64_t m, int64_t n) { return m <= 192 || m * n <= int64_t(4096) * 4096; }

// GBNORM_LINEAR="pair=0,bn=64,splits=4,joint=0" forces fields (for sweeps): the form,
// tile width and cluster size, where a product can have them, and whether both
// gradients' products go into one launch.
struct LinForce {
  bool any = false;
  int pair = -1, joint = -1, bn = 0, splits = 0;
};

LinForce read_force() {
  LinForce f;
  if (const char *o = std::getenv("GBNORM_LINEAR")) {
    f.any = true;
    if (const char *q = std::strstr(o, "pair=")) f.pair = std::atoi(q + 5) != 0;
    if (const char *q = std::strstr(o, "joint=")) f.joint = std::atoi(q + 6) != 0;
    if (const char *q = std::strstr(o, "bn=")) f.bn = std::atoi(q + 3);
    if (const char *q = std::strstr(o, "splits=")) f.splits = std::atoi(q + 7);
    if (f.splits < 1 || f.splits > 8) f.splits = 0;
  }
  return f;
}

// The form of least estimate.
norm_status_t best_form(const Device &d, int64_t m, int64_t n, int64_t k, bool a_mn, bool b_mn,
                        bool bf16, const LinForce &f, ProductPlan *best) {
  const int nk = static_cast<int>((k + kLinBK - 1) / kLinBK);
  norm_status_t st;
  *best = ProductPlan{};
  const void *pair = linear_pair_kernel_ptr(a_mn, b_mn, bf16);
  const void *split = linear_split_kernel_ptr(!a_mn && !b_mn, bf16);
  if ((st = function_ready(d.dev, pair, d.optin)) != NORM_OK) return st;
  if ((st = function_ready(d.dev, split, d.optin)) != NORM_OK) return st;
  int pairs = 0;
  if ((st = resident(d, pair, kPairThreads, 2, pair_smem(), &pairs)) != NORM_OK) return st;
  const int64_t high = (m + 255) / 256;  // tiles of 256 rows
  if (f.pair != 0 && (f.pair == 1 || m > 192)) {
    // Tiles of 64 for what does not fill the GPU otherwise: operands cross L2 twice
    // as often as for 128 (256 x 4096 x 4096 14.1 us and 15.5, 2048 x 1024 x 4096
    // 22.8 and 17.7), and a K block of an MN-major B loads as long.
    const bool few = !b_mn && high * ((n + 63) / 64) <= pairs;
    for (int bn : {64, 128, 192, 224, 256}) {
      if (bn == 64 && !few && f.pair != 1) continue;
      if (f.pair == 1 && f.bn >= 64 && f.bn <= 256 && f.bn % 32 == 0) bn = f.bn;
      const double t = pair_time(m, n, nk, bn, b_mn, pairs);
      if (t < best->time) *best = ProductPlan{true, bn, 1, 0, t};
    }
  }
  // With many rows the split form is for products that leave many SMs to it: with
  // 40 tiles of 256 x 128 (777 x 1232 x 1000) it takes 8.6 us where pairs take 10.0,
  // with 64 (8192 x 256 x 1024) 11.4 and 9.1.
  const bool gaps = m <= 192 || high * ((n + 127) / 128) * 3 <= int64_t(pairs) * 2;
  if (f.pair != 1 && (f.pair == 0 || (split_size(m, n) && gaps))) {
    for (int s : {1, 2, 3, 4, 6, 8}) {
      if (f.pair == 0 && f.splits) s = f.splits;
      if (s > nk) s = nk;
      ProductPlan p;
      st = split_form(d, split, m, n, nk, a_mn, s, f.pair == 0 ? f.bn : 0, &p);
      if (st != NORM_OK) return st;
      if (p.time < best->time) *best = p;
    }
  }
  return NORM_OK;
}

// Plans of sizes seen before, per device, storage of the operands and type.
PlanCache<std::tuple<int, int64_t, int64_t, int64_t>, ProductPlan> g_plans(kMaxPlans);

norm_status_t plan_product(const Device &d, int64_t m, int64_t n, int64_t k, bool a_mn, bool b_mn,
                           bool bf16, ProductPlan *out) {
  const LinForce force = read_force();
  const auto key = std::make_tuple(d.dev * 8 + a_mn * 4 + b_mn * 2 + bf16, m, n, k);
  if (!force.any && g_plans.find(key, out)) return NORM_OK;
  ProductPlan p;
  const norm_status_t st = best_form(d, m, n, k, a_mn, b_mn, bf16, force, &p);
  if (st != NORM_OK) return st;
  if (!force.any) g_plans.keep(key, p);
  *out = p;
  return NORM_OK;
}

// A launch of the split form: one or two products, and a sum of rows behind them.
struct SplitLaunch {
  SplitMaps maps = {};
  SplitArgs args = {};
  uint32_t smem = 0;
  int count = 0;

  SplitLaunch(const Device &d, int splits) {
    args.splits = splits;
    args.tmem = 32;
    args.err = d.err;
  }
  norm_status_t add(const Matrix &a, bool a_mn, const Matrix &b, bool b_mn, int64_t m, int64_t n,
                    int nk, const ProductPlan &plan, const LinEpilogue &e, bool bf16) {
    norm_status_t st;
    if ((st = map_of(&maps.a[count], a, bf16, a_mn ? kLinBK : uint32_t(plan.bn))) != NORM_OK)
      return st;
    if ((st = map_of(&maps.b[count], b, bf16, b_mn ? kLinBK : 128)) != NORM_OK) return st;
    SplitProblem &p = args.q[count++];
    p.e = e;
    p.m = static_cast<int>(m);
    p.n = static_cast<int>(n);
    p.nk = nk;
    p.bn = plan.bn;
    p.stages = plan.stages;
    p.tiles_j = static_cast<int>((m + plan.bn - 1) / plan.bn);
    const int64_t clusters = int64_t(p.tiles_j) * ((n + 127) / 128);
    if (clusters * args.splits > 0x3fffffff) return NORM_ERR_UNSUPPORTED;
    p.clusters = static_cast<int>(clusters);
    p.a_mn = a_mn;
    p.b_mn = b_mn;
    p.vec = 1;
    const Matrix rows[4] = {{e.y, e.ldy, m, n}, {e.z, e.ldz, m, n}, {e.r, e.ldr, m, n},
                            {e.bias, 0, 1, n}};
    for (const Matrix &t : rows)
      if (reinterpret_cast<uintptr_t>(t.p) % 8 || (t.rows > 1 && t.p && t.ld % 4)) p.vec = 0;
    if (tmem_columns(p.bn) > args.tmem) args.tmem = tmem_columns(p.bn);
    const uint32_t need = split_smem(p.bn, args.splits, p.stages);
    if (need > smem) smem = need;
    return NORM_OK;
  }
  norm_status_t go(const Device &d, bool bf16, cudaStream_t s) {
    const bool fwd = count == 1 && !args.part && !args.q[0].a_mn && !args.q[0].b_mn;
    const void *fn = linear_split_kernel_ptr(fwd, bf16);
    if (d.optin < int(smem)) return NORM_ERR_UNSUPPORTED;
    norm_status_t st = function_ready(d.dev, fn, d.optin);
    if (st != NORM_OK) return st;
    int64_t clusters = int64_t(args.q[0].clusters) + args.q[1].clusters;
    if (args.part)
      clusters += (args.cols + kSplitThreads * args.splits - 1) / (kSplitThreads * args.splits);
    void *a[] = {&maps, &args};
    return launch_serial(fn, dim3(unsigned(clusters * args.splits)), dim3(kSplitThreads), smem,
                         args.splits, a, s);
  }
};

// out[j, i] = epilogue(sum_k A[j, k] B[i, k]); A and B are addressable by tensor
// copies, stored [m or n, k], or [k, m or n] where a_mn / b_mn.
norm_status_t product(const Device &d, const Matrix &a, bool a_mn, const Matrix &b, bool b_mn,
                      int64_t m, int64_t n, int64_t k, const LinEpilogue &e, bool bf16,
                      cudaStream_t s) {
  ProductPlan plan;
  norm_status_t st = plan_product(d, m, n, k, a_mn, b_mn, bf16, &plan);
  if (st != NORM_OK) return st;
  const int nk = static_cast<int>((k + kLinBK - 1) / kLinBK);
  CUtensorMap ta, tb;
  if (plan.pair) {
    const void *fn = linear_pair_kernel_ptr(a_mn, b_mn, bf16);
    if (d.optin < int(pair_smem())) return NORM_ERR_UNSUPPORTED;
    if ((st = function_ready(d.dev, fn, d.optin)) != NORM_OK) return st;
    int pairs = 0;
    if ((st = resident(d, fn, kPairThreads, 2, pair_smem(), &pairs)) != NORM_OK) return st;
    if ((st = map_of(&ta, a, bf16, a_mn ? kLinBK : 128)) != NORM_OK) return st;
    if ((st = map_of(&tb, b, bf16, b_mn ? kLinBK : uint32_t(plan.bn / 2))) != NORM_OK) return st;
    PairArgs p = {};
    p.e = e;
    p.m = static_cast<int>(m);
    p.n = static_cast<int>(n);
    p.nk = nk;
    p.bn = plan.bn;
    // (with many K blocks a residual tile that is loaded when its slice begins is
    // in time, and the room goes to the operands)
    p.bufs = e.z || (e.r && nk < 32) ? 4 : 2;
    p.stages = pair_stages(p.bn, b_mn, p.bufs);
    p.sets = p.bufs / 2 / (e.z ? 2 : 1);
    p.gm = 8;
    p.err = d.err;
    CUtensorMap ty = ta, tz = ta, tr = ta;
    const Matrix out[3] = {{e.y, e.ldy, m, n}, {e.z, e.ldz, m, n}, {e.r, e.ldr, m, n}};
    CUtensorMap *maps[3] = {&ty, &tz, &tr};
    int *flags[3] = {&p.tma_y, &p.tma_z, &p.tma_r};
    for (int i = 0; i < 3; ++i) {
      if (!out[i].p || !tma_ready(out[i])) continue;
      if ((st = check_device_memory(out[i].p, d.dev)) != NORM_OK) return st;
      if ((st = map_of(maps[i], out[i], bf16, 32)) != NORM_OK) return st;
      *flags[i] = 1;
    }
    const int64_t tiles = ((m + 255) / 256) * ((n + plan.bn - 1) / plan.bn);
    const int64_t grid = 2 * (tiles < pairs ? tiles : pairs);
    void *args[] = {&ta, &tb, &ty, &tz, &tr, &p};
    return launch_serial(fn, dim3(unsigned(grid)), dim3(kPairThreads), pair_smem(), 2, args, s);
  }
  SplitLaunch l(d, plan.splits);
  if ((st = l.add(a, a_mn, b, b_mn, m, n, nk, plan, e, bf16)) != NORM_OK) return st;
  return l.go(d, bf16, s);
}

// Whether both gradients' products of a layer go into one launch of the split
// form, and their plans there, with clusters of the same size.  Each product
// alone takes 3 us or so from the launch to the first byte and from the last, and
// fills part of the GPU: 531 x 648 x 1001 with the bias takes 11 us in one launch
// where it took 19 in three, 1024 x 1024 x 1024 13 in place of 19.
struct JointPlan {
  bool joint = false;
  ProductPlan dx, dw;
};
PlanCache<std::tuple<int, int64_t, int64_t, int64_t>, JointPlan> g_joint(kMaxPlans);

norm_status_t plan_joint(const Device &d, int64_t M, int64_t N, int64_t K, bool bf16, JointPlan *out) {
  const LinForce force = read_force();
  const auto key = std::make_tuple(d.dev * 2 + bf16, M, N, K);
  if (!force.any && g_joint.find(key, out)) return NORM_OK;
  JointPlan j;
  norm_status_t st;
  ProductPlan one[2];
  if ((st = plan_product(d, M, K, N, false, true, bf16, &one[0])) != NORM_OK) return st;
  if ((st = plan_product(d, N, K, M, true, true, bf16, &one[1])) != NORM_OK) return st;
  const bool open = force.joint >= 0 ? force.joint == 1
                                     : force.any ? !one[0].pair : split_size(M, K) && split_size(N, K);
  if (open) {
    const int nk = static_cast<int>((N + kLinBK - 1) / kLinBK);
    const int mk = static_cast<int>((M + kLinBK - 1) / kLinBK);
    const void *fn = linear_split_kernel_ptr(false, bf16);
    double best = force.any ? 1e30 : one[0].time + one[1].time;
    for (int s : {1, 2, 3, 4, 6, 8}) {
      if (force.splits) s = force.splits < nk && force.splits < mk ? force.splits : nk < mk ? nk : mk;
      if (s > nk || s > mk) break;
      ProductPlan p[2];
      if ((st = split_form(d, fn, M, K, nk, false, s, force.bn, &p[0])) != NORM_OK) return st;
      if ((st = split_form(d, fn, N, K, mk, true, s, force.bn, &p[1])) != NORM_OK) return st;
      const double t = p[0].time + p[1].time - 4.0;  // one start for two
      if (t < best) {
        best = t;
        j = JointPlan{true, p[0], p[1]};
      }
    }
  }
  if (!force.any) g_joint.keep(key, j);
  *out = j;
  return NORM_OK;
}

// Copies of operands in a workspace: whole multiples of 256 bytes.
size_t packed_bytes(const Matrix &t) {
  return (size_t(t.rows) * size_t(round_up(t.cols, 8)) * 2 + 255) & ~size_t(255);
}

// Copies those of the matrices that are not null and not addressable, in one
// launch, and has them point to the copies.
norm_status_t pack(Matrix *t0, Matrix *t1, char **ws, cudaStream_t s) {
  PackArgs a = {};
  int n = 0, most = 0;
  bool two = true;
  for (const Matrix *t : {t0, t1})
    if (t && !tma_ready(*t) &&
        (reinterpret_cast<uintptr_t>(t->p) % 4 || t->cols % 2 || (t->rows > 1 && t->ld % 2)))
      two = false;
  for (Matrix *t : {t0, t1}) {
    if (!t || tma_ready(*t)) continue;
    a.src[n] = static_cast<const uint16_t *>(t->p);
    a.dst[n] = reinterpret_cast<uint16_t *>(*ws);
    a.ld[n] = t->ld;
    a.ldd[n] = round_up(t->cols, 8);
    a.rows[n] = static_cast<int>(t->rows);
    a.cols[n] = static_cast<int>(t->cols);
    a.strips[n] = (a.cols[n] / (two ? 2 : 1) + 255) / 256;
    if (a.rows[n] > most) most = a.rows[n];
    *ws += packed_bytes(*t);
    t->p = a.dst[n];
    t->ld = a.ldd[n];
    ++n;
  }
  if (n == 0) return NORM_OK;
  const int gy = (most + 7) / 8 < 65535 ? (most + 7) / 8 : 65535;
  void *args[] = {&a};
  return launch_serial(linear_pack_kernel_ptr(two), dim3(unsigned(a.strips[0] + a.strips[1]), unsigned(gy)),
                       dim3(256), 0, 1, args, s);
}

norm_status_t check_shape(int64_t M, int64_t K, int64_t N) {
  const int64_t wide = int64_t(1) << 20;
  if (M < 1 || M > (int64_t(1) << 24) || K < 1 || K > wide || N < 1 || N > wide)
    return NORM_ERR_SHAPE;
  return NORM_OK;
}

norm_status_t check_matrix(const Matrix &t) {
  if (t.rows > 1 && (t.ld < t.cols || t.ld > (int64_t(1) << 32))) return NORM_ERR_SHAPE;
  return reinterpret_cast<uintptr_t>(t.p) % 2 ? NORM_ERR_ALIGN : NORM_OK;
}

bool known_act(int act) {
  return act == NORM_ACT_NONE || act == NORM_ACT_SILU || act == NORM_ACT_GELU;
}

// Row chunks of the gradient pass: enough CTAs to fill the GPU a few times, and
// 32 rows or more in each.
int grad_chunks(int64_t M, int64_t N, bool vec, int sms) {
  const int64_t strips = (N + (vec ? 255 : 31)) / (vec ? 256 : 32);
  int64_t c = (int64_t(sms) * 8 + strips - 1) / strips;
  if (c > (M + 31) / 32) c = (M + 31) / 32;
  if (c > 65535) c = 65535;
  return static_cast<int>(c < 1 ? 1 : c);
}

// The parts of a backward workspace.
struct GradPlan {
  bool need_dz, vec;
  int chunks;
  size_t dz, part, x, w;
  size_t total() const { return dz + part + x + w; }
};

// What a backward call reads: x, w and z as null matrices where they are not needed.
struct GradIn {
  Matrix dy, x, w, z;
};

norm_status_t grad_in(GradIn *in, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                      const void *w, int64_t ldw, const void *z, int64_t ldz, int64_t M, int64_t K,
                      int64_t N, int act, bool dx, bool dw) {
  if (act == NORM_ACT_NONE) z = nullptr;
  *in = {{dy, lddy, M, N},
         {dw ? x : nullptr, dw ? ldx : K, M, K},
         {dx ? w : nullptr, dx ? ldw : K, N, K},
         {z, z ? ldz : N, M, N}};
  for (const Matrix &t : {in->dy, in->x, in->w, in->z}) {
    const norm_status_t st = check_matrix(t);
    if (st != NORM_OK) return st;
  }
  return NORM_OK;
}

GradPlan grad_plan(const GradIn &in, int act, bool dx, bool dw, bool dbias, int sms) {
  const Matrix &dy = in.dy, &x = in.x, &w = in.w, &z = in.z;
  GradPlan g = {};
  const bool products = dx || dw;
  g.need_dz = products && (act != NORM_ACT_NONE || !tma_ready(dy));
  g.vec = dy.cols % 8 == 0 && tma_ready(dy) && (act == NORM_ACT_NONE || tma_ready(z));
  g.chunks = grad_chunks(dy.rows, dy.cols, g.vec, sms);
  if (g.need_dz) g.dz = packed_bytes(dy);
  if (dbias) g.part = (size_t(g.chunks) * size_t(dy.cols) * 4 + 255) & ~size_t(255);
  if (dw && !tma_ready(x)) g.x = packed_bytes(x);
  if (dx && !tma_ready(w)) g.w = packed_bytes(w);
  return g;
}

norm_status_t device_of(Device *d) {
  return device_context(&d->dev, &d->sms, &d->optin, &d->err, nullptr);
}

}  // namespace

}  // namespace gbn

using namespace gbn;

extern "C" {

norm_status_t norm_linear_fwd_workspace_bytes(const void *x, int64_t ldx, const void *w,
                                              int64_t ldw, int64_t M, int64_t K, int64_t N,
                                              size_t *bytes) {
  if (!bytes || !x || !w) return NORM_ERR_NULL;
  norm_status_t st = check_shape(M, K, N);
  if (st != NORM_OK) return st;
  *bytes = 0;
  for (const Matrix &t : {Matrix{x, ldx, M, K}, Matrix{w, ldw, N, K}}) {
    if ((st = check_matrix(t)) != NORM_OK) return st;
    if (!tma_ready(t)) *bytes += packed_bytes(t);
  }
  return NORM_OK;
}

norm_status_t norm_linear_fwd(const void *x, int64_t ldx, const void *w, int64_t ldw,
                              const void *bias, const void *r, int64_t ldr, int64_t M, int64_t K,
                              int64_t N, norm_act_t act, norm_dtype_t dtype, void *y, int64_t ldy,
                              void *z, int64_t ldz, void *workspace, size_t workspace_bytes,
                              norm_stream_t stream) {
  if (!x || !w || !y) return NORM_ERR_NULL;
  norm_status_t st = check_shape(M, K, N);
  if (st != NORM_OK) return st;
  if (!known_act(act) || (dtype != NORM_BF16 && dtype != NORM_FP16)) return NORM_ERR_ARG;
  Matrix mx{x, ldx, M, K}, mw{w, ldw, N, K};
  for (const Matrix &t : {mx, mw, Matrix{y, ldy, M, N}, Matrix{z, z ? ldz : N, M, N},
                          Matrix{r, r ? ldr : N, M, N}, Matrix{bias, N, 1, N}})
    if ((st = check_matrix(t)) != NORM_OK) return st;
  size_t need = 0;
  if ((st = norm_linear_fwd_workspace_bytes(x, ldx, w, ldw, M, K, N, &need)) != NORM_OK) return st;
  if (need && (!workspace || workspace_bytes < need)) return NORM_ERR_WORKSPACE;
  if (need && !aligned_to_16(workspace)) return NORM_ERR_ALIGN;
  Device d;
  if ((st = device_of(&d)) != NORM_OK) return st;
  for (const void *p : {x, w})
    if ((st = check_device_memory(p, d.dev)) != NORM_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  if ((st = pack(&mx, &mw, &ws, s)) != NORM_OK) return st;
  const LinEpilogue e = {bias, r, z, y, ldr, ldz, ldy, int(act)};
  return product(d, mx, false, mw, false, M, N, K, e, dtype == NORM_BF16, s);
}

norm_status_t norm_linear_bwd_workspace_bytes(const void *dy, int64_t lddy, const void *x,
                                              int64_t ldx, const void *w, int64_t ldw,
                                              const void *z, int64_t ldz, int64_t M, int64_t K,
                                              int64_t N, norm_act_t act, int want_dx, int want_dw,
                                              int want_dbias, size_t *bytes) {
  if (!bytes || !dy) return NORM_ERR_NULL;
  if ((want_dw && !x) || (want_dx && !w)) return NORM_ERR_NULL;
  norm_status_t st = check_shape(M, K, N);
  if (st != NORM_OK) return st;
  if (!known_act(act)) return NORM_ERR_ARG;
  if (act != NORM_ACT_NONE && !z) return NORM_ERR_NULL;
  GradIn in;
  if ((st = grad_in(&in, dy, lddy, x, ldx, w, ldw, z, ldz, M, K, N, act, want_dx, want_dw)) !=
      NORM_OK)
    return st;
  Device d;
  if ((st = device_of(&d)) != NORM_OK) return st;
  *bytes = grad_plan(in, act, want_dx, want_dw, want_dbias, d.sms).total();
  return NORM_OK;
}

norm_status_t norm_linear_bwd(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                              const void *w, int64_t ldw, const void *z, int64_t ldz, int64_t M,
                              int64_t K, int64_t N, norm_act_t act, norm_dtype_t dtype, void *dx,
                              int64_t lddx, void *dw, int64_t lddw, float *dbias, void *workspace,
                              size_t workspace_bytes, norm_stream_t stream) {
  if (!dy) return NORM_ERR_NULL;
  if ((dw && !x) || (dx && !w)) return NORM_ERR_NULL;
  norm_status_t st = check_shape(M, K, N);
  if (st != NORM_OK) return st;
  if (!known_act(act) || (dtype != NORM_BF16 && dtype != NORM_FP16)) return NORM_ERR_ARG;
  if (!dx && !dw && !dbias) return NORM_ERR_ARG;
  if (act != NORM_ACT_NONE && !z) return NORM_ERR_NULL;
  GradIn in;
  if ((st = grad_in(&in, dy, lddy, x, ldx, w, ldw, z, ldz, M, K, N, act, dx, dw)) != NORM_OK)
    return st;
  for (const Matrix &t : {Matrix{dx, dx ? lddx : K, M, K}, Matrix{dw, dw ? lddw : K, N, K}})
    if ((st = check_matrix(t)) != NORM_OK) return st;
  if (reinterpret_cast<uintptr_t>(dbias) % 4) return NORM_ERR_ALIGN;
  Device d;
  if ((st = device_of(&d)) != NORM_OK) return st;
  const GradPlan g = grad_plan(in, act, dx, dw, dbias, d.sms);
  if (g.total() && (!workspace || workspace_bytes < g.total())) return NORM_ERR_WORKSPACE;
  if (g.total() && !aligned_to_16(workspace)) return NORM_ERR_ALIGN;
  for (const void *p : {dy, in.x.p, in.w.p})
    if (p && (st = check_device_memory(p, d.dev)) != NORM_OK) return st;
  const bool bf16 = dtype == NORM_BF16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  Matrix mdz = in.dy, mx = in.x, mw = in.w;
  const float *part = nullptr;
  if (g.need_dz || dbias) {
    GradArgs a = {};
    a.dy = dy;
    a.z = in.z.p;
    a.lddy = lddy;
    a.ldz = ldz;
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.chunks = g.chunks;
    a.act = act;
    if (g.need_dz) {
      a.dz = ws;
      a.lddz = round_up(N, 8);
      ws += g.dz;
      mdz.p = a.dz;
      mdz.ld = a.lddz;
    }
    if (dbias) {
      part = a.part = reinterpret_cast<float *>(ws);
      ws += g.part;
    }
    void *args[] = {&a};
    const int64_t strips = (N + (g.vec ? 255 : 31)) / (g.vec ? 256 : 32);
    st = launch_serial(linear_grad_kernel_ptr(bf16, g.vec), dim3(unsigned(strips), unsigned(g.chunks)),
                       dim3(kGradThreads), 0, 1, args, s);
    if (st != NORM_OK) return st;
  }
  if ((st = pack(dx ? &mw : nullptr, dw ? &mx : nullptr, &ws, s)) != NORM_OK) return st;
  const LinEpilogue ex = {nullptr, nullptr, nullptr, dx, 0, 0, lddx, kLinNone};
  const LinEpilogue ew = {nullptr, nullptr, nullptr, dw, 0, 0, lddw, kLinNone};
  if (dx && dw) {  // one launch for both, and the sum, where both are small
    JointPlan plan;
    if ((st = plan_joint(d, M, N, K, bf16, &plan)) != NORM_OK) return st;
    if (plan.joint) {
      SplitLaunch l(d, plan.dx.splits);
      const int nk = static_cast<int>((N + kLinBK - 1) / kLinBK);
      const int mk = static_cast<int>((M + kLinBK - 1) / kLinBK);
      if ((st = l.add(mdz, false, mw, true, M, K, nk, plan.dx, ex, bf16)) != NORM_OK) return st;
      if ((st = l.add(mdz, true, mx, true, N, K, mk, plan.dw, ew, bf16)) != NORM_OK) return st;
      l.args.part = part;
      l.args.sums = dbias;
      l.args.rows = g.chunks;
      l.args.cols = static_cast<int>(N);
      return l.go(d, bf16, s);
    }
  }
  if (dx && (st = product(d, mdz, false, mw, true, M, K, N, ex, bf16, s)) != NORM_OK) return st;
  if (dw && (st = product(d, mdz, true, mx, true, N, K, M, ew, bf16, s)) != NORM_OK) return st;
  if (dbias) {
    int n = static_cast<int>(N), rows = g.chunks;
    void *fold[] = {&part, &n, &rows, &dbias};
    st = launch_serial(linear_fold_kernel_ptr(), dim3(unsigned((n + 31) / 32)), dim3(1024), 0, 1,
                       fold, s);
  }
  return st;
}

}  // extern "C"
