// Group norm with an activation: C entry points, argument checks and launch
// plan.
#include <math.h>

#include "../../include/normfuse.h"
#include "gn_kernels.cuh"
#include "launch.h"
#include "validate.h"

namespace nf {

const void* gn_table_f32(bool bwd, bool cluster, bool fine, int act);
const void* gn_table_bf16(bool bwd, bool cluster, bool fine, int act);
const void* gn_table_f16(bool bwd, bool cluster, bool fine, int act);

namespace {

ln_status cuda_fail(cudaError_t e) {
  nf_set_last_cuda_error((int)e);
  return LN_ERR_CUDA;
}

int gcd(int a, int b) {
  while (b) {
    const int t = a % b;
    a = b;
    b = t;
  }
  return a;
}

// How a call is cut up: column tiles, slices of the rows and, where it takes
// more than one launch, batches of panels (a panel is one sample's column
// tile).
struct GnPlan {
  bool cluster;            // one launch, a cluster a panel
  int clusters;            // of the launch
  int tiles, tile_ch, tw, max_groups, slices;
  int64_t slice_rows;
  int64_t panels, batch;   // all panels, and those of one launch
  size_t part_bytes, cols_bytes;
  size_t bytes() const { return part_bytes + cols_bytes; }
};

constexpr int kGnMaxVecs = 64;                 // most vectors of a tile
constexpr int kPerSm[2] = {3, 2};            // resident CTAs, forward and backward
constexpr int64_t kBatchBytes[2] = {68ll << 20, 90ll << 20};
constexpr int64_t kSlabBytes = 2ll << 20;

// Column tiles of about `bytes`: of whole groups that start on the rows'
// alignment, in units of `unit` channels, where a tile can be that wide; false
// when a tile may end inside a group.
bool gn_tiles(int channels, int unit, int bytes, int es, GnPlan* p) {
  const int V = 16 / es, most = kGnMaxVecs * V;
  int target = bytes / es;
  if (target > most) target = most;
  int ch = channels;
  bool whole = channels <= most;
  if (channels > target) {
    if (unit <= most) {
      whole = true;
      const int units = (channels + unit - 1) / unit;
      int per = (target + unit - 1) / unit;
      if (per * unit > most) per = most / unit;
      if (per > units) per = units;
      const int t = (units + per - 1) / per;
      ch = (units + t - 1) / t * unit;
      if (ch > channels) ch = channels;
    } else if (!whole) {
      const int t = (channels + target - 1) / target;
      ch = ((channels + t - 1) / t + V - 1) / V * V;
    }
  }
  p->tile_ch = ch;
  p->tw = (ch + V - 1) / V;
  p->tiles = (channels + ch - 1) / ch;
  return whole;
}

bool gn_plan(int64_t samples, int64_t rows, int channels, int groups, size_t elem, bool bwd,
             int grain, int sms, int most_cluster, GnPlan* p) {
  const int es = (int)elem, cpg = channels / groups;
  const int unit = cpg * (grain / gcd(cpg * es, grain));
  const int64_t places = (int64_t)sms * kPerSm[bwd];
  const auto max_groups = [&](bool whole) {
    const int tc = p->tile_ch;
    const int m = whole ? (tc + cpg - 1) / cpg : (tc - 2 > 0 ? (tc - 2) / cpg : 0) + 2;
    return m < groups ? m : groups;
  };
  // Forward: one launch, a cluster a panel, where a thread's rows all stay in
  // its slots (4 x 205 x 192 bf16 5.8 us, two launches 9.3), and for vectors
  // where panels are small and clusters of 16 fill the SMs (16 x 1024 x 1280
  // bf16 26 us against 32, 2 x 4096 x 320 fp16 10.6 against 13.2; but with a
  // panel of 3 MB, 2 x 39760 x 160 fp16, 30 against 26, and with 64 CTAs, 4 x
  // 12708 x 104, 18 against 15). How much all panels at a time are is not in
  // the rule: past the L2 cache the rows come out of DRAM twice, which costs
  // less than the second launch for 64 x 4096 x 320 fp16 (168 MB of rows at a
  // time, 89 us against 95) and more for 64 x 4096 x 640 (299 MB, 189 against
  // 172). The backward, whose rows take twice the
  // shared memory and registers, has its two launches always: one launch of
  // clusters took 22 us for 2 x 4096 x 640 fp16 (two 20), 62 for 13 x 9961 x
  // 40 bf16 (36).
  // What a CTA does besides its rows costs as much as some eight rows of each
  // thread, so there are no more CTAs than it takes to give every SM one and
  // most a second (1.5 an SM; with 3 an SM 16 x 1024 x 1280 took 29 us):
  // narrow tiles first, which make more panels, then clusters of more CTAs.
  bool whole = false;
  int s = 1;
  p->cluster = false;
  p->clusters = 0;
  if (!bwd) {
    whole = gn_tiles(channels, unit, 128, es, p);
    while (whole && samples * p->tiles * 8 < (int64_t)sms * 3 / 2 && p->tile_ch > unit &&
           (p->tile_ch - unit) * es >= 64) {
      const int was = p->tile_ch;
      whole = gn_tiles(channels, unit, (was - unit) * es, es, p);
      if (p->tile_ch >= was) break;
    }
  }
  if (whole) {
    p->panels = samples * p->tiles;
    p->max_groups = max_groups(whole);
    const int64_t TY = kGnThreads / p->tw;
    // Clusters of 16 need 16 free places in one part of the chip: fewer of
    // them fit than the SMs would hold CTAs. most_cluster: what the device
    // places at all.
    while (s < most_cluster && p->panels * s < (int64_t)sms * 3 / 2 && rows > s * TY * 2 &&
           !(s == 8 && p->panels > sms / 8))
      s *= 2;
    p->cluster = rows <= s * TY * kGnRing ||
                 (grain == 16 && (double)rows * p->tile_ch * es <= (double)kSlabBytes &&
                  p->panels * s >= (int64_t)sms * 3 / 4);
  }
  if (p->cluster) {
    p->slices = s;
    p->clusters = (int)(p->panels * s <= places ? p->panels : places / s);
    p->slice_rows = (rows + s - 1) / s;
    p->batch = p->panels;
    p->part_bytes = 0;
  } else {
    // Batches whose rows stay in the L2 cache (129 MB) from the launch that
    // sums them to the one that applies them, with the outputs beside them
    // (2 x 262144 x 256 bf16: 139 us, with batches of half the size 155; 8 x
    // 16384 x 320 backward 82 and 90; with twice the size 141 and 80).
    whole = gn_tiles(channels, unit, 128, es, p);
    p->panels = samples * p->tiles;
    p->max_groups = max_groups(whole);
    const double slab = (double)rows * p->tile_ch * es * (bwd ? 2 : 1);   // what a panel reads
    p->batch = p->panels;
    if (slab * p->panels > (double)kBatchBytes[bwd]) {
      const int64_t step = whole ? 1 : p->tiles;
      int64_t b = (int64_t)(kBatchBytes[bwd] / slab) / step * step;
      if (b < step) b = step;
      // As many batches, of about one size.
      const int64_t n = (p->panels + b - 1) / b;
      b = ((p->panels + n - 1) / n + step - 1) / step * step;
      p->batch = b < p->panels ? b : p->panels;
    }
    const int64_t TY = kGnThreads / p->tw;
    int64_t slices = places / p->batch;   // not a CTA more than fit at a time
    if (slices > kGnMaxSlices) slices = kGnMaxSlices;
    const int64_t least = 4 * TY;       // rows of a slice: four a thread
    if (slices > (rows + least - 1) / least) slices = (rows + least - 1) / least;
    if (slices < 1) slices = 1;
    p->slice_rows = (rows + slices - 1) / slices;
    p->slices = (int)((rows + p->slice_rows - 1) / p->slice_rows);
    p->part_bytes = (size_t)p->panels * p->slices * p->max_groups * sizeof(float2);
    p->part_bytes = (p->part_bytes + 15) / 16 * 16;
  }
  p->cols_bytes = bwd ? (size_t)samples * p->slices * 2 * channels * sizeof(float) : 0;
  return p->panels * p->slices <= INT32_MAX && p->slice_rows <= INT32_MAX;
}

struct GnCall {
  int64_t samples, rows, channels, groups;
  ln_dtype dtype;
};

ln_status check_shape(const GnCall& c) {
  if (!known_dtype(c.dtype)) return LN_ERR_UNSUPPORTED;
  if (c.samples < 0 || c.samples > INT32_MAX || c.rows < 0 || c.rows > (1ll << 40) ||
      c.channels < 1 || c.channels > GN_MAX_CHANNELS ||
      c.groups < 1 || c.channels % c.groups != 0)
    return LN_ERR_SHAPE;
  return LN_OK;
}

Strided tensor(const void* p, int64_t sample, int64_t row, const GnCall& c) {
  const int64_t es = (int64_t)elem_size(c.dtype);
  Strided s;
  s.p = p;
  s.n[0] = c.samples;
  s.n[1] = c.rows;
  s.stride[0] = sample * es;
  s.stride[1] = row * es;
  s.width = c.channels * es;
  return s;
}

// The bytes that a tensor's rows are aligned to, `most` at most.
int grain_of(const Strided& s, int most) {
  if (s.empty()) return most;
  while (most > 1 &&
         (!aligned(s.p, most) || s.width % most != 0 || (s.n[0] > 1 && s.stride[0] % most != 0) ||
          (s.n[1] > 1 && s.stride[1] % most != 0)))
    most /= 2;
  return most;
}

ln_status plan_call(const GnCall& c, bool bwd, int grain, GnPlan* p) {
  int sms = 0, most_cluster = 1;
  cudaError_t e = (cudaError_t)device_sm_count(&sms);
  if (e == cudaSuccess && !bwd)
    e = (cudaError_t)cluster_limit(gn_table_f32(false, true, true, kActNone), kGnThreads,
                                   gn_smem_bytes(1, true), &most_cluster);
  if (e != cudaSuccess) return cuda_fail(e);
  return gn_plan(c.samples, c.rows, (int)c.channels, (int)c.groups, elem_size(c.dtype), bwd, grain,
                 sms, most_cluster, p)
             ? LN_OK
             : LN_ERR_SHAPE;
}

ln_status launch(const GnCall& c, const GnPlan& p, GnArgs a, bool bwd, int grain, int act,
                 cudaStream_t st) {
  a.slice_rows = p.slice_rows;
  a.slices = p.slices;
  a.channels = (int)c.channels;
  a.groups = (int)c.groups;
  a.cpg = (int)(c.channels / c.groups);
  a.tiles = p.tiles;
  a.tile_ch = p.tile_ch;
  a.tw = p.tw;
  a.grain = grain;
  a.by_tile_ch.set(p.tile_ch);
  a.max_groups = p.max_groups;
  a.by_slices.set(p.slices);
  a.by_tiles.set(p.tiles);
  a.by_tw.set(p.tw);
  a.by_tc.set(p.tw * (int)(16 / elem_size(c.dtype)));
  a.by_ty.set(kGnThreads / p.tw);
  a.by_cpg.set(a.cpg);
  a.rows = c.rows;
  a.inv_m = (float)(1.0 / ((double)c.rows * a.cpg));
  const void* fn = c.dtype == LN_F32    ? gn_table_f32(bwd, p.cluster, grain < 16, act)
                   : c.dtype == LN_BF16 ? gn_table_bf16(bwd, p.cluster, grain < 16, act)
                                        : gn_table_f16(bwd, p.cluster, grain < 16, act);
  const size_t smem = gn_smem_bytes(bwd ? 2 : 1, p.cluster);
  const cudaError_t opt = (cudaError_t)allow_dyn_smem(fn, smem);
  if (opt != cudaSuccess) return cuda_fail(opt);
  if (p.cluster) {
    if (p.slices > 8) {
      const cudaError_t e =
          cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return cuda_fail(e);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.clusters * p.slices));
    cfg.blockDim = dim3(kGnThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.slices;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int panels = (int)p.panels;
    void* args[] = {&a, &panels};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
    return e == cudaSuccess ? LN_OK : cuda_fail(e);
  }
  // Launch j takes the statistics of batch j and applies batch j - 1, whose
  // rows are then still in the L2 cache.
  const int64_t batches = (p.panels + p.batch - 1) / p.batch;
  const auto first = [&](int64_t j) { return (int)(j * p.batch < p.panels ? j * p.batch : p.panels); };
  for (int64_t j = 0; j <= batches; ++j) {
    int s0 = first(j), s1 = first(j + 1);
    int a0 = j > 0 ? first(j - 1) : 0, a1 = j > 0 ? s0 : 0;
    const int n = s1 - s0 > a1 - a0 ? s1 - s0 : a1 - a0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n * p.slices));
    cfg.blockDim = dim3(kGnThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = j > 0 ? 1 : 0;   // the first launch waits for the stream as any other
    void* args[] = {&a, &s0, &s1, &a0, &a1};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return LN_OK;
}

}  // namespace
}  // namespace nf

using namespace nf;

extern "C" {

ln_status gn_workspace_bytes(int64_t samples, int64_t rows, int64_t channels, int64_t groups,
                             ln_dtype dtype, int backward, size_t* bytes) {
  if (bytes == nullptr) return LN_ERR_NULL;
  const GnCall c = {samples, rows, channels, groups, dtype};
  ln_status s = check_shape(c);
  if (s != LN_OK) return s;
  *bytes = 0;
  if (samples == 0 || rows == 0) return LN_OK;
  size_t need = 0;
  for (int grain = 16; grain >= (int)elem_size(dtype); grain /= 2) {
    if ((channels * (int64_t)elem_size(dtype)) % grain != 0) continue;
    GnPlan p;
    s = plan_call(c, backward != 0, grain, &p);
    if (s != LN_OK) return s;
    if (p.bytes() > need) need = p.bytes();
  }
  *bytes = need;
  return LN_OK;
}

ln_status gn_fwd(const void* x, int64_t x_sample, int64_t x_row, const void* gamma,
                 const void* beta, int64_t param_sample, float eps, gn_act act,
                 int zero_centered_gamma, void* y, int64_t y_sample, int64_t y_row, float* mean,
                 float* rstd, cudaStream_t stream, int64_t samples, int64_t rows,
                 int64_t channels, int64_t groups, ln_dtype dtype, void* workspace,
                 size_t workspace_bytes) {
  const GnCall c = {samples, rows, channels, groups, dtype};
  ln_status s = check_shape(c);
  if (s != LN_OK) return s;
  if (act != GN_ACT_NONE && act != GN_ACT_SILU && act != GN_ACT_GELU) return LN_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f) || !isfinite(eps)) return LN_ERR_INVALID;
  if (x_sample < 0 || x_row < 0 || y_sample < 0 || y_row < 0) return LN_ERR_INVALID;
  if (param_sample != 0 && param_sample < channels) return LN_ERR_INVALID;
  const bool some = samples > 0 && rows > 0;
  if (some && (x == nullptr || y == nullptr)) return LN_ERR_NULL;
  const size_t es = elem_size(dtype);
  const void* tensors[] = {x, gamma, beta, y};
  for (const void* t : tensors)
    if (!aligned(t, es)) return LN_ERR_ALIGN;
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return LN_ERR_ALIGN;
  const Strided sx = tensor(x, x_sample, x_row, c), sy = tensor(y, y_sample, y_row, c);
  if (self_overlaps(sy) || may_overlap(sy, sx)) return LN_ERR_INVALID;
  const size_t stats = (size_t)samples * groups * 4;
  const size_t params = samples > 0 ? ((size_t)(samples - 1) * param_sample + channels) * es : 0;
  const Range outs[] = {{mean, stats}, {rstd, stats}, {workspace, workspace_bytes}};
  const Range ins[] = {sx.range(), {gamma, params}, {beta, params}, sy.range()};
  if (any_overlap(outs, 3, ins, 4)) return LN_ERR_INVALID;
  const Range yr = sy.range();
  if (any_overlap(&yr, 1, ins + 1, 2)) return LN_ERR_INVALID;
  if (samples == 0) return LN_OK;
  if (rows == 0) {
    cudaError_t e = cudaSuccess;
    if (mean) e = cudaMemsetAsync(mean, 0, stats, stream);
    if (e == cudaSuccess && rstd) e = cudaMemsetAsync(rstd, 0, stats, stream);
    return e == cudaSuccess ? LN_OK : cuda_fail(e);
  }
  const int grain = grain_of(sy, grain_of(sx, 16));
  GnPlan p;
  s = plan_call(c, false, grain, &p);
  if (s != LN_OK) return s;
  if (p.bytes() > 0 &&
      (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < p.bytes()))
    return LN_ERR_WORKSPACE;
  GnArgs a = {};
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.out = y;
  a.mean = mean;
  a.rstd = rstd;
  a.part = static_cast<float2*>(workspace);
  a.x_sample = x_sample;
  a.x_row = x_row;
  a.out_sample = y_sample;
  a.out_row = y_row;
  a.param_sample = param_sample;
  a.eps = eps;
  a.zero_centered = zero_centered_gamma ? 1 : 0;
  return launch(c, p, a, false, grain, (int)act, stream);
}

ln_status gn_bwd(const void* dy, int64_t dy_sample, int64_t dy_row, const void* x,
                 int64_t x_sample, int64_t x_row, const void* gamma, const void* beta,
                 int64_t param_sample, gn_act act, int zero_centered_gamma, const float* mean,
                 const float* rstd, void* dx, int64_t dx_sample, int64_t dx_row, void* dgamma,
                 void* dbeta, cudaStream_t stream, int64_t samples, int64_t rows,
                 int64_t channels, int64_t groups, ln_dtype dtype, ln_dtype grad_dtype,
                 void* workspace, size_t workspace_bytes) {
  const GnCall c = {samples, rows, channels, groups, dtype};
  ln_status s = check_shape(c);
  if (s != LN_OK) return s;
  if (!known_dtype(grad_dtype)) return LN_ERR_UNSUPPORTED;
  if (act != GN_ACT_NONE && act != GN_ACT_SILU && act != GN_ACT_GELU) return LN_ERR_UNSUPPORTED;
  if (dy_sample < 0 || dy_row < 0 || x_sample < 0 || x_row < 0 || dx_sample < 0 || dx_row < 0)
    return LN_ERR_INVALID;
  if (param_sample != 0 && param_sample < channels) return LN_ERR_INVALID;
  const bool some = samples > 0 && rows > 0;
  if (some && (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr ||
               dx == nullptr))
    return LN_ERR_NULL;
  const size_t es = elem_size(dtype), gs = elem_size(grad_dtype);
  const void* tensors[] = {dy, x, gamma, beta, dx};
  for (const void* t : tensors)
    if (!aligned(t, es)) return LN_ERR_ALIGN;
  if (!aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dgamma, gs) || !aligned(dbeta, gs))
    return LN_ERR_ALIGN;
  const Strided sx = tensor(x, x_sample, x_row, c), sd = tensor(dy, dy_sample, dy_row, c),
                so = tensor(dx, dx_sample, dx_row, c);
  if (self_overlaps(so) || may_overlap(so, sx) || may_overlap(so, sd)) return LN_ERR_INVALID;
  const size_t stats = (size_t)samples * groups * 4;
  const size_t params = samples > 0 ? ((size_t)(samples - 1) * param_sample + channels) * es : 0;
  const int64_t grad_rows = param_sample != 0 ? samples : 1;
  const size_t grads = (size_t)grad_rows * channels * gs;
  const Range outs[] = {{dgamma, grads}, {dbeta, grads}, {workspace, workspace_bytes}};
  const Range ins[] = {sd.range(), sx.range(), {gamma, params}, {beta, params}, {mean, stats},
                       {rstd, stats}, so.range()};
  if (any_overlap(outs, 3, ins, 7)) return LN_ERR_INVALID;
  const Range dr = so.range();
  if (any_overlap(&dr, 1, ins + 2, 4)) return LN_ERR_INVALID;
  if (!some) {
    cudaError_t e = cudaSuccess;
    if (dgamma && grads) e = cudaMemsetAsync(dgamma, 0, grads, stream);
    if (e == cudaSuccess && dbeta && grads) e = cudaMemsetAsync(dbeta, 0, grads, stream);
    return e == cudaSuccess ? LN_OK : cuda_fail(e);
  }
  if (grad_rows > 65535 && (dgamma != nullptr || dbeta != nullptr))
    return LN_ERR_SHAPE;   // rows of the finalize's grid
  const int grain = grain_of(so, grain_of(sd, grain_of(sx, 16)));
  GnPlan p;
  s = plan_call(c, true, grain, &p);
  if (s != LN_OK) return s;
  if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < p.bytes())
    return LN_ERR_WORKSPACE;
  GnArgs a = {};
  a.x = x;
  a.dy = dy;
  a.gamma = gamma;
  a.beta = beta;
  a.out = dx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.part = static_cast<float2*>(workspace);
  a.cols = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part_bytes);
  a.x_sample = x_sample;
  a.x_row = x_row;
  a.dy_sample = dy_sample;
  a.dy_row = dy_row;
  a.out_sample = dx_sample;
  a.out_row = dx_row;
  a.param_sample = param_sample;
  a.zero_centered = zero_centered_gamma ? 1 : 0;
  s = launch(c, p, a, true, grain, (int)act, stream);
  if (s != LN_OK || (dgamma == nullptr && dbeta == nullptr)) return s;
  const int H = (int)channels;
  const int64_t P = (param_sample != 0 ? 1 : samples) * p.slices;
  const cudaError_t e = launch_bwd_finalize(a.cols, (int)P, 2 * H, H, true, dgamma, dbeta, nullptr,
                                            (int)grad_dtype, stream, (int)grad_rows);
  return e == cudaSuccess ? LN_OK : cuda_fail(e);
}

}  // extern "C"
