// Rotary positions with the heads' RMSNorm: C entry points, argument checks
// and launch plan.
#include <math.h>

#include "../../include/normfuse.h"
#include "launch.h"
#include "rope_kernels.cuh"
#include "validate.h"

namespace nf {

const void* rope_table_f32(int vec, int ns, bool inter, bool aligned, bool full, bool bwd);
const void* rope_table_bf16(int vec, int ns, bool inter, bool aligned, bool full, bool bwd);
const void* rope_table_f16(int vec, int ns, bool inter, bool aligned, bool full, bool bwd);

namespace {

ln_status cuda_fail(cudaError_t e) {
  nf_set_last_cuda_error((int)e);
  return LN_ERR_CUDA;
}

struct Shape {
  int64_t batch, tokens, dim;
  ln_dtype dtype;
};

constexpr int kBwdBlocksPerSm = 2;   // backward CTAs an SM, each with a row of partials
constexpr int kFwdBlocksPerSm = 3;
// Heads of a tile for each group of threads: with 4 the forward over 1 x 16384
// tokens takes 71 us for 62, with 16 the one over 3 x 1023 takes 18 for 17.
constexpr int kRopeItems = 8;

Strided strided(const void* p, const int64_t* st, int64_t heads, const Shape& c) {
  const int64_t es = (int64_t)elem_size(c.dtype);
  Strided s;
  s.p = p;
  s.n[0] = c.batch;
  s.n[1] = c.tokens;
  s.n[2] = heads;
  for (int i = 0; i < 3; ++i) s.stride[i] = st[i] * es;
  s.width = c.dim * es;
  return s;
}

bool same(const Strided& a, const Strided& b) {
  if (a.p != b.p) return false;
  for (int i = 0; i < 3; ++i)
    if (a.n[i] > 1 && a.stride[i] != b.stride[i]) return false;
  return true;
}

ln_status check_positions(const rope_positions* r, const Shape& c) {
  if (r == nullptr) return LN_ERR_NULL;
  if (r->bits != 32 && r->bits != 64) return LN_ERR_UNSUPPORTED;
  if (r->layout != ROPE_HALF && r->layout != ROPE_INTERLEAVED) return LN_ERR_UNSUPPORTED;
  if (r->axes < 1 || r->axes > kRopeMaxAxes) return LN_ERR_SHAPE;
  if (r->rot < 2 || r->rot % 2 != 0 || r->rot > c.dim) return LN_ERR_SHAPE;
  if (!isfinite(r->scale)) return LN_ERR_INVALID;
  for (int i = 0; i < 3; ++i)
    if (r->stride[i] < 0) return LN_ERR_INVALID;
  if (c.batch > 0 && c.tokens > 0 && (r->pos == nullptr || r->freqs == nullptr)) return LN_ERR_NULL;
  if (!aligned(r->pos, r->bits / 8) || !aligned(r->freqs, 8)) return LN_ERR_ALIGN;
  return LN_OK;
}

ln_status check_shape(const Shape& c) {
  if (!known_dtype(c.dtype)) return LN_ERR_UNSUPPORTED;
  if (c.batch < 0 || c.tokens < 0 || c.batch > (1ll << 40) || c.tokens > (1ll << 40))
    return LN_ERR_SHAPE;
  if (c.batch > 0 && c.tokens > (1ll << 40) / c.batch) return LN_ERR_SHAPE;
  if (c.dim < 2 || c.dim % 2 != 0 || c.dim > kRopeMaxDim) return LN_ERR_SHAPE;
  return LN_OK;
}

Range pos_range(const rope_positions* r, const Shape& c) {
  if (c.batch == 0 || c.tokens == 0) return {nullptr, 0};
  const int64_t n = (r->axes - 1) * r->stride[0] + (c.batch - 1) * r->stride[1] +
                    (c.tokens - 1) * r->stride[2] + 1;
  return {r->pos, (size_t)n * (r->bits / 8)};
}

// Whether a tensor can be read and written `bytes` at a time.
bool can(const Strided& s, int64_t bytes) {
  if (s.empty()) return true;
  if (!aligned(s.p, bytes) || s.width % bytes != 0) return false;
  for (int i = 0; i < 3; ++i)
    if (s.n[i] > 1 && s.stride[i] % bytes != 0) return false;
  return true;
}

struct RopePlan {
  const void* fn = nullptr;
  int grid = 0;
};

ln_status plan(const Shape& c, const rope_positions* r, const Strided* tensors, int n_tensors,
               bool bwd, RopeArgs* a, RopePlan* p) {
  const int es = (int)elem_size(c.dtype), dim = (int)c.dim, rot = (int)r->rot;
  const bool inter = r->layout == ROPE_INTERLEAVED;
  int sms = 0;
  const cudaError_t e = (cudaError_t)device_sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  // Widest access that divides the head, the rotated half and every stride.
  int v = 16 / es;
  const auto fits = [&](int w) {
    if (dim % w != 0 || (!inter && rot / 2 % w != 0)) return false;
    for (int i = 0; i < n_tensors; ++i)
      if (!can(tensors[i], (int64_t)w * es)) return false;
    return true;
  };
  while (v > 1 && !fits(v)) v /= 2;
  bool al = true;
  if (v == 1) {
    al = false;
    if (inter) v = 2;   // pairs of neighbours, element by element
  }
  const int nv = dim / v;
  const int slots = inter ? (nv + 1) / 2 : rot / 2 / v + (nv - rot / v + 1) / 2;
  // Heads of more than 32 slots: as few a lane as 32 lanes take, so that
  // neighbouring lanes' accesses are neighbours and registers last (element by
  // element, fp16: heads of 98, 15 x 3804 tokens forward 264 us, with 8 slots a
  // lane 372; heads of 128, 21 x 8322 tokens backward 299 and 792). The
  // backward in pairs of elements takes as many as a lane holds, four, because
  // fewer lanes have less to do besides (fp16 heads of 170, 53 x 248 tokens: 190
  // us, with two a lane 248).
  int ns = 1;
  if (slots > 32 && bwd && v > 1) ns = 8 / v;
  while (32 * ns < slots) ns *= 2;
  int lanes = 1;
  while (lanes * ns < slots) lanes *= 2;
  const bool full = rot == dim && slots == lanes * ns && dim == 2 * v * lanes * ns;
  p->fn = c.dtype == LN_F32    ? rope_table_f32(v, ns, inter, al, full, bwd)
          : c.dtype == LN_BF16 ? rope_table_bf16(v, ns, inter, al, full, bwd)
                               : rope_table_f16(v, ns, inter, al, full, bwd);
  if (p->fn == nullptr) return LN_ERR_UNSUPPORTED;
  const int per_cta = kRopeThreads / lanes;
  const int per_sm = bwd ? kBwdBlocksPerSm : kFwdBlocksPerSm;
  a->lanes = lanes;
  a->row = (dim / 2 + 3) / 4 * 4;
  a->wide = 1;
  while (a->wide < rot / 2) a->wide *= 2;
  // What a token costs a side: its heads' rows, and its angles, which cost a
  // thread about a sixth of a row.
  int64_t cost[2], all = 0;
  for (int s = 0; s < 2; ++s) {
    cost[s] = a->side[s].heads > 0 ? (int64_t)a->side[s].heads * lanes * 6 + rot / 2 : 0;
    all += cost[s];
  }
  const int most_tile = kRopeMaxTable / a->row;
  for (int s = 0; s < 2; ++s) {
    RopeSide& d = a->side[s];
    d.head_lanes = d.heads < per_cta ? (d.heads > 0 ? d.heads : 1) : per_cta;
    d.token_lanes = per_cta / d.head_lanes;
    d.tile = 1;
    d.row_tiles = d.tiles = 0;
    a->blocks[s] = 0;
    if (d.heads == 0) continue;
    // Tokens of a tile: kRopeItems rows for every group, fewer where the
    // device would not have a CTA for each of its places.
    const int64_t rounds = (d.heads + d.head_lanes - 1) / d.head_lanes;
    int64_t tile = (kRopeItems + rounds - 1) / rounds * d.token_lanes;
    const int64_t places = sms * per_sm * cost[s] / all;
    const int64_t even = a->batch * a->tokens / (places > 0 ? places : 1);
    if (tile > even) tile = even;
    if (tile < d.token_lanes && a->batch * a->tokens >= d.token_lanes * (int64_t)sms / 4)
      tile = d.token_lanes;
    if (tile > a->tokens) tile = a->tokens;
    if (tile > most_tile) tile = most_tile;
    if (bwd && tile > d.token_lanes && places > 0) {
      // Whole rounds of the CTAs that there are places for.
      const int64_t rows = a->batch * a->tokens, rounds_of = (rows + places * tile - 1) / (places * tile);
      const int64_t need = (rows + places * rounds_of - 1) / (places * rounds_of);
      const int64_t even_tile = (need + d.token_lanes - 1) / d.token_lanes * d.token_lanes;
      if (even_tile < tile) tile = even_tile;
    }
    if (tile < 1) tile = 1;
    d.tile = (int)tile;
    d.row_tiles = (a->tokens + tile - 1) / tile;
    d.tiles = a->batch * d.row_tiles;
    // Forward: a CTA a tile, so that the device deals them out; backward: no
    // more than a CTA for each place, which leave a row of partials each.
    const int64_t most = !bwd ? (1 << 30) - 1 : places > 0 ? places : 1;
    a->blocks[s] = (int)(d.tiles < most ? d.tiles : most);
  }
  p->grid = a->blocks[0] + a->blocks[1];
  return LN_OK;
}

void fill(RopeArgs* a, const Shape& c, const rope_positions* r, float eps, int zero_centered) {
  a->pos = r->pos;
  a->freqs = r->freqs;
  for (int i = 0; i < 3; ++i) a->pos_s[i] = r->stride[i];
  // Sequences that lie one behind the other in every tensor, and single
  // tokens, are one sequence.
  a->batch = c.batch;
  a->tokens = c.tokens;
  bool flat = c.tokens == 1 || c.batch == 1 || r->stride[1] == c.tokens * r->stride[2];
  for (RopeSide& d : a->side)
    if (d.heads > 0 && c.tokens > 1 && c.batch > 1)
      flat = flat && d.in_s[0] == c.tokens * d.in_s[1] && d.out_s[0] == c.tokens * d.out_s[1] &&
             (d.x == nullptr || d.x_s[0] == c.tokens * d.x_s[1]);
  if (flat && c.batch > 1) {
    if (c.tokens == 1) {
      a->pos_s[2] = a->pos_s[1];
      for (RopeSide& d : a->side) {
        d.in_s[1] = d.in_s[0];
        d.out_s[1] = d.out_s[0];
        d.x_s[1] = d.x_s[0];
      }
    }
    a->tokens = c.batch * c.tokens;
    a->batch = 1;
  }
  a->pos64 = r->bits == 64;
  a->axes = (int)r->axes;
  a->dim = (int)c.dim;
  a->rot = (int)r->rot;
  a->scale_c = a->scale_s = r->scale;
  a->eps = eps;
  a->inv_dim = 1.0f / (float)c.dim;
  a->zero_centered = zero_centered ? 1 : 0;
}

bool strides_ok(const int64_t* s) {
  return s[0] >= 0 && s[1] >= 0 && s[2] >= 0;
}

}  // namespace
}  // namespace nf

using namespace nf;

extern "C" {

ln_status rope_frequencies(int64_t rot, double base, rope_scaling scaling, double factor,
                           int64_t original, double turns_fast, double turns_slow,
                           double* freqs, float* scale) {
  if (freqs == nullptr || scale == nullptr) return LN_ERR_NULL;
  if (rot < 2 || rot % 2 != 0 || rot > kRopeMaxDim) return LN_ERR_SHAPE;
  if (scaling != ROPE_SCALING_NONE && scaling != ROPE_SCALING_LINEAR &&
      scaling != ROPE_SCALING_NTK && scaling != ROPE_SCALING_YARN)
    return LN_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !isfinite(base)) return LN_ERR_INVALID;
  if (scaling != ROPE_SCALING_NONE && (!(factor >= 1.0) || !isfinite(factor)))
    return LN_ERR_INVALID;
  const bool yarn = scaling == ROPE_SCALING_YARN;
  if (yarn && (original < 1 || !(turns_slow > 0.0) || !(turns_fast >= turns_slow) ||
               !isfinite(turns_fast)))
    return LN_ERR_INVALID;
  const double d = (double)rot;
  if (scaling == ROPE_SCALING_NTK && rot > 2) base *= pow(factor, d / (d - 2.0));
  double low = 0.0, width = 1.0;
  if (yarn) {
    // The pair (a real number) that makes `turns` turns in the original context.
    const double kTwoPi = 6.283185307179586;
    const auto pair = [&](double turns) {
      return d * log((double)original / (turns * kTwoPi)) / (2.0 * log(base));
    };
    low = fmax(floor(pair(turns_fast)), 0.0);
    width = fmax(fmin(ceil(pair(turns_slow)), d - 1.0) - low, 1e-3);
  }
  for (int64_t j = 0; j < rot / 2; ++j) {
    const double f = pow(base, -2.0 * (double)j / d);
    double v = f;
    if (scaling == ROPE_SCALING_LINEAR) v = f / factor;
    if (yarn) {
      const double share = fmin(fmax(((double)j - low) / width, 0.0), 1.0);
      v = f / factor * share + f * (1.0 - share);
    }
    freqs[j] = v;
  }
  *scale = yarn ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
  return LN_OK;
}

ln_status rope_fwd(const rope_heads* q, const rope_heads* k, const rope_positions* positions,
                   float eps, int zero_centered_gamma, cudaStream_t stream, int64_t batch,
                   int64_t tokens, int64_t head_dim, ln_dtype dtype) {
  const Shape c = {batch, tokens, head_dim, dtype};
  ln_status s = check_shape(c);
  if (s != LN_OK) return s;
  if (q == nullptr) return LN_ERR_NULL;
  s = check_positions(positions, c);
  if (s != LN_OK) return s;
  if (!(eps >= 0.0f) || !isfinite(eps)) return LN_ERR_INVALID;
  const rope_heads* sides[2] = {q, k};
  const size_t es = elem_size(dtype);
  const bool some = batch > 0 && tokens > 0;
  Strided in[2], out[2], all[4];
  Range small[4] = {};
  RopeArgs a = {};
  for (int i = 0; i < 2; ++i) {
    const rope_heads* h = sides[i];
    if (h == nullptr) continue;
    if (h->heads < 0 || h->heads > ROPE_MAX_HEADS) return LN_ERR_SHAPE;
    if (!strides_ok(h->x_stride) || !strides_ok(h->y_stride)) return LN_ERR_INVALID;
    if (some && h->heads > 0 && (h->x == nullptr || h->y == nullptr)) return LN_ERR_NULL;
    if (!aligned(h->x, es) || !aligned(h->y, es) || !aligned(h->gamma, es)) return LN_ERR_ALIGN;
    in[i] = strided(h->x, h->x_stride, h->heads, c);
    out[i] = strided(h->y, h->y_stride, h->heads, c);
    small[i] = {h->gamma, (size_t)head_dim * es};
    RopeSide& d = a.side[i];
    d.in = h->x;
    d.out = h->y;
    d.gamma = h->gamma;
    d.heads = (int)h->heads;
    for (int j = 0; j < 3; ++j) {
      d.in_s[j] = h->x_stride[j];
      d.out_s[j] = h->y_stride[j];
    }
  }
  small[2] = pos_range(positions, c);
  small[3] = {positions->freqs, (size_t)positions->axes * (positions->rot / 2) * 8};
  for (int i = 0; i < 2; ++i) {
    if (out[i].empty()) continue;
    if (self_overlaps(out[i])) return LN_ERR_INVALID;
    for (int j = 0; j < 2; ++j)
      if (!(i == j && same(out[i], in[j])) && may_overlap(out[i], in[j])) return LN_ERR_INVALID;
    const Range r = out[i].range();
    if (any_overlap(&r, 1, small, 4)) return LN_ERR_INVALID;
  }
  if (may_overlap(out[0], out[1])) return LN_ERR_INVALID;
  if (!some || a.side[0].heads + a.side[1].heads == 0) return LN_OK;
  fill(&a, c, positions, eps, zero_centered_gamma);
  for (int i = 0; i < 2; ++i) {
    all[i] = in[i];
    all[2 + i] = out[i];
  }
  RopePlan p;
  s = plan(c, positions, all, 4, false, &a, &p);
  if (s != LN_OK) return s;
  void* args[] = {&a};
  const cudaError_t e = cudaLaunchKernel(p.fn, dim3(p.grid), dim3(kRopeThreads), args, 0,
                                         stream);
  return e == cudaSuccess ? LN_OK : cuda_fail(e);
}

ln_status rope_bwd_workspace_bytes(int64_t head_dim, size_t* bytes) {
  if (bytes == nullptr) return LN_ERR_NULL;
  *bytes = 0;
  if (head_dim < 2 || head_dim % 2 != 0 || head_dim > kRopeMaxDim) return LN_ERR_SHAPE;
  int sms = 0;
  const cudaError_t e = (cudaError_t)device_sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  *bytes = (size_t)sms * kBwdBlocksPerSm * 2 * head_dim * sizeof(float);
  return LN_OK;
}

ln_status rope_bwd(const rope_heads_grad* q, const rope_heads_grad* k,
                   const rope_positions* positions, float eps, int zero_centered_gamma,
                   cudaStream_t stream, int64_t batch, int64_t tokens, int64_t head_dim,
                   ln_dtype dtype, ln_dtype grad_dtype, void* workspace,
                   size_t workspace_bytes) {
  const Shape c = {batch, tokens, head_dim, dtype};
  ln_status s = check_shape(c);
  if (s != LN_OK) return s;
  if (!known_dtype(grad_dtype)) return LN_ERR_UNSUPPORTED;
  if (q == nullptr) return LN_ERR_NULL;
  s = check_positions(positions, c);
  if (s != LN_OK) return s;
  if (!(eps >= 0.0f) || !isfinite(eps)) return LN_ERR_INVALID;
  const rope_heads_grad* sides[2] = {q, k};
  const size_t es = elem_size(dtype), gs = elem_size(grad_dtype);
  const bool some = batch > 0 && tokens > 0;
  Strided dy[2], x[2], out[2], all[6];
  Range small[4] = {}, grads[3] = {};
  RopeArgs a = {};
  bool sums = false;
  for (int i = 0; i < 2; ++i) {
    const rope_heads_grad* h = sides[i];
    if (h == nullptr) continue;
    if (h->heads < 0 || h->heads > ROPE_MAX_HEADS) return LN_ERR_SHAPE;
    if (!strides_ok(h->dy_stride) || !strides_ok(h->dx_stride) ||
        (h->gamma != nullptr && !strides_ok(h->x_stride)))
      return LN_ERR_INVALID;
    const bool live = some && h->heads > 0;
    if (live && (h->dy == nullptr || h->dx == nullptr || (h->gamma != nullptr && h->x == nullptr)))
      return LN_ERR_NULL;
    if (!aligned(h->dy, es) || !aligned(h->dx, es) || !aligned(h->gamma, es) ||
        (h->gamma != nullptr && !aligned(h->x, es)) || !aligned(h->dgamma, gs))
      return LN_ERR_ALIGN;
    if (h->gamma == nullptr && h->dgamma != nullptr) return LN_ERR_INVALID;
    dy[i] = strided(h->dy, h->dy_stride, h->heads, c);
    if (h->gamma != nullptr) x[i] = strided(h->x, h->x_stride, h->heads, c);
    out[i] = strided(h->dx, h->dx_stride, h->heads, c);
    small[i] = {h->gamma, (size_t)head_dim * es};
    grads[i] = {h->dgamma, (size_t)head_dim * gs};
    sums = sums || h->dgamma != nullptr;
    RopeSide& d = a.side[i];
    d.in = h->dy;
    d.x = h->x;
    d.out = h->dx;
    d.gamma = h->gamma;
    d.heads = (int)h->heads;
    for (int j = 0; j < 3; ++j) {
      d.in_s[j] = h->dy_stride[j];
      d.x_s[j] = h->x_stride[j];
      d.out_s[j] = h->dx_stride[j];
    }
  }
  small[2] = pos_range(positions, c);
  small[3] = {positions->freqs, (size_t)positions->axes * (positions->rot / 2) * 8};
  grads[2] = {workspace, workspace_bytes};
  const Range ins[] = {small[0], small[1], small[2], small[3], dy[0].range(), dy[1].range(),
                       x[0].range(), x[1].range(), out[0].range(), out[1].range()};
  if (any_overlap(grads, 3, ins, 10)) return LN_ERR_INVALID;
  for (int i = 0; i < 2; ++i) {
    if (out[i].empty()) continue;
    if (self_overlaps(out[i])) return LN_ERR_INVALID;
    for (int j = 0; j < 2; ++j) {
      if (!(i == j && same(out[i], dy[j])) && may_overlap(out[i], dy[j])) return LN_ERR_INVALID;
      if (may_overlap(out[i], x[j])) return LN_ERR_INVALID;
    }
    if (any_overlap(&ins[8 + i], 1, small, 4)) return LN_ERR_INVALID;
  }
  if (may_overlap(out[0], out[1])) return LN_ERR_INVALID;
  if (!some || a.side[0].heads + a.side[1].heads == 0) {
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 2; ++i)
      if (e == cudaSuccess && grads[i].p)
        e = cudaMemsetAsync(const_cast<void*>(grads[i].p), 0, grads[i].bytes, stream);
    return e == cudaSuccess ? LN_OK : cuda_fail(e);
  }
  fill(&a, c, positions, eps, zero_centered_gamma);
  if (sums) {
    if (workspace == nullptr || !aligned(workspace, 16)) return LN_ERR_WORKSPACE;
    a.ws = static_cast<float*>(workspace);
  }
  for (int i = 0; i < 2; ++i) {
    all[i] = dy[i];
    all[2 + i] = x[i];
    all[4 + i] = out[i];
  }
  // Without any gamma it is the forward of dy with the angles turned round.
  const bool norm = a.side[0].gamma != nullptr || a.side[1].gamma != nullptr;
  if (!norm) a.scale_s = -a.scale_s;
  RopePlan p;
  s = plan(c, positions, all, 6, norm, &a, &p);
  if (s != LN_OK) return s;
  const int rows = a.blocks[0] > a.blocks[1] ? a.blocks[0] : a.blocks[1];
  if (sums && workspace_bytes < (size_t)rows * 2 * head_dim * sizeof(float))
    return LN_ERR_WORKSPACE;
  void* args[] = {&a};
  cudaError_t e = cudaLaunchKernel(p.fn, dim3(p.grid), dim3(kRopeThreads), args, 0, stream);
  if (e == cudaSuccess && sums)
    e = launch_bwd_finalize(a.ws, rows, 2 * (int)head_dim, (int)head_dim, true,
                            const_cast<void*>(grads[0].p), const_cast<void*>(grads[1].p), nullptr,
                            (int)grad_dtype, stream);
  return e == cudaSuccess ? LN_OK : cuda_fail(e);
}

}  // extern "C"
