// Group norm with an activation over channels-last activations
// x [samples, rows, channels] (Wu and He, 2018): the groups' statistics run
// over all rows and the group's channels,
//   xhat = (x - mean) * rstd, z = xhat * w + beta, y = act(z),
// and the backward needs, with dz = dy * act'(z), two sums a channel,
//   A[n, c] = sum_r dz, B[n, c] = sum_r dz * xhat,
// from which c1 = sum_{c in group} w A / M, c2 = sum_{c in group} w B / M,
//   dx = rstd * (w dz - c1 - xhat c2), dgamma = sum_n B, dbeta = sum_n A.
//
// A thread owns one 16-byte vector of channels (one element where rows are
// not 16-byte aligned) for the whole launch, so every sum over rows stays in
// its registers and the channel parameters are loaded once. Sums are fp32.
#pragma once

#include "common.cuh"

namespace nf {

constexpr int kGnThreads = 256;
constexpr int kGnWarps = kGnThreads / 32;
constexpr int kGnMaxTileCh = 512;   // most channels of a column tile

constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2;

// Arguments of the group norm kernels (validated on the host).
struct GnArgs {
  const void* x;
  const void* dy;        // backward
  const void* gamma;     // nullable: 1
  const void* beta;      // nullable: 0
  void* out;             // y, or dx
  float* mean;           // [samples, groups]; forward: output, nullable
  float* rstd;
  float2* part;          // [panel][slice][max_groups] partials of the groups
  float* cols;           // backward: [sample][slice][2 * channels] B, then A
  int64_t x_sample, x_row, dy_sample, dy_row, out_sample, out_row;   // elements
  int64_t param_sample;  // elements between samples of gamma / beta, 0 = shared
  int64_t rows;
  int64_t slice_rows;
  int slices;
  int channels;
  int cpg;               // channels of a group
  int groups;
  int tiles;             // column tiles
  int tw;                // vectors of a column tile
  int max_groups;        // most groups that meet one tile
  float eps;
  float inv_m;           // 1 / (rows * cpg)
  int zero_centered;
};

// ---- activations ------------------------------------------------------------
// sigmoid by the hardware exponential and division (a few 2^-23 relative);
// e^-z may overflow to infinity, which gives 0.
__device__ __forceinline__ float sigmoid_f(float z) {
  return __fdividef(1.f, 1.f + __expf(-z));
}
template <int ACT> __device__ __forceinline__ float act_f(float z) {
  if (ACT == kActSilu) return __fdividef(z, 1.f + __expf(-z));
  // normcdff keeps relative accuracy in the lower tail, where (1 + erf) / 2
  // cancels.
  if (ACT == kActGelu) return z * normcdff(z);
  return z;
}
template <int ACT> __device__ __forceinline__ float act_grad_f(float z) {
  if (ACT == kActSilu) {
    const float s = sigmoid_f(z);
    return s * (1.f + z * (1.f - s));
  }
  if (ACT == kActGelu) return normcdff(z) + z * 0.3989422804f * __expf(-0.5f * z * z);
  return 1.f;
}

// ---- loads and stores of VEC elements ---------------------------------------
template <typename T, int VEC> struct Pack;
template <typename T> struct Pack<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = v; }
  __device__ __forceinline__ void get(float* f) const { f[0] = to_f(v); }
  __device__ __forceinline__ void set(const float* f) { v = from_f<T>(f[0]); }
};
template <typename T> struct PackVec {
  uint4 v;
  __device__ __forceinline__ void load(const T* p) { v = ld_vec(p); }
  __device__ __forceinline__ void store(T* p) const { st_vec(p, v); }
  __device__ __forceinline__ void get(float* f) const { unpack<T>(v, f); }
  __device__ __forceinline__ void set(const float* f) { v = pack<T>(f); }
};
template <> struct Pack<float, 4> : PackVec<float> {};
template <> struct Pack<bf16, 8> : PackVec<bf16> {};
template <> struct Pack<f16, 8> : PackVec<f16> {};

// ---- geometry -----------------------------------------------------------------
// One CTA's share of a panel (a sample's column tile): a slice of its rows.
struct GnUnit {
  int n, tile, slice;
  int c0, c1;            // channels of the tile
  int g0, ng;            // its groups
  int64_t r0, r1;        // rows of the slice
};
template <int VEC>
__device__ __forceinline__ GnUnit gn_unit(const GnArgs& a, int panel, int slice) {
  GnUnit u;
  u.n = panel / a.tiles;
  u.tile = panel - u.n * a.tiles;
  u.slice = slice;
  u.c0 = u.tile * a.tw * VEC;
  u.c1 = min(a.channels, u.c0 + a.tw * VEC);
  u.g0 = u.c0 / a.cpg;
  u.ng = (u.c1 - 1) / a.cpg - u.g0 + 1;
  u.r0 = min(a.rows, (int64_t)slice * a.slice_rows);   // a cluster's last CTAs may have none
  u.r1 = min(a.rows, u.r0 + a.slice_rows);
  return u;
}

// The rows a thread of row lane `ty` (of TY) takes from n rows.
__device__ __forceinline__ int gn_lane_rows(int64_t n, int ty, int TY) {
  return n > ty ? (int)((n - ty - 1) / TY) + 1 : 0;
}

// Channel parameters of a thread: w and beta of its VEC channels.
template <typename T, int VEC>
__device__ __forceinline__ void gn_params(const GnArgs& a, int n, int c, float* w, float* b) {
  float g[VEC];
  Pack<T, VEC> p;
  if (a.gamma != nullptr) {
    p.load(static_cast<const T*>(a.gamma) + n * a.param_sample + c);
    p.get(g);
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    w[i] = a.gamma == nullptr ? 1.f : (a.zero_centered ? 1.f + g[i] : g[i]);
  if (a.beta != nullptr) {
    p.load(static_cast<const T*>(a.beta) + n * a.param_sample + c);
    p.get(b);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) b[i] = 0.f;
  }
}

struct GnSmem {
  float a[kGnThreads * 8];
  float b[kGnThreads * 8];
  float g0[kGnMaxTileCh];       // merged: mean, or c1, of the tile's groups
  float g1[kGnMaxTileCh];       // rstd, or c2
};

// ---- forward: partial statistics of one unit -------------------------------------
// Each thread sums d = x - K and d^2 per channel, K the channel's first value
// in its rows. K is one of the data, so (mean - K)^2 is itself a term of the
// variance: with n_t rows a thread, cancellation in s2 - s1^2 / n_t costs at
// most about n_t * 2^-24 of the group's sum of squares, whatever the mean.
// The threads' (mean, M2) are merged by the parallel-variance identity
// M2 = sum M2_i + n_i (mean_i - mean)^2.
template <typename T, int VEC>
__device__ __forceinline__ void gn_stats_unit(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                              float2* out) {
  const int tx = threadIdx.x % a.tw, ty = threadIdx.x / a.tw, TY = kGnThreads / a.tw;
  const int c = u.c0 + tx * VEC;
  const bool on = ty < TY && c < u.c1;
  const int64_t n_rows = u.r1 - u.r0;
  if (on) {
    const T* p = static_cast<const T*>(a.x) + (int64_t)u.n * a.x_sample + (u.r0 + ty) * a.x_row + c;
    const int64_t step = (int64_t)TY * a.x_row;
    const int rows = gn_lane_rows(n_rows, ty, TY);
    float k[VEC], s1[VEC], s2[VEC], v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) k[i] = s1[i] = s2[i] = 0.f;
    if (rows > 0) {
      Pack<T, VEC> q;
      q.load(p);
      q.get(k);
    }
    int r = 0;
    for (; r + 4 <= rows; r += 4) {
      Pack<T, VEC> q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j].load(p + j * step);
      p += 4 * step;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        q[j].get(v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float d = v[i] - k[i];
          s1[i] += d;
          s2[i] = fmaf(d, d, s2[i]);
        }
      }
    }
    for (; r < rows; ++r, p += step) {
      Pack<T, VEC> q;
      q.load(p);
      q.get(v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float d = v[i] - k[i];
        s1[i] += d;
        s2[i] = fmaf(d, d, s2[i]);
      }
    }
    const float inv = rows > 0 ? 1.f / (float)rows : 0.f;
    const int at = ty * (a.tw * VEC) + tx * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float m = s1[i] * inv;
      sm.a[at + i] = k[i] + m;
      sm.b[at + i] = s2[i] - s1[i] * m;
    }
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int lg = threadIdx.x >> 5; lg < u.ng; lg += kGnWarps) {
    const int cs = max((u.g0 + lg) * a.cpg, u.c0) - u.c0;
    const int ce = min((u.g0 + lg + 1) * a.cpg, u.c1) - u.c0;
    const int nc = ce - cs, total = nc * TY;
    // Means are averaged as differences from one of them, which keeps a
    // constant group's mean exact and a large common mean out of the sum.
    const float base = sm.a[cs];
    float s = 0.f;
    for (int e = lane; e < total; e += 32) {
      const int y = e / nc, at = y * (a.tw * VEC) + cs + (e - y * nc);
      const int k = gn_lane_rows(n_rows, y, TY);
      if (k > 0) s = fmaf((float)k, sm.a[at] - base, s);
    }
    s = group_sum<32>(s);
    const float m = n_rows > 0 ? base + s / ((float)n_rows * (float)nc) : 0.f;
    s = 0.f;
    for (int e = lane; e < total; e += 32) {
      const int y = e / nc, at = y * (a.tw * VEC) + cs + (e - y * nc);
      const int k = gn_lane_rows(n_rows, y, TY);
      const float d = sm.a[at] - m;
      if (k > 0) s += fmaf((float)k * d, d, sm.b[at]);
    }
    s = group_sum<32>(s);
    if (lane == 0) out[lg] = make_float2(m, s);
  }
  __syncthreads();
}

// What the merged sums become: mean and rstd (forward, stored by one CTA of
// the group's), or c1 and c2.
template <bool BWD>
__device__ __forceinline__ void gn_merged(const GnArgs& a, const GnUnit& u, GnSmem& sm, int lg,
                                          float s0, float s1, bool store) {
  if (!BWD) {
    if (s1 < 0.f) s1 = 0.f;   // rounding alone; a NaN stays one
    s1 = 1.f / sqrtf(s1 + a.eps);
    if (store) {
      const int64_t g = (int64_t)u.n * a.groups + u.g0 + lg;
      if (a.mean != nullptr) a.mean[g] = s0;
      if (a.rstd != nullptr) a.rstd[g] = s1;
    }
  }
  sm.g0[lg] = s0;
  sm.g1[lg] = s1;
}

// Merge the partials of the unit's groups into sm.g0 = mean, sm.g1 = rstd
// (forward) or into sm.g0 = c1, sm.g1 = c2 (backward): one warp a group, the
// slices dealt to its lanes, the same order in every CTA.
template <int VEC, bool BWD>
__device__ __forceinline__ void gn_combine(const GnArgs& a, const GnUnit& u, GnSmem& sm) {
  const int lane = threadIdx.x & 31;
  const int tc = a.tw * VEC;
  for (int lg = threadIdx.x >> 5; lg < u.ng; lg += kGnWarps) {
    const int g = u.g0 + lg, ch0 = g * a.cpg, ch1 = ch0 + a.cpg;
    const int t0 = ch0 / tc, t1 = (ch1 - 1) / tc;
    float s0 = 0.f, s1 = 0.f, base = 0.f;
    if (!BWD)   // the mean of the first slice of the group's first tile
      base = a.part[((int64_t)u.n * a.tiles + t0) * a.slices * a.max_groups + g - t0 * tc / a.cpg].x;
    for (int t = t0; t <= t1; ++t) {
      const int nc = min(ch1, (t + 1) * tc) - max(ch0, t * tc);
      const float2* p = a.part + ((int64_t)u.n * a.tiles + t) * a.slices * a.max_groups +
                        (g - t * tc / a.cpg);
      for (int i = lane; i < a.slices; i += 32) {
        const float2 v = p[(int64_t)i * a.max_groups];
        if (BWD) {
          s0 += v.x;
          s1 += v.y;
        } else {
          const int64_t nr = min(a.slice_rows, a.rows - i * a.slice_rows);
          s0 = fmaf((float)nr * (float)nc, v.x - base, s0);
        }
      }
    }
    s0 = base + group_sum<32>(s0) * a.inv_m;
    if (BWD) {
      s1 = group_sum<32>(s1) * a.inv_m;
    } else {
      for (int t = t0; t <= t1; ++t) {
        const int nc = min(ch1, (t + 1) * tc) - max(ch0, t * tc);
        const float2* p = a.part + ((int64_t)u.n * a.tiles + t) * a.slices * a.max_groups +
                          (g - t * tc / a.cpg);
        for (int i = lane; i < a.slices; i += 32) {
          const float2 v = p[(int64_t)i * a.max_groups];
          const int64_t nr = min(a.slice_rows, a.rows - i * a.slice_rows);
          const float d = v.x - s0;
          s1 += fmaf((float)nr * (float)nc * d, d, v.y);
        }
      }
      s1 = group_sum<32>(s1) * a.inv_m;
    }
    if (lane == 0) gn_merged<BWD>(a, u, sm, lg, s0, s1, u.slice == 0 && u.tile == t0);
  }
  __syncthreads();
}

// ---- clusters -----------------------------------------------------------------------
// A thread-block cluster shares a panel: its CTAs are the slices, and the
// partials stay in their shared memory, read from one another.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float2 cluster_read(const float2* p, int rank) {
  const unsigned at = (unsigned)__cvta_generic_to_shared(p);
  unsigned far;
  float2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(far) : "memory");
  return v;
}

// The merge of gn_combine over the cluster's CTAs: a lane a CTA.
template <bool BWD>
__device__ __forceinline__ void gn_combine_cluster(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                                   const float2* part) {
  const int lane = threadIdx.x & 31;
  for (int lg = threadIdx.x >> 5; lg < u.ng; lg += kGnWarps) {
    float2 v = make_float2(0.f, 0.f);
    if (lane < a.slices) v = cluster_read(part + lg, lane);
    float s0, s1;
    if (BWD) {
      s0 = group_sum<32>(v.x) * a.inv_m;
      s1 = group_sum<32>(v.y) * a.inv_m;
    } else {
      const float base = __shfl_sync(0xffffffffu, v.x, 0);
      const int64_t nr = min(a.slice_rows, a.rows - lane * a.slice_rows);
      const float cnt = lane < a.slices && nr > 0 ? (float)nr * (float)a.cpg : 0.f;
      s0 = base + group_sum<32>(cnt * (lane < a.slices ? v.x - base : 0.f)) * a.inv_m;
      const float d = v.x - s0;
      s1 = group_sum<32>(lane < a.slices ? fmaf(cnt * d, d, v.y) : 0.f) * a.inv_m;
    }
    if (lane == 0) gn_merged<BWD>(a, u, sm, lg, s0, s1, u.slice == 0);
  }
  __syncthreads();
}

// ---- forward: normalize one unit -------------------------------------------------
template <typename T, int VEC, int ACT>
__device__ __forceinline__ void gn_apply_unit(const GnArgs& a, const GnUnit& u, GnSmem& sm) {
  const int tx = threadIdx.x % a.tw, ty = threadIdx.x / a.tw, TY = kGnThreads / a.tw;
  const int c = u.c0 + tx * VEC;
  if (ty < TY && c < u.c1) {
    float m[VEC], w[VEC], b[VEC], v[VEC];
    gn_params<T, VEC>(a, u.n, c, w, b);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int lg = (c + i) / a.cpg - u.g0;
      m[i] = sm.g0[lg];
      w[i] *= sm.g1[lg];
    }
    const T* p = static_cast<const T*>(a.x) + (int64_t)u.n * a.x_sample + (u.r0 + ty) * a.x_row + c;
    T* o = static_cast<T*>(a.out) + (int64_t)u.n * a.out_sample + (u.r0 + ty) * a.out_row + c;
    const int64_t step = (int64_t)TY * a.x_row, ostep = (int64_t)TY * a.out_row;
    const int rows = gn_lane_rows(u.r1 - u.r0, ty, TY);
    int r = 0;
    for (; r + 4 <= rows; r += 4) {
      Pack<T, VEC> q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j].load(p + j * step);
      p += 4 * step;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        q[j].get(v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = act_f<ACT>(fmaf(v[i] - m[i], w[i], b[i]));
        q[j].set(v);
        q[j].store(o + j * ostep);
      }
      o += 4 * ostep;
    }
    for (; r < rows; ++r, p += step, o += ostep) {
      Pack<T, VEC> q;
      q.load(p);
      q.get(v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = act_f<ACT>(fmaf(v[i] - m[i], w[i], b[i]));
      q.set(v);
      q.store(o);
    }
  }
  __syncthreads();
}

// ---- backward: sums of one unit ----------------------------------------------------
template <typename T, int VEC, int ACT>
__device__ __forceinline__ void gn_bwd_stats_unit(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                                  float2* out) {
  const int tx = threadIdx.x % a.tw, ty = threadIdx.x / a.tw, TY = kGnThreads / a.tw;
  const int tc = a.tw * VEC;
  const int c = u.c0 + tx * VEC;
  const bool on = ty < TY && c < u.c1;
  if (on) {
    float m[VEC], rs[VEC], w[VEC], b[VEC], sa[VEC], sb[VEC], v[VEC], d[VEC];
    gn_params<T, VEC>(a, u.n, c, w, b);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int64_t g = (int64_t)u.n * a.groups + (c + i) / a.cpg;
      m[i] = a.mean[g];
      rs[i] = a.rstd[g];
      sa[i] = sb[i] = 0.f;
    }
    const T* p = static_cast<const T*>(a.x) + (int64_t)u.n * a.x_sample + (u.r0 + ty) * a.x_row + c;
    const T* q = static_cast<const T*>(a.dy) + (int64_t)u.n * a.dy_sample + (u.r0 + ty) * a.dy_row + c;
    const int64_t ps = (int64_t)TY * a.x_row, qs = (int64_t)TY * a.dy_row;
    const int rows = gn_lane_rows(u.r1 - u.r0, ty, TY);
    int r = 0;
    auto add = [&](const Pack<T, VEC>& px, const Pack<T, VEC>& pd) {
      px.get(v);
      pd.get(d);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float xh = (v[i] - m[i]) * rs[i];
        const float dz = d[i] * act_grad_f<ACT>(fmaf(xh, w[i], b[i]));
        sa[i] += dz;
        sb[i] = fmaf(dz, xh, sb[i]);
      }
    };
    for (; r + 2 <= rows; r += 2) {
      Pack<T, VEC> px[2], pd[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        px[j].load(p + j * ps);
        pd[j].load(q + j * qs);
      }
      p += 2 * ps;
      q += 2 * qs;
#pragma unroll
      for (int j = 0; j < 2; ++j) add(px[j], pd[j]);
    }
    if (r < rows) {
      Pack<T, VEC> px, pd;
      px.load(p);
      pd.load(q);
      add(px, pd);
    }
    const int at = ty * tc + tx * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      sm.a[at + i] = sa[i];
      sm.b[at + i] = sb[i];
    }
  }
  __syncthreads();
  // Column sums over the row lanes, in their order; the first row of the
  // arrays then holds the columns' totals.
  float* cols = a.cols + ((int64_t)u.n * a.slices + u.slice) * 2 * a.channels;
  for (int k = threadIdx.x; k < u.c1 - u.c0; k += kGnThreads) {
    float ta = 0.f, tb = 0.f;
    for (int y = 0; y < TY; ++y) {
      ta += sm.a[y * tc + k];
      tb += sm.b[y * tc + k];
    }
    cols[u.c0 + k] = tb;
    cols[a.channels + u.c0 + k] = ta;
    float w = 1.f;
    if (a.gamma != nullptr) {
      w = to_f(static_cast<const T*>(a.gamma)[u.n * a.param_sample + u.c0 + k]);
      if (a.zero_centered) w += 1.f;
    }
    sm.a[k] = w * ta;
    sm.b[k] = w * tb;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int lg = threadIdx.x >> 5; lg < u.ng; lg += kGnWarps) {
    const int cs = max((u.g0 + lg) * a.cpg, u.c0) - u.c0;
    const int ce = min((u.g0 + lg + 1) * a.cpg, u.c1) - u.c0;
    float2 s = make_float2(0.f, 0.f);
    for (int k = cs + lane; k < ce; k += 32) {
      s.x += sm.a[k];
      s.y += sm.b[k];
    }
    s = group_sum2<32>(s);
    if (lane == 0) out[lg] = s;
  }
  __syncthreads();
}

// ---- backward: dx of one unit --------------------------------------------------------
template <typename T, int VEC, int ACT>
__device__ __forceinline__ void gn_bwd_apply_unit(const GnArgs& a, const GnUnit& u, GnSmem& sm) {
  const int tx = threadIdx.x % a.tw, ty = threadIdx.x / a.tw, TY = kGnThreads / a.tw;
  const int c = u.c0 + tx * VEC;
  if (ty < TY && c < u.c1) {
    float m[VEC], rs[VEC], w[VEC], b[VEC], c1[VEC], c2[VEC], v[VEC], d[VEC];
    gn_params<T, VEC>(a, u.n, c, w, b);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int lg = (c + i) / a.cpg - u.g0;
      const int64_t g = (int64_t)u.n * a.groups + u.g0 + lg;
      m[i] = a.mean[g];
      rs[i] = a.rstd[g];
      c1[i] = sm.g0[lg];
      c2[i] = sm.g1[lg];
    }
    const T* p = static_cast<const T*>(a.x) + (int64_t)u.n * a.x_sample + (u.r0 + ty) * a.x_row + c;
    const T* q = static_cast<const T*>(a.dy) + (int64_t)u.n * a.dy_sample + (u.r0 + ty) * a.dy_row + c;
    T* o = static_cast<T*>(a.out) + (int64_t)u.n * a.out_sample + (u.r0 + ty) * a.out_row + c;
    const int64_t ps = (int64_t)TY * a.x_row, qs = (int64_t)TY * a.dy_row,
                  os = (int64_t)TY * a.out_row;
    const int rows = gn_lane_rows(u.r1 - u.r0, ty, TY);
    auto put = [&](const Pack<T, VEC>& px, const Pack<T, VEC>& pd, T* to) {
      px.get(v);
      pd.get(d);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float xh = (v[i] - m[i]) * rs[i];
        const float dz = d[i] * act_grad_f<ACT>(fmaf(xh, w[i], b[i]));
        // The product is rounded before c1 is taken off (no fma): in a group
        // of one value c1 is that very product and dx is exactly 0.
        v[i] = rs[i] * fmaf(-xh, c2[i], __fmul_rn(w[i], dz) - c1[i]);
      }
      Pack<T, VEC> po;
      po.set(v);
      po.store(to);
    };
    int r = 0;
    for (; r + 2 <= rows; r += 2) {
      Pack<T, VEC> px[2], pd[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        px[j].load(p + j * ps);
        pd[j].load(q + j * qs);
      }
      p += 2 * ps;
      q += 2 * qs;
#pragma unroll
      for (int j = 0; j < 2; ++j) put(px[j], pd[j], o + j * os);
      o += 2 * os;
    }
    if (r < rows) {
      Pack<T, VEC> px, pd;
      px.load(p);
      pd.load(q);
      put(px, pd, o);
    }
  }
  __syncthreads();
}

// ---- kernels ----------------------------------------------------------------------
__device__ __forceinline__ float2* gn_part(const GnArgs& a, const GnUnit& u) {
  return a.part + (((int64_t)u.n * a.tiles + u.tile) * a.slices + u.slice) * a.max_groups;
}

// One launch takes the statistics of the panels [stat0, stat1) and applies
// those of [app0, app1), which an earlier launch gathered.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnThreads)
    gn_fwd_kernel(GnArgs a, int stat0, int stat1, int app0, int app1) {
  __shared__ GnSmem sm;
  const int p = blockIdx.x / a.slices, s = blockIdx.x - p * a.slices;
  if (stat0 + p < stat1) {
    const GnUnit u = gn_unit<VEC>(a, stat0 + p, s);
    gn_stats_unit<T, VEC>(a, u, sm, gn_part(a, u));
  }
  if (app0 + p < app1) {
    const GnUnit u = gn_unit<VEC>(a, app0 + p, s);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    gn_combine<VEC, false>(a, u, sm);
    gn_apply_unit<T, VEC, ACT>(a, u, sm);
  }
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnThreads)
    gn_bwd_kernel(GnArgs a, int stat0, int stat1, int app0, int app1) {
  __shared__ GnSmem sm;
  const int p = blockIdx.x / a.slices, s = blockIdx.x - p * a.slices;
  if (stat0 + p < stat1) {
    const GnUnit u = gn_unit<VEC>(a, stat0 + p, s);
    gn_bwd_stats_unit<T, VEC, ACT>(a, u, sm, gn_part(a, u));
  }
  if (app0 + p < app1) {
    const GnUnit u = gn_unit<VEC>(a, app0 + p, s);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    gn_combine<VEC, true>(a, u, sm);
    gn_bwd_apply_unit<T, VEC, ACT>(a, u, sm);
  }
}

// A panel a cluster, in one launch: the statistics, a barrier of the
// cluster, and the rows again, out of the L2 cache.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnThreads) gn_fwd_cluster_kernel(GnArgs a) {
  __shared__ GnSmem sm;
  __shared__ float2 part[kGnMaxTileCh];
  const int p = blockIdx.x / a.slices;
  const GnUnit u = gn_unit<VEC>(a, p, blockIdx.x - p * a.slices);
  gn_stats_unit<T, VEC>(a, u, sm, part);
  cluster_arrive();
  cluster_wait();
  gn_combine_cluster<false>(a, u, sm, part);
  cluster_arrive();
  gn_apply_unit<T, VEC, ACT>(a, u, sm);
  cluster_wait();   // no CTA leaves while another reads its partials
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnThreads) gn_bwd_cluster_kernel(GnArgs a) {
  __shared__ GnSmem sm;
  __shared__ float2 part[kGnMaxTileCh];
  const int p = blockIdx.x / a.slices;
  const GnUnit u = gn_unit<VEC>(a, p, blockIdx.x - p * a.slices);
  gn_bwd_stats_unit<T, VEC, ACT>(a, u, sm, part);
  cluster_arrive();
  cluster_wait();
  gn_combine_cluster<true>(a, u, sm, part);
  cluster_arrive();
  gn_bwd_apply_unit<T, VEC, ACT>(a, u, sm);
  cluster_wait();
}

}  // namespace nf
