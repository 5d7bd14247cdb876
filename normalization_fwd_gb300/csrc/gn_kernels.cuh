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
// its registers; the CTA then adds up its columns in shared memory, and one
// warp a group merges the columns. Sums are fp32. Values go in pairs, which
// this part adds, multiplies and fmas in one instruction.
#pragma once

#include "common.cuh"

namespace nf {

constexpr int kGnThreads = 256;
constexpr int kGnWarps = kGnThreads / 32;
constexpr int kGnMaxTileCh = 512;   // most channels of a column tile
constexpr int kGnFwdHold = 8;       // rows a thread keeps in registers in one launch
constexpr int kGnBwdHold = 4;

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

// ---- activations, of pairs ----------------------------------------------------
__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcpf(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + e^-z) by the hardware's exponential and reciprocal (each good to
// about 2^-23, relative); an e^-z that overflows gives 0.
__device__ __forceinline__ float2 sigmoid2(float2 z) {
  const float2 t = mul2(z, splat2(-1.4426950408889634f));
  const float2 d = add2(make_float2(ex2f(t.x), ex2f(t.y)), splat2(1.f));
  return make_float2(rcpf(d.x), rcpf(d.y));
}
template <int ACT> __device__ __forceinline__ float2 act2(float2 z) {
  if (ACT == kActSilu) return mul2(z, sigmoid2(z));
  // normcdff keeps relative accuracy in the lower tail, where (1 + erf) / 2
  // cancels.
  if (ACT == kActGelu) return mul2(z, make_float2(normcdff(z.x), normcdff(z.y)));
  return z;
}
__device__ __forceinline__ float gelu_grad(float z) {
  return normcdff(z) + z * 0.3989422804f * __expf(-0.5f * z * z);
}
template <int ACT> __device__ __forceinline__ float2 act_grad2(float2 z) {
  if (ACT == kActSilu) {
    const float2 s = sigmoid2(z);
    const float2 o = fma2(s, splat2(-1.f), splat2(1.f));   // 1 - s
    return mul2(s, fma2(z, o, splat2(1.f)));
  }
  if (ACT == kActGelu) return make_float2(gelu_grad(z.x), gelu_grad(z.y));
  return splat2(1.f);
}

// ---- a thread's VEC elements, as NP pairs ---------------------------------------
// A vector of 16 bytes, or one element (whose pair has an idle second half).
template <typename T, int VEC> struct Pack {
  static constexpr int NP = VEC / 2;
  uint4 v;
  __device__ __forceinline__ void load(const T* p) { v = ld_vec(p); }
  __device__ __forceinline__ void store(T* p) const { st_vec(p, v); }
  __device__ __forceinline__ void get(float2* f) const { unpack2<T>(v, f); }
  __device__ __forceinline__ void set(const float2* f) { v = pack2<T>(f); }
  __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
};
template <typename T> struct Pack<T, 1> {
  static constexpr int NP = 1;
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = v; }
  __device__ __forceinline__ void get(float2* f) const { f[0] = make_float2(to_f(v), 0.f); }
  __device__ __forceinline__ void set(const float2* f) { v = from_f<T>(f[0].x); }
  __device__ __forceinline__ void clear() { v = from_f<T>(0.f); }
};

// Shared memory: the row lanes' sums before they are added up, and in their
// place, afterwards, the parameters of the tile's columns.
struct GnSmem {
  union {
    struct {
      float a[kGnThreads * 8];
      float b[kGnThreads * 8];
    } lane;
    float par[6][kGnMaxTileCh];
  };
  float ca[2 * kGnMaxTileCh];   // column sums, in parts, then whole
  float cb[2 * kGnMaxTileCh];
  float k[kGnMaxTileCh];        // forward: what the columns are shifted by
  float g0[kGnMaxTileCh];       // merged: mean, or c1, of the tile's groups
  float g1[kGnMaxTileCh];       // rstd, or c2
};

template <int VEC> __device__ __forceinline__ void put_pairs(float* s, const float2* f) {
  if (VEC == 1) {
    s[0] = f[0].x;
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      reinterpret_cast<float4*>(s)[i] = make_float4(f[2 * i].x, f[2 * i].y, f[2 * i + 1].x,
                                                    f[2 * i + 1].y);
  }
}
template <int VEC> __device__ __forceinline__ void get_pairs(const float* s, float2* f) {
  if (VEC == 1) {
    f[0] = make_float2(s[0], 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const float4 v = reinterpret_cast<const float4*>(s)[i];
      f[2 * i] = make_float2(v.x, v.y);
      f[2 * i + 1] = make_float2(v.z, v.w);
    }
  }
}

// ---- geometry -----------------------------------------------------------------
// One CTA's share of a panel (a sample's column tile): a slice of its rows;
// and a thread's place in it.
struct GnUnit {
  int n, tile, slice;
  int c0, nc;            // first channel, number of channels of the tile
  int g0, ng;            // its groups
  int64_t r0, nr;        // rows of the slice
  int tc;                // channels of a full tile
  int TY;                // row lanes
  int tx, ty;            // the thread's vector and row lane
  int rows;              // its rows
  bool on;               // it has a vector
};
template <int VEC>
__device__ __forceinline__ GnUnit gn_unit(const GnArgs& a, int panel, int slice) {
  GnUnit u;
  u.n = panel / a.tiles;
  u.tile = panel - u.n * a.tiles;
  u.slice = slice;
  u.tc = a.tw * VEC;
  u.c0 = u.tile * u.tc;
  u.nc = min(a.channels - u.c0, u.tc);
  u.g0 = u.c0 / a.cpg;
  u.ng = (u.c0 + u.nc - 1) / a.cpg - u.g0 + 1;
  u.r0 = min(a.rows, (int64_t)slice * a.slice_rows);   // a cluster's last CTAs may have none
  u.nr = min(a.rows - u.r0, a.slice_rows);
  u.TY = kGnThreads / a.tw;
  u.ty = threadIdx.x / a.tw;
  u.tx = threadIdx.x - u.ty * a.tw;
  u.on = u.ty < u.TY && u.tx * VEC < u.nc;
  u.rows = u.on && u.nr > u.ty ? (int)((u.nr - u.ty - 1) / u.TY) + 1 : 0;
  return u;
}
// Where a thread's first row of a tensor starts.
template <typename T, int VEC>
__device__ __forceinline__ int64_t gn_at(const GnUnit& u, int64_t sample, int64_t row) {
  return u.n * sample + (u.r0 + u.ty) * row + u.c0 + u.tx * VEC;
}

// gamma (as w) or beta of one channel of the tile.
template <typename T>
__device__ __forceinline__ float gn_weight(const GnArgs& a, const GnUnit& u, int col) {
  if (a.gamma == nullptr) return 1.f;
  const float g = to_f(static_cast<const T*>(a.gamma)[u.n * a.param_sample + u.c0 + col]);
  return a.zero_centered ? 1.f + g : g;
}
template <typename T>
__device__ __forceinline__ float gn_bias(const GnArgs& a, const GnUnit& u, int col) {
  if (a.beta == nullptr) return 0.f;
  return to_f(static_cast<const T*>(a.beta)[u.n * a.param_sample + u.c0 + col]);
}

// ---- column sums ------------------------------------------------------------------
// Add up two quantities of every column over the row lanes: each column's
// lanes are dealt to as many threads as there are, then those parts are
// added; the order depends on the launch's shape only. Returns with the
// totals of column `col` in sm.ca, sm.cb after the caller's next barrier, via
// `done(col, a, b)`.
template <int VEC, typename F>
__device__ __forceinline__ void gn_columns(const GnUnit& u, GnSmem& sm, const float2* va,
                                           const float2* vb, F&& done) {
  if (u.on) {
    put_pairs<VEC>(sm.lane.a + u.ty * u.tc + u.tx * VEC, va);
    put_pairs<VEC>(sm.lane.b + u.ty * u.tc + u.tx * VEC, vb);
  }
  __syncthreads();
  const int parts = kGnThreads / u.tc;   // threads a column
  if (parts > 1) {
    const int part = threadIdx.x / u.tc, col = threadIdx.x - part * u.tc;
    if (part < parts && col < u.nc) {
      float sa = 0.f, sb = 0.f;
      for (int y = part; y < u.TY; y += parts) {
        sa += sm.lane.a[y * u.tc + col];
        sb += sm.lane.b[y * u.tc + col];
      }
      sm.ca[threadIdx.x] = sa;
      sm.cb[threadIdx.x] = sb;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < u.nc; c += kGnThreads) {
      float sa = 0.f, sb = 0.f;
      for (int p = 0; p < parts; ++p) {
        sa += sm.ca[p * u.tc + c];
        sb += sm.cb[p * u.tc + c];
      }
      done(c, sa, sb);
    }
  } else {
    for (int c = threadIdx.x; c < u.nc; c += kGnThreads) {
      float sa = 0.f, sb = 0.f;
      for (int y = 0; y < u.TY; ++y) {
        sa += sm.lane.a[y * u.tc + c];
        sb += sm.lane.b[y * u.tc + c];
      }
      done(c, sa, sb);
    }
  }
}

// ---- forward: partial statistics of one unit -------------------------------------
// Each column is summed as d = x - k and d^2, k the column's value in the
// slice's first row. k is one of the data, so (mean - k)^2 is itself a term
// of the variance: with n rows a slice, cancellation in s2 - s1^2 / n costs
// at most about n * 2^-24 of the group's sum of squares, whatever the mean.
// Columns, and later slices, are merged by the parallel-variance identity
// M2 = sum M2_i + n_i (mean_i - mean)^2. The first HOLD rows stay in `held`.
template <typename T, int VEC, int HOLD>
__device__ __forceinline__ void gn_stats_unit(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                              Pack<T, VEC>* held, float2* out) {
  constexpr int NP = Pack<T, VEC>::NP;
  float2 k[NP], s1[NP], s2[NP], v[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) k[i] = s1[i] = s2[i] = splat2(0.f);
  const T* p = static_cast<const T*>(a.x) + gn_at<T, VEC>(u, a.x_sample, a.x_row);
  const int64_t step = (int64_t)u.TY * a.x_row;
  if (u.rows > 0) {
    Pack<T, VEC> first;
    first.load(p - u.ty * a.x_row);
#pragma unroll
    for (int j = 0; j < HOLD; ++j)
      if (j < u.rows) held[j].load(p + j * step);
    first.get(k);
    auto add = [&](const Pack<T, VEC>& q) {
      q.get(v);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float2 d = fma2(k[i], splat2(-1.f), v[i]);
        s1[i] = add2(s1[i], d);
        s2[i] = fma2(d, d, s2[i]);
      }
    };
#pragma unroll
    for (int j = 0; j < HOLD; ++j)
      if (j < u.rows) add(held[j]);
    int r = HOLD;
    p += HOLD * step;
    constexpr int UN = HOLD > 0 ? 4 : 8;
    for (; r + UN <= u.rows; r += UN, p += UN * step) {
      Pack<T, VEC> q[UN];
#pragma unroll
      for (int j = 0; j < UN; ++j) q[j].load(p + j * step);
#pragma unroll
      for (int j = 0; j < UN; ++j) add(q[j]);
    }
    for (; r < u.rows; ++r, p += step) {
      Pack<T, VEC> q;
      q.load(p);
      add(q);
    }
  }
  if (u.on && u.ty == 0) put_pairs<VEC>(sm.k + u.tx * VEC, k);
  const float n = (float)u.nr, inv = u.nr > 0 ? 1.f / n : 0.f;
  gn_columns<VEC>(u, sm, s1, s2, [&](int c, float sa, float sb) {
    const float m = sa * inv;
    sm.ca[c] = sm.k[c] + m;    // the part this thread has just read, or nobody's
    sm.cb[c] = fmaf(-sa, m, sb);
  });
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int lg = threadIdx.x >> 5; lg < u.ng; lg += kGnWarps) {
    const int cs = max((u.g0 + lg) * a.cpg - u.c0, 0);
    const int ce = min((u.g0 + lg + 1) * a.cpg - u.c0, u.nc);
    // Means are averaged as differences from one of them, which keeps a
    // constant group's mean exact and a large common mean out of the sum.
    const float base = sm.ca[cs];
    float s = 0.f;
    for (int c = cs + lane; c < ce; c += 32) s += sm.ca[c] - base;
    const float m = base + group_sum<32>(s) / (float)(ce - cs);
    s = 0.f;
    for (int c = cs + lane; c < ce; c += 32) {
      const float d = sm.ca[c] - m;
      s += fmaf(n * d, d, sm.cb[c]);
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
template <bool BWD>
__device__ __forceinline__ void gn_combine(const GnArgs& a, const GnUnit& u, GnSmem& sm) {
  const int lane = threadIdx.x & 31;
  for (int lg = threadIdx.x >> 5; lg < u.ng; lg += kGnWarps) {
    const int g = u.g0 + lg, ch0 = g * a.cpg, ch1 = ch0 + a.cpg;
    const int t0 = ch0 / u.tc, t1 = (ch1 - 1) / u.tc;
    float s0 = 0.f, s1 = 0.f, base = 0.f;
    if (!BWD)   // the mean of the first slice of the group's first tile
      base = a.part[((int64_t)u.n * a.tiles + t0) * a.slices * a.max_groups + g -
                    t0 * u.tc / a.cpg].x;
    for (int t = t0; t <= t1; ++t) {
      const int nc = min(ch1, (t + 1) * u.tc) - max(ch0, t * u.tc);
      const float2* p = a.part + ((int64_t)u.n * a.tiles + t) * a.slices * a.max_groups +
                        (g - t * u.tc / a.cpg);
#pragma unroll 4
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
        const int nc = min(ch1, (t + 1) * u.tc) - max(ch0, t * u.tc);
        const float2* p = a.part + ((int64_t)u.n * a.tiles + t) * a.slices * a.max_groups +
                          (g - t * u.tc / a.cpg);
#pragma unroll 4
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
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(far)
               : "memory");
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
      const bool some = lane < a.slices && nr > 0;
      const float cnt = some ? (float)nr * (float)a.cpg : 0.f;
      s0 = base + group_sum<32>(some ? cnt * (v.x - base) : 0.f) * a.inv_m;
      const float d = v.x - s0;
      s1 = group_sum<32>(some ? fmaf(cnt * d, d, v.y) : 0.f) * a.inv_m;
    }
    if (lane == 0) gn_merged<BWD>(a, u, sm, lg, s0, s1, u.slice == 0);
  }
  __syncthreads();
}

// ---- forward: normalize one unit -------------------------------------------------
template <typename T, int VEC, int ACT, int HOLD>
__device__ __forceinline__ void gn_apply_unit(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                              const Pack<T, VEC>* held) {
  constexpr int NP = Pack<T, VEC>::NP;
  for (int c = threadIdx.x; c < u.nc; c += kGnThreads) {
    const int lg = (u.c0 + c) / a.cpg - u.g0;
    sm.par[0][c] = -sm.g0[lg];
    sm.par[1][c] = gn_weight<T>(a, u, c) * sm.g1[lg];
    sm.par[2][c] = gn_bias<T>(a, u, c);
  }
  __syncthreads();
  if (u.rows > 0) {
    float2 m[NP], w[NP], b[NP], v[NP];
    get_pairs<VEC>(sm.par[0] + u.tx * VEC, m);
    get_pairs<VEC>(sm.par[1] + u.tx * VEC, w);
    get_pairs<VEC>(sm.par[2] + u.tx * VEC, b);
    const T* p = static_cast<const T*>(a.x) + gn_at<T, VEC>(u, a.x_sample, a.x_row);
    T* o = static_cast<T*>(a.out) + gn_at<T, VEC>(u, a.out_sample, a.out_row);
    const int64_t step = (int64_t)u.TY * a.x_row, ostep = (int64_t)u.TY * a.out_row;
    auto put = [&](const Pack<T, VEC>& q, T* to) {
      q.get(v);
#pragma unroll
      for (int i = 0; i < NP; ++i) v[i] = act2<ACT>(fma2(add2(v[i], m[i]), w[i], b[i]));
      Pack<T, VEC> r;
      r.set(v);
      r.store(to);
    };
#pragma unroll
    for (int j = 0; j < HOLD; ++j)
      if (j < u.rows) put(held[j], o + j * ostep);
    int r = HOLD;
    p += HOLD * step;
    o += HOLD * ostep;
    constexpr int UN = 4;
    for (; r + UN <= u.rows; r += UN, p += UN * step, o += UN * ostep) {
      Pack<T, VEC> q[UN];
#pragma unroll
      for (int j = 0; j < UN; ++j) q[j].load(p + j * step);
#pragma unroll
      for (int j = 0; j < UN; ++j) put(q[j], o + j * ostep);
    }
    for (; r < u.rows; ++r, p += step, o += ostep) {
      Pack<T, VEC> q;
      q.load(p);
      put(q, o);
    }
  }
}

// ---- backward ------------------------------------------------------------------------
// What a thread keeps of its first rows: x, and dz in fp32 (dy itself where
// there is no activation), so that the activation's slope is not taken twice.
template <typename T, int VEC, int ACT> struct Held {
  Pack<T, VEC> x;
  float2 dz[Pack<T, VEC>::NP];
};
template <typename T, int VEC> struct Held<T, VEC, kActNone> {
  Pack<T, VEC> x, dy;
};

// mean, rstd, w and beta of the unit's columns.
template <typename T>
__device__ __forceinline__ void gn_bwd_params(const GnArgs& a, const GnUnit& u, GnSmem& sm) {
  for (int c = threadIdx.x; c < u.nc; c += kGnThreads) {
    const int64_t g = (int64_t)u.n * a.groups + (u.c0 + c) / a.cpg;
    sm.par[0][c] = -a.mean[g];
    sm.par[1][c] = a.rstd[g];
    sm.par[2][c] = gn_weight<T>(a, u, c);
    sm.par[3][c] = gn_bias<T>(a, u, c);
  }
}

// Sums of one unit.
template <typename T, int VEC, int ACT, int HOLD>
__device__ __forceinline__ void gn_bwd_stats_unit(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                                  Held<T, VEC, ACT>* held, float2* out) {
  constexpr int NP = Pack<T, VEC>::NP;
  float2 sa[NP], sb[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) sa[i] = sb[i] = splat2(0.f);
  const T* p = static_cast<const T*>(a.x) + gn_at<T, VEC>(u, a.x_sample, a.x_row);
  const T* q = static_cast<const T*>(a.dy) + gn_at<T, VEC>(u, a.dy_sample, a.dy_row);
  const int64_t ps = (int64_t)u.TY * a.x_row, qs = (int64_t)u.TY * a.dy_row;
  Pack<T, VEC> hd[HOLD > 0 ? HOLD : 1];
#pragma unroll
  for (int j = 0; j < HOLD; ++j)
    if (j < u.rows) {
      held[j].x.load(p + j * ps);
      hd[j].load(q + j * qs);
    }
  gn_bwd_params<T>(a, u, sm);
  __syncthreads();
  if (u.rows > 0) {
    float2 m[NP], rs[NP], w[NP], b[NP], v[NP], d[NP];
    get_pairs<VEC>(sm.par[0] + u.tx * VEC, m);
    get_pairs<VEC>(sm.par[1] + u.tx * VEC, rs);
    get_pairs<VEC>(sm.par[2] + u.tx * VEC, w);
    get_pairs<VEC>(sm.par[3] + u.tx * VEC, b);
    auto add = [&](const Pack<T, VEC>& px, const Pack<T, VEC>& pd) {   // leaves dz in d
      px.get(v);
      pd.get(d);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float2 xh = mul2(add2(v[i], m[i]), rs[i]);
        if (ACT != kActNone) d[i] = mul2(d[i], act_grad2<ACT>(fma2(xh, w[i], b[i])));
        sa[i] = add2(sa[i], d[i]);
        sb[i] = fma2(d[i], xh, sb[i]);
      }
    };
#pragma unroll
    for (int j = 0; j < HOLD; ++j)
      if (j < u.rows) {
        add(held[j].x, hd[j]);
        if constexpr (ACT == kActNone) {
          held[j].dy = hd[j];
        } else {
#pragma unroll
          for (int i = 0; i < NP; ++i) held[j].dz[i] = d[i];
        }
      }
    int r = HOLD;
    p += HOLD * ps;
    q += HOLD * qs;
    constexpr int UN = 4;
    for (; r + UN <= u.rows; r += UN, p += UN * ps, q += UN * qs) {
      Pack<T, VEC> px[UN], pd[UN];
#pragma unroll
      for (int j = 0; j < UN; ++j) {
        px[j].load(p + j * ps);
        pd[j].load(q + j * qs);
      }
#pragma unroll
      for (int j = 0; j < UN; ++j) add(px[j], pd[j]);
    }
    for (; r < u.rows; ++r, p += ps, q += qs) {
      Pack<T, VEC> px, pd;
      px.load(p);
      pd.load(q);
      add(px, pd);
    }
  }
  __syncthreads();   // the parameters give way to the sums
  float* cols = a.cols + ((int64_t)u.n * a.slices + u.slice) * 2 * a.channels + u.c0;
  gn_columns<VEC>(u, sm, sa, sb, [&](int c, float ta, float tb) {
    cols[c] = tb;
    cols[a.channels + c] = ta;
    const float w = gn_weight<T>(a, u, c);
    sm.ca[c] = w * ta;
    sm.cb[c] = w * tb;
  });
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int lg = threadIdx.x >> 5; lg < u.ng; lg += kGnWarps) {
    const int cs = max((u.g0 + lg) * a.cpg - u.c0, 0);
    const int ce = min((u.g0 + lg + 1) * a.cpg - u.c0, u.nc);
    float2 s = make_float2(0.f, 0.f);
    for (int c = cs + lane; c < ce; c += 32) {
      s.x += sm.ca[c];
      s.y += sm.cb[c];
    }
    s = group_sum2<32>(s);
    if (lane == 0) out[lg] = s;
  }
  __syncthreads();
}

// dx of one unit.
template <typename T, int VEC, int ACT, int HOLD>
__device__ __forceinline__ void gn_bwd_apply_unit(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                                  const Held<T, VEC, ACT>* held) {
  constexpr int NP = Pack<T, VEC>::NP;
  gn_bwd_params<T>(a, u, sm);
  for (int c = threadIdx.x; c < u.nc; c += kGnThreads) {
    const int lg = (u.c0 + c) / a.cpg - u.g0;
    sm.par[4][c] = -sm.g0[lg];
    sm.par[5][c] = -sm.g1[lg];
  }
  __syncthreads();
  if (u.rows > 0) {
    float2 m[NP], rs[NP], w[NP], b[NP], c1[NP], c2[NP], v[NP], d[NP];
    get_pairs<VEC>(sm.par[0] + u.tx * VEC, m);
    get_pairs<VEC>(sm.par[1] + u.tx * VEC, rs);
    get_pairs<VEC>(sm.par[2] + u.tx * VEC, w);
    get_pairs<VEC>(sm.par[3] + u.tx * VEC, b);
    get_pairs<VEC>(sm.par[4] + u.tx * VEC, c1);
    get_pairs<VEC>(sm.par[5] + u.tx * VEC, c2);
    const T* p = static_cast<const T*>(a.x) + gn_at<T, VEC>(u, a.x_sample, a.x_row);
    const T* q = static_cast<const T*>(a.dy) + gn_at<T, VEC>(u, a.dy_sample, a.dy_row);
    T* o = static_cast<T*>(a.out) + gn_at<T, VEC>(u, a.out_sample, a.out_row);
    const int64_t ps = (int64_t)u.TY * a.x_row, qs = (int64_t)u.TY * a.dy_row,
                  os = (int64_t)u.TY * a.out_row;
    // The product w dz is rounded before c1 is taken off (no fma): in a group
    // of one value c1 is that very product and dx is exactly 0.
    auto put = [&](const Pack<T, VEC>& px, T* to, bool have_dz) {
      px.get(v);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float2 xh = mul2(add2(v[i], m[i]), rs[i]);
        if (ACT != kActNone && !have_dz) d[i] = mul2(d[i], act_grad2<ACT>(fma2(xh, w[i], b[i])));
        const float2 g = make_float2(__fmul_rn(w[i].x, d[i].x), __fmul_rn(w[i].y, d[i].y));
        v[i] = mul2(rs[i], fma2(xh, c2[i], add2(g, c1[i])));
      }
      Pack<T, VEC> r;
      r.set(v);
      r.store(to);
    };
#pragma unroll
    for (int j = 0; j < HOLD; ++j)
      if (j < u.rows) {
        if constexpr (ACT == kActNone) {
          held[j].dy.get(d);
        } else {
#pragma unroll
          for (int i = 0; i < NP; ++i) d[i] = held[j].dz[i];
        }
        put(held[j].x, o + j * os, true);
      }
    int r = HOLD;
    p += HOLD * ps;
    q += HOLD * qs;
    o += HOLD * os;
    constexpr int UN = 2;
    for (; r + UN <= u.rows; r += UN, p += UN * ps, q += UN * qs, o += UN * os) {
      Pack<T, VEC> px[UN], pd[UN];
#pragma unroll
      for (int j = 0; j < UN; ++j) {
        px[j].load(p + j * ps);
        pd[j].load(q + j * qs);
      }
#pragma unroll
      for (int j = 0; j < UN; ++j) {
        pd[j].get(d);
        put(px[j], o + j * os, false);
      }
    }
    for (; r < u.rows; ++r, p += ps, q += qs, o += os) {
      Pack<T, VEC> px, pd;
      px.load(p);
      pd.load(q);
      pd.get(d);
      put(px, o, false);
    }
  }
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
    gn_stats_unit<T, VEC, 0>(a, u, sm, nullptr, gn_part(a, u));
  }
  if (app0 + p < app1) {
    const GnUnit u = gn_unit<VEC>(a, app0 + p, s);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    gn_combine<false>(a, u, sm);
    gn_apply_unit<T, VEC, ACT, 0>(a, u, sm, nullptr);
  }
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnThreads)
    gn_bwd_kernel(GnArgs a, int stat0, int stat1, int app0, int app1) {
  __shared__ GnSmem sm;
  const int p = blockIdx.x / a.slices, s = blockIdx.x - p * a.slices;
  if (stat0 + p < stat1) {
    const GnUnit u = gn_unit<VEC>(a, stat0 + p, s);
    gn_bwd_stats_unit<T, VEC, ACT, 0>(a, u, sm, nullptr, gn_part(a, u));
  }
  if (app0 + p < app1) {
    const GnUnit u = gn_unit<VEC>(a, app0 + p, s);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    gn_combine<true>(a, u, sm);
    gn_bwd_apply_unit<T, VEC, ACT, 0>(a, u, sm, nullptr);
  }
}

// A panel a cluster, in one launch: the statistics, a barrier of the
// cluster, and the rows again: those that are held, then the others out of
// the L2 cache.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnThreads, 3) gn_fwd_cluster_kernel(GnArgs a) {
  __shared__ GnSmem sm;
  __shared__ float2 part[kGnMaxTileCh];
  const int p = blockIdx.x / a.slices;
  const GnUnit u = gn_unit<VEC>(a, p, blockIdx.x - p * a.slices);
  Pack<T, VEC> held[kGnFwdHold];
  gn_stats_unit<T, VEC, kGnFwdHold>(a, u, sm, held, part);
  cluster_arrive();
  cluster_wait();
  gn_combine_cluster<false>(a, u, sm, part);
  cluster_arrive();
  gn_apply_unit<T, VEC, ACT, kGnFwdHold>(a, u, sm, held);
  cluster_wait();   // no CTA leaves while another reads its partials
}

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGnThreads, 2) gn_bwd_cluster_kernel(GnArgs a) {
  __shared__ GnSmem sm;
  __shared__ float2 part[kGnMaxTileCh];
  const int p = blockIdx.x / a.slices;
  const GnUnit u = gn_unit<VEC>(a, p, blockIdx.x - p * a.slices);
  Held<T, VEC, ACT> held[kGnBwdHold];
  gn_bwd_stats_unit<T, VEC, ACT, kGnBwdHold>(a, u, sm, held, part);
  cluster_arrive();
  cluster_wait();
  gn_combine_cluster<true>(a, u, sm, part);
  cluster_arrive();
  gn_bwd_apply_unit<T, VEC, ACT, kGnBwdHold>(a, u, sm, held);
  cluster_wait();
}

}  // namespace nf
