// Group norm with an activation over channels-last activations
// x [samples, rows, channels] (Wu and He, 2018): the groups' statistics run
// over all rows and the group's channels,
//   xhat = (x - mean) * rstd, z = xhat * w + beta, y = act(z),
// and the backward needs, with dz = dy * act'(z), two sums a channel,
//   A[n, c] = sum_r dz, B[n, c] = sum_r dz * xhat,
// from which c1 = sum_{c in group} w A / M, c2 = sum_{c in group} w B / M,
//   dx = rstd * (w dz - c1 - xhat c2), dgamma = sum_n B, dbeta = sum_n A.
//
// A thread owns 16 bytes of channels for the whole launch, so every sum over
// rows stays in its registers; the CTA then adds up its columns in shared
// memory, and one warp a group merges the columns. Sums are fp32. Values go in
// pairs, which this part adds, multiplies and fmas in one instruction.
//
// Statistics and result need two passes over the rows. The second comes out of
// the thread's slots in shared memory or the L2 cache, so that DRAM sees each
// tensor once, except where the panels that clusters work on at a time are
// more than the cache holds (64 x 4096 x 320 fp16: 168 MB of rows at a time,
// 327 MB read for 168). No unit is full in the large cases: DRAM 56 % of its
// peak, the FMA pipe 38 % (its heavy half 45 %) in the forward and 45 % (50 %)
// in the backward, with a third and a quarter of the warps that an SM could
// have. The kernels wait, for memory and for the results of their own
// instructions, with too few warps to cover it: 80 registers and 58 KB of
// shared memory a CTA in the forward, 126 registers in the backward. Measured,
// SiLU, back to back:
//   forward  2 x 262144 x 256 bf16   137 us, 3.9 TB/s
//            16 x 1024 x 1280 bf16    26 us, 3.2 TB/s (out of the L2 cache)
//            2 x 4096 x 320 fp16      10.6 us: latency of load, merge and store
//   backward 8 x 16384 x 320 bf16     82 us, 3.1 TB/s
//            2 x 4096 x 640 fp16      20 us, 1.5 TB/s
#pragma once

#include "common.cuh"
#include "fastdiv.h"

namespace nf {

constexpr int kGnThreads = 256;
constexpr int kGnMaxTileCh = 512;   // most channels of a column tile
constexpr int kGnRing = 8;          // rows a thread has in flight, or keeps
constexpr int kGnStep = 2;          // rows of one step
constexpr int kGnMaxSlices = 512;   // most slices of a panel

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
  float2* part;          // [panel][max_groups][slice] partials of the groups
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
  int tile_ch;           // channels of a tile
  int tw;                // vectors of a tile, the last of which may be in part
  int grain;             // bytes of an access: 16, 8, 4 or 2, what rows are aligned to
  int max_groups;        // most groups that meet one tile
  FastDiv by_slices, by_tiles, by_tile_ch, by_tw, by_tc, by_ty, by_cpg;
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
// 1 / (1 + e^-z) of NP pairs. The special-function unit takes 16 lanes a
// cycle and would bound the kernels with an exponential and a reciprocal for
// each value, so four values share a reciprocal: with d = 1 + e^-z,
// 1 / d0 = d1 d2 d3 / (d0 d1 d2 d3). Where that product passes 2^126 (every z
// below -21, say), or a NaN is among the four that the others must not get,
// the thread takes the reciprocals one by one. The exponential and the
// reciprocal are good to about 2^-23, relative; an e^-z that overflows gives 0.
template <int NP> __device__ __forceinline__ void sigmoid(const float2* z, float2* s) {
  float2 d[NP];
  float prod[NP / 2 + 1];
  bool fine = NP % 2 == 0;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const float2 t = mul2(z[i], splat2(-1.4426950408889634f));
    d[i] = add2(make_float2(ex2f(t.x), ex2f(t.y)), splat2(1.f));
  }
#pragma unroll
  for (int i = 0; i + 1 < NP; i += 2) {
    s[i] = mul2(d[i], d[i + 1]);   // (d0 d2, d1 d3)
    prod[i / 2] = s[i].x * s[i].y;
    fine = fine && prod[i / 2] < 0x1p126f;
  }
  if (fine) {
#pragma unroll
    for (int i = 0; i + 1 < NP; i += 2) {
      const float2 q = mul2(make_float2(s[i].y, s[i].x), splat2(rcpf(prod[i / 2])));
      s[i] = mul2(q, d[i + 1]);
      s[i + 1] = mul2(q, d[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NP; ++i) s[i] = make_float2(rcpf(d[i].x), rcpf(d[i].y));
  }
}
// The normal distribution function of a pair, and e^(-z^2/2). Its lower tail
// is e^(-z^2/2) R(|z|), where R falls from 1/2 like 1 / (sqrt(2 pi) |z|): a
// polynomial of t = 1 / (1 + p |z|), nine terms without a constant, fitted to
// the least relative error over [0, 14.5] (2^-26). In fp32 it is good to
// 12 + 1.5 z^2 roundings, relative, in the lower tail (where (1 + erf) / 2
// would cancel). A backward over 3 x 85374 x 250 bf16 takes 266 us with it, and
// took 540 with CUDA's normcdff and an exponential.
__device__ __forceinline__ void gauss(float2 z, float2* cdf, float2* e) {
  const float2 d = fma2(make_float2(fabsf(z.x), fabsf(z.y)), splat2(0.26499999f), splat2(1.f));
  const float2 t = make_float2(rcpf(d.x), rcpf(d.y));
  const float2 h = mul2(mul2(z, z), splat2(-0.72134752f));
  *e = make_float2(ex2f(h.x), ex2f(h.y));
  float2 r = fma2(t, splat2(0.030624436f), splat2(-0.14330049f));
  r = fma2(r, t, splat2(0.21595012f));
  r = fma2(r, t, splat2(-0.11428611f));
  r = fma2(r, t, splat2(0.13655469f));
  r = fma2(r, t, splat2(0.060895126f));
  r = fma2(r, t, splat2(0.10255506f));
  r = fma2(r, t, splat2(0.10526678f));
  r = fma2(r, t, splat2(0.10574039f));
  const float2 low = mul2(mul2(r, t), *e);
  const float2 up = fma2(low, splat2(-1.f), splat2(1.f));
  *cdf = make_float2(z.x < 0.f ? low.x : up.x, z.y < 0.f ? low.y : up.y);
}
// z -> act(z) of NP pairs.
template <int ACT, int NP> __device__ __forceinline__ void activate(float2* z) {
  if (ACT == kActSilu) {
    float2 s[NP];
    sigmoid<NP>(z, s);
#pragma unroll
    for (int i = 0; i < NP; ++i) z[i] = mul2(z[i], s[i]);
  }
  if (ACT == kActGelu) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float2 c, e;
      gauss(z[i], &c, &e);
      z[i] = mul2(z[i], c);
    }
  }
}
// d -> d * act'(z) of NP pairs.
template <int ACT, int NP> __device__ __forceinline__ void through(float2* d, const float2* z) {
  if (ACT == kActSilu) {
    float2 s[NP];
    sigmoid<NP>(z, s);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float2 o = fma2(s[i], splat2(-1.f), splat2(1.f));   // 1 - s
      d[i] = mul2(d[i], mul2(s[i], fma2(z[i], o, splat2(1.f))));
    }
  }
  if (ACT == kActGelu) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float2 c, e;
      gauss(z[i], &c, &e);
      d[i] = mul2(d[i], fma2(mul2(z[i], splat2(0.39894228f)), e, c));
    }
  }
}

// ---- a thread's VEC elements, as NP pairs ---------------------------------------
// Sixteen bytes in registers, and one access in memory. FINE: rows that are
// not aligned to 16 bytes are moved `grain` bytes at a time, what they are
// aligned to, and the first `valid` elements only (all but a row's last
// vector have all of them).
template <typename T, int VEC> struct Pack {
  static constexpr int NP = VEC / 2, B = (int)sizeof(T);
  union {
    uint4 v;
    uint2 d[2];
    unsigned w[4];
    T t[VEC];
  };
  __device__ __forceinline__ Pack() {}
  template <bool FINE> __device__ __forceinline__ void load(const T* p, int grain, int valid) {
    if (!FINE) {
      v = ld_vec(p);
    } else if (B == 4 || grain > 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i * (4 / B) < valid) w[i] = reinterpret_cast<const unsigned*>(p)[i];
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < valid) t[i] = p[i];
    }
  }
  template <bool FINE>
  __device__ __forceinline__ void store(T* p, int grain, int valid) const {
    if (!FINE) {
      st_vec(p, v);
    } else if (grain == 8) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i * (8 / B) < valid) reinterpret_cast<uint2*>(p)[i] = d[i];
    } else if (B == 4 || grain == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i * (4 / B) < valid) reinterpret_cast<unsigned*>(p)[i] = w[i];
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < valid) p[i] = t[i];
    }
  }
  __device__ __forceinline__ void get(float2* f) const { unpack2<T>(v, f); }
  __device__ __forceinline__ void set(const float2* f) { v = pack2<T>(f); }
  __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
};

// Shared memory: the row lanes' sums before they are added up, and in their
// place, afterwards, the parameters of the tile's columns.
struct alignas(16) GnSmem {
  union {
    float2 lane[kGnThreads * 8];
    float par[6][kGnMaxTileCh];
  };
  float2 col[kGnMaxTileCh];   // column sums, in parts, then whole (backward)
  float n[kGnThreads / 4];      // forward: rows of the parts
  float g0[kGnMaxTileCh];       // merged: mean, or c1, of the tile's groups
  float g1[kGnMaxTileCh];       // rstd, or c2
};

template <int VEC> __device__ __forceinline__ void put_pairs(float* s, const float2* f) {
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i)
    reinterpret_cast<float4*>(s)[i] = make_float4(f[2 * i].x, f[2 * i].y, f[2 * i + 1].x,
                                                  f[2 * i + 1].y);
}
template <int VEC> __device__ __forceinline__ void get_pairs(const float* s, float2* f) {
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(s)[i];
    f[2 * i] = make_float2(v.x, v.y);
    f[2 * i + 1] = make_float2(v.z, v.w);
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
  int tc;                // places of a tile's channels, tw * VEC
  int TY;                // row lanes
  int tx, ty;            // the thread's vector and row lane
  int rows;              // its rows
  int valid;             // elements of its vector
  bool on;               // it has one
};
template <int VEC>
__device__ __forceinline__ GnUnit gn_unit(const GnArgs& a, int panel, int slice) {
  GnUnit u;
  u.n = a.by_tiles.div(panel);
  u.tile = panel - u.n * a.tiles;
  u.slice = slice;
  u.tc = a.tw * VEC;
  u.c0 = u.tile * a.tile_ch;
  u.nc = min(a.channels - u.c0, a.tile_ch);
  u.g0 = a.by_cpg.div(u.c0);
  u.ng = a.by_cpg.div(u.c0 + u.nc - 1) - u.g0 + 1;
  u.r0 = min(a.rows, (int64_t)slice * a.slice_rows);   // a cluster's last CTAs may have none
  u.nr = min(a.rows - u.r0, a.slice_rows);
  u.TY = a.by_tw.div(kGnThreads);
  u.ty = a.by_tw.div(threadIdx.x);
  u.tx = threadIdx.x - u.ty * a.tw;
  u.valid = min(u.nc - u.tx * VEC, VEC);
  u.on = u.ty < u.TY && u.valid > 0;
  u.rows = u.on && u.nr > u.ty ? a.by_ty.div((int)(u.nr - u.ty - 1)) + 1 : 0;
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
// added; the order depends on the launch's shape only. done(col, sums) gets
// the totals; where it writes sm.col[col] no other thread reads that place.
template <int VEC, typename F>
__device__ __forceinline__ void gn_columns(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                           const float2* va, const float2* vb, F&& done) {
  if (u.on) {
    float2* to = sm.lane + u.ty * u.tc + u.tx * VEC;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i)
      reinterpret_cast<float4*>(to)[i] = make_float4(va[i].x, vb[i].x, va[i].y, vb[i].y);
  }
  __syncthreads();
  const int parts = a.by_tc.div(kGnThreads);   // threads a column
  if (parts > 1) {
    const int part = a.by_tc.div(threadIdx.x), col = threadIdx.x - part * u.tc;
    if (part < parts && col < u.nc) {
      float2 s = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int y = part; y < u.TY; y += parts) s = add2(s, sm.lane[y * u.tc + col]);
      sm.col[threadIdx.x] = s;
    }
    __syncthreads();
    if (threadIdx.x < u.nc) {
      float2 s = sm.col[threadIdx.x];
#pragma unroll 2
      for (int p = 1; p < parts; ++p) s = add2(s, sm.col[p * u.tc + threadIdx.x]);
      done(threadIdx.x, s);
    }
  } else {
    for (int c = threadIdx.x; c < u.nc; c += kGnThreads) {
      float2 s = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int y = 0; y < u.TY; ++y) s = add2(s, sm.lane[y * u.tc + c]);
      done(c, s);
    }
  }
}

// ---- rows in flight -----------------------------------------------------------------
// A thread streams its vectors of one or two tensors through slots of shared
// memory that nobody else touches (so no barrier is needed, only a wait for
// its own copies): kGnRing rows are on their way at any time, in steps of
// kGnStep rows. Of a pass over more rows than that the last kGnRing stay in
// the slots, and a second pass starts with those while it fetches the others
// again. Copies are of 16, 8 or 4 bytes, by the rows' alignment; rows that are
// aligned to 2 bytes pass through registers. Eight rows: with four 16 x 1024 x
// 1280 bf16 took 29 us for 26 and 2 x 262144 x 256 took 147 for 139; with
// sixteen a CTA fewer fits an SM.
__device__ __forceinline__ void copy_async16(unsigned dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N> __device__ __forceinline__ void copy_async(unsigned dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T, int VEC, int TENSORS, bool FINE> struct Rows {
  static constexpr int NG = kGnRing / kGnStep;   // steps in flight
  const T* p[TENSORS];      // the thread's first row
  int64_t step[TENSORS];    // from one of its rows to the next
  const T* next[TENSORS];   // the next one to fetch
  int rows, steps;
  int grain, valid;         // of the copies
  int held;                 // valid elements of what is in the slots
  unsigned place;           // in the ring, of step 0
  unsigned slots;           // this thread's first slot
  Pack<T, VEC> v[TENSORS][kGnStep];

  __device__ __forceinline__ unsigned at(unsigned place) const {
    return slots + place % NG * (kGnStep * kGnThreads * 16);
  }
  // A vector, from memory into a slot.
  __device__ __forceinline__ void copy(unsigned to, const T* from) const {
    constexpr int B = (int)sizeof(T);
    if (!FINE) {
      copy_async16(to, from);
    } else if (B == 2 && grain == 2) {
      Pack<T, VEC> x;
      x.template load<true>(from, 2, valid);
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(x.v.x), "r"(x.v.y),
                   "r"(x.v.z), "r"(x.v.w)
                   : "memory");
    } else if (grain == 8) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i * (8 / B) < valid) copy_async<8>(to + 8 * i, from + i * (8 / B));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i * (4 / B) < valid) copy_async<4>(to + 4 * i, from + i * (4 / B));
    }
  }
  // Step g of n rows, into a place of the ring.
  __device__ __forceinline__ void fetch(int g, int n, unsigned place) {
    const unsigned to = at(place);
#pragma unroll
    for (int j = 0; j < kGnStep; ++j)
      if (g * kGnStep + j < n) {
#pragma unroll
        for (int t = 0; t < TENSORS; ++t) {
          copy(to + t * (kGnRing * kGnThreads * 16) + j * (kGnThreads * 16), next[t]);
          next[t] += step[t];
        }
      }
    copy_commit();
  }
  __device__ __forceinline__ void take(unsigned place) {
    const unsigned from = at(place);
#pragma unroll
    for (int t = 0; t < TENSORS; ++t)
#pragma unroll
      for (int j = 0; j < kGnStep; ++j) {
        uint4& u = v[t][j].v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "r"(from + t * (kGnRing * kGnThreads * 16) + j * (kGnThreads * 16)));
        // What is behind the row counts as 0: it shares reciprocals with the rest.
        if (FINE) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int left = held * (int)sizeof(T) - 4 * i;
            v[t][j].w[i] &= left >= 4 ? ~0u : left == 2 ? 0xffffu : 0u;
          }
        }
      }
  }
  __device__ __forceinline__ void rewind() {
#pragma unroll
    for (int t = 0; t < TENSORS; ++t) next[t] = p[t];
  }
  __device__ __forceinline__ void take_rows(int n) {
    rows = n;
    steps = (n + kGnStep - 1) / kGnStep;
  }
  // Start the first pass (or the only one) over a unit's rows.
  __device__ __forceinline__ void start(const GnArgs& a, const GnUnit& u, void* ring) {
    take_rows(u.rows);
    grain = a.grain;
    valid = held = u.valid;
    place = 0;
    slots = (unsigned)__cvta_generic_to_shared(ring) + threadIdx.x * 16;
    rewind();
#pragma unroll
    for (int g = 0; g < NG; ++g) fetch(g, rows, g);
  }
  // The thread's first row (zeros where it has none).
  __device__ __forceinline__ void first(float2* f) {
    copy_wait<NG - 1>();
    take(place);
    if (rows == 0) v[0][0].clear();
    v[0][0].get(f);
  }
  // body(j, to) for every row, j its place in v, `to` its place in an output
  // whose first row is at `o`; end(g) after step g.
  template <typename F, typename E>
  __device__ __forceinline__ void pass(T* o, int64_t ostep, F&& body, E&& end) {
    for (int g = 0; g < steps; ++g) {
      copy_wait<NG - 1>();
      take(place + g);
#pragma unroll
      for (int j = 0; j < kGnStep; ++j) {
        if (g * kGnStep + j < rows) body(j, o);
        o += ostep;
      }
      fetch(g + NG, rows, place + g);
      end(g);
    }
  }
  template <typename F> __device__ __forceinline__ void pass(T* o, int64_t ostep, F&& body) {
    pass(o, ostep, body, [](int) {});
  }
  // The second pass over the same rows, those in the slots first; places that
  // it has no more rows for take the first ones of another unit at q.
  template <typename F>
  __device__ __forceinline__ void again(T* o, int64_t ostep, F&& body, const T* const* q, int n,
                                        int n_valid) {
    const int far = steps > NG ? steps - NG : 0;   // steps that have left the slots
    rewind();
    T* const first = o;
    o += far * kGnStep * ostep;
    place += far;
    // Steps far, ..., steps - 1 out of their slots, which take 0, 1, ... after them.
    for (int k = 0; k < steps; ++k) {
      const int g = far + k < steps ? far + k : far + k - steps;
      if (g == 0) o = first;
      copy_wait<NG - 1>();
      take(place + k);
#pragma unroll
      for (int j = 0; j < kGnStep; ++j) {
        if (g * kGnStep + j < rows) body(j, o);
        o += ostep;
      }
      if (k == far) {
#pragma unroll
        for (int t = 0; t < TENSORS; ++t) next[t] = q[t];
      }
      valid = k < far ? held : n_valid;
      if (k < far) fetch(k, rows, place + k);
      else fetch(k - far, n, place + k);
    }
    if (steps == 0) {
#pragma unroll
      for (int t = 0; t < TENSORS; ++t) next[t] = q[t];
    }
    valid = n_valid;
    place += far;
#pragma unroll
    for (int g = 0; g < NG; ++g)
      if (g >= steps) fetch(g, n, place + g);
#pragma unroll
    for (int t = 0; t < TENSORS; ++t) p[t] = q[t];
    take_rows(n);
    held = n_valid;
  }
};

// ---- forward: partial statistics of one unit -------------------------------------
// A thread sums a column of its rows as d = x - k and d^2 about a k that it
// moves to the mean of its rows so far: after 8 and 32 rows, then every 32.
// With s1, s2 the sums of a block of rows, N the rows so far and t the move,
// about s1 / N, what is left is s1 - N t, and the block adds s2 - t (2 s1 - N t)
// to the column's sum of squares M2. No row is special: k begins as the
// thread's own first row, so the first block's s2 is at most 8 M2, and with b
// rows a later block Cauchy's inequality gives s1^2 / N <= s2 b / N, b / N <= 3/4,
// so that the later ones come to at most 4 M2, whatever the data. M2 is good
// to 8 * 10 + 4 * 34 roundings and one more a block, relative; measured, rstd
// is off by 9 roundings at most over rows that begin with an outlier or padding. One shift for all rows, the slice's first one, was off by 1e-3
// after an outlier and 16384 rows; it saved 0.7 us of 2 x 4096 x 320 fp16's
// 10.7 and nothing of 2 x 262144 x 256 bf16's 137.
// Row lanes, columns and slices are merged by the parallel-variance identity
// M2 = sum M2_i + n_i (mean_i - mean)^2, the mean first.
__device__ __forceinline__ bool gn_moves(int g) { return g == 3 || g % 16 == 15; }

// Merge the columns' (mean, M2) over the row lanes: each column's lanes are
// dealt to as many threads as there are, part p of column c into
// sm.col[p * tc + c] and its rows into sm.n[p]. The order depends on the
// launch's shape only. Returns the parts.
template <int VEC>
__device__ __forceinline__ int gn_merge_lanes(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                              const float2* mean, const float2* m2) {
  if (u.on) {
    float2* to = sm.lane + u.ty * u.tc + u.tx * VEC;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i)
      reinterpret_cast<float4*>(to)[i] = make_float4(mean[i].x, m2[i].x, mean[i].y, m2[i].y);
  }
  __syncthreads();
  const int each = a.by_ty.div((int)u.nr), more = (int)u.nr - each * u.TY;
  const auto merge = [&](int part, int parts, int col) {
    const auto rows = [&](int y) { return (float)(each + (y < more ? 1 : 0)); };
    const float base = sm.lane[part * u.tc + col].x;
    float n = 0.f, s = 0.f, q = 0.f;
#pragma unroll 4
    for (int y = part; y < u.TY; y += parts) {
      n += rows(y);
      s = fmaf(rows(y), sm.lane[y * u.tc + col].x - base, s);
    }
    const float m = n > 0.f ? fmaf(s, rcpf(n), base) : base;
#pragma unroll 4
    for (int y = part; y < u.TY; y += parts) {
      const float2 v = sm.lane[y * u.tc + col];
      const float d = v.x - m;
      q += fmaf(rows(y) * d, d, v.y);
    }
    sm.col[part * u.tc + col] = make_float2(m, q);
    if (col == 0) sm.n[part] = n;
  };
  const int parts = a.by_tc.div(kGnThreads);   // threads a column
  if (parts > 1) {
    const int part = a.by_tc.div(threadIdx.x), col = threadIdx.x - part * u.tc;
    if (part < parts && col < u.nc) merge(part, parts, col);
    return parts;
  }
  for (int c = threadIdx.x; c < u.nc; c += kGnThreads) merge(0, 1, c);
  return 1;
}

template <typename T, int VEC, bool FINE>
__device__ __forceinline__ void gn_stats_unit(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                              Rows<T, VEC, 1, FINE>& rows, float2* out,
                                              int stride) {
  constexpr int NP = Pack<T, VEC>::NP;
  float2 k[NP], s1[NP], s2[NP], m2[NP], v[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) s1[i] = s2[i] = m2[i] = splat2(0.f);
  rows.first(k);
  const auto move = [&](int n) {
    const float2 inv = splat2(rcpf((float)n)), neg = splat2(-(float)n);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float2 to = fma2(s1[i], inv, k[i]);
      const float2 t = fma2(k[i], splat2(-1.f), to);
      const float2 left = fma2(neg, t, s1[i]);
      const float2 sum = add2(s1[i], left);
      m2[i] = add2(m2[i], fma2(mul2(t, splat2(-1.f)), sum, s2[i]));
      k[i] = to;
      s1[i] = left;
      s2[i] = splat2(0.f);
    }
  };
  rows.pass(
      static_cast<T*>(nullptr), 0,
      [&](int j, T*) {
        rows.v[0][j].get(v);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const float2 d = fma2(k[i], splat2(-1.f), v[i]);
          s1[i] = add2(s1[i], d);
          s2[i] = fma2(d, d, s2[i]);
        }
      },
      [&](int g) {
        if (gn_moves(g) && (g + 1) * kGnStep < rows.rows) move((g + 1) * kGnStep);
      });
  if (rows.rows > 0) move(rows.rows);
  const int parts = gn_merge_lanes<VEC>(a, u, sm, k, m2);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int lg = threadIdx.x >> 5; lg < u.ng; lg += kGnThreads / 32) {
    const int cs = max((u.g0 + lg) * a.cpg - u.c0, 0);
    const int width = min((u.g0 + lg + 1) * a.cpg - u.c0, u.nc) - cs;
    // The group's columns and parts, dealt to the lanes as one list. Means are
    // averaged as differences from one of them, which keeps a constant
    // group's mean exact and a large common mean out of the sum.
    const int dp = 32 / width, dc = 32 - dp * width, p0 = lane / width, c0 = lane - p0 * width;
    const auto walk = [&](auto&& body) {
      for (int p = p0, c = c0; p < parts;) {
        body(sm.n[p], sm.col[p * u.tc + cs + c]);
        p += dp;
        c += dc;
        if (c >= width) {
          c -= width;
          ++p;
        }
      }
    };
    const float base = sm.col[cs].x;
    float s = 0.f;
    walk([&](float n, float2 v) { s = fmaf(n, v.x - base, s); });
    const float m = base + group_sum<32>(s) / ((float)u.nr * (float)width);
    s = 0.f;
    walk([&](float n, float2 v) {
      const float d = v.x - m;
      s += fmaf(n * d, d, v.y);
    });
    s = group_sum<32>(s);
    if (lane == 0) out[(int64_t)lg * stride] = make_float2(m, s);
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
// slices dealt to its lanes, the same order in every CTA. A lane has all its
// partials of a tile on their way at once and keeps them for the second sum.
template <bool BWD>
__device__ __forceinline__ void gn_combine(const GnArgs& a, const GnUnit& u, GnSmem& sm) {
  constexpr int N = kGnMaxSlices / 32;
  const int lane = threadIdx.x & 31;
  for (int lg = threadIdx.x >> 5; lg < u.ng; lg += kGnThreads / 32) {
    const int g = u.g0 + lg, ch0 = g * a.cpg, ch1 = ch0 + a.cpg;
    const int t0 = a.by_tile_ch.div(ch0), t1 = a.by_tile_ch.div(ch1 - 1);
    float s0 = 0.f, s1 = 0.f, base = 0.f;
    float2 v[N];
    const auto fetch = [&](int t) {
      const float2* p = a.part + (((int64_t)u.n * a.tiles + t) * a.max_groups +
                                  (g - a.by_cpg.div(t * a.tile_ch))) * a.slices;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        v[j] = make_float2(0.f, 0.f);
        if (lane + 32 * j < a.slices) v[j] = p[lane + 32 * j];
      }
    };
    // values of the group in slice i of tile t
    const auto count = [&](int t, int i) {
      const int nc = min(ch1, (t + 1) * a.tile_ch) - max(ch0, t * a.tile_ch);
      return (float)min(a.slice_rows, a.rows - i * a.slice_rows) * (float)nc;
    };
    for (int t = t0; t <= t1; ++t) {
      fetch(t);
      if (!BWD && t == t0) base = __shfl_sync(0xffffffffu, v[0].x, 0);
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (lane + 32 * j < a.slices) {
          s0 = BWD ? s0 + v[j].x : fmaf(count(t, lane + 32 * j), v[j].x - base, s0);
          if (BWD) s1 += v[j].y;
        }
    }
    s0 = base + group_sum<32>(s0) * a.inv_m;
    if (!BWD) {
      for (int t = t0; t <= t1; ++t) {
        if (t1 > t0) fetch(t);
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (lane + 32 * j < a.slices) {
            const float d = v[j].x - s0;
            s1 += fmaf(count(t, lane + 32 * j) * d, d, v[j].y);
          }
      }
    }
    s1 = group_sum<32>(s1) * a.inv_m;
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
__device__ __forceinline__ void gn_combine_cluster(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                                   const float2* part) {
  const int lane = threadIdx.x & 31;
  for (int lg = threadIdx.x >> 5; lg < u.ng; lg += kGnThreads / 32) {
    float2 v = make_float2(0.f, 0.f);
    if (lane < a.slices) v = cluster_read(part + lg, lane);
    const float base = __shfl_sync(0xffffffffu, v.x, 0);
    const int64_t nr = min(a.slice_rows, a.rows - lane * a.slice_rows);
    const bool some = lane < a.slices && nr > 0;
    const float cnt = some ? (float)nr * (float)a.cpg : 0.f;
    const float mean = base + group_sum<32>(some ? cnt * (v.x - base) : 0.f) * a.inv_m;
    const float d = v.x - mean;
    const float var = group_sum<32>(some ? fmaf(cnt * d, d, v.y) : 0.f) * a.inv_m;
    if (lane == 0) gn_merged<false>(a, u, sm, lg, mean, var, u.slice == 0);
  }
  __syncthreads();
}

// ---- forward: normalize one unit -------------------------------------------------
template <typename T, int VEC, int ACT, bool FINE, typename W>
__device__ __forceinline__ void gn_apply_unit(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                              Rows<T, VEC, 1, FINE>& rows, W&& walk) {
  constexpr int NP = Pack<T, VEC>::NP;
  for (int c = threadIdx.x; c < u.tc; c += kGnThreads) {
    if (c < u.nc) {
      const int lg = a.by_cpg.div(u.c0 + c) - u.g0;
      sm.par[0][c] = -sm.g0[lg];
      sm.par[1][c] = gn_weight<T>(a, u, c) * sm.g1[lg];
      sm.par[2][c] = gn_bias<T>(a, u, c);
    } else {
      sm.par[0][c] = sm.par[1][c] = sm.par[2][c] = 0.f;
    }
  }
  __syncthreads();
  float2 m[NP], w[NP], b[NP], v[NP];
  get_pairs<VEC>(sm.par[0] + u.tx * VEC, m);
  get_pairs<VEC>(sm.par[1] + u.tx * VEC, w);
  get_pairs<VEC>(sm.par[2] + u.tx * VEC, b);
  T* o = static_cast<T*>(a.out) + gn_at<T, VEC>(u, a.out_sample, a.out_row);
  const int64_t ostep = (int64_t)u.TY * a.out_row;
  auto body = [&](int j, T* to) {
    rows.v[0][j].get(v);
#pragma unroll
    for (int i = 0; i < NP; ++i) v[i] = fma2(add2(v[i], m[i]), w[i], b[i]);
    activate<ACT, NP>(v);
    Pack<T, VEC> y;
    y.set(v);
    y.template store<FINE>(to, a.grain, u.valid);
  };
  walk(o, ostep, body);
}

// ---- backward ------------------------------------------------------------------------
// mean, rstd, w and beta of the unit's columns.
template <typename T>
__device__ __forceinline__ void gn_bwd_params(const GnArgs& a, const GnUnit& u, GnSmem& sm) {
  for (int c = threadIdx.x; c < u.tc; c += kGnThreads) {
    if (c < u.nc) {
      const int64_t g = (int64_t)u.n * a.groups + a.by_cpg.div(u.c0 + c);
      sm.par[0][c] = -a.mean[g];
      sm.par[1][c] = a.rstd[g];
      sm.par[2][c] = gn_weight<T>(a, u, c);
      sm.par[3][c] = gn_bias<T>(a, u, c);
    } else {
      sm.par[0][c] = sm.par[1][c] = sm.par[2][c] = sm.par[3][c] = 0.f;
    }
  }
}

// Sums of one unit.
template <typename T, int VEC, int ACT, bool FINE>
__device__ __forceinline__ void gn_bwd_stats_unit(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                                  Rows<T, VEC, 2, FINE>& rows, float2* out,
                                                  int stride) {
  constexpr int NP = Pack<T, VEC>::NP;
  float2 sa[NP], sb[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) sa[i] = sb[i] = splat2(0.f);
  gn_bwd_params<T>(a, u, sm);
  __syncthreads();
  if (u.rows > 0) {
    float2 m[NP], rs[NP], w[NP], b[NP], v[NP], d[NP];
    get_pairs<VEC>(sm.par[0] + u.tx * VEC, m);
    get_pairs<VEC>(sm.par[1] + u.tx * VEC, rs);
    get_pairs<VEC>(sm.par[2] + u.tx * VEC, w);
    get_pairs<VEC>(sm.par[3] + u.tx * VEC, b);
    rows.pass(static_cast<T*>(nullptr), 0, [&](int j, T*) {
      rows.v[0][j].get(v);
      rows.v[1][j].get(d);
      float2 z[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        v[i] = mul2(add2(v[i], m[i]), rs[i]);
        z[i] = fma2(v[i], w[i], b[i]);
      }
      through<ACT, NP>(d, z);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        sa[i] = add2(sa[i], d[i]);
        sb[i] = fma2(d[i], v[i], sb[i]);
      }
    });
  }
  __syncthreads();   // the parameters give way to the sums
  float* cols = a.cols + ((int64_t)u.n * a.slices + u.slice) * 2 * a.channels + u.c0;
  gn_columns<VEC>(a, u, sm, sa, sb, [&](int c, float2 s) {
    cols[c] = s.y;
    cols[a.channels + c] = s.x;
    const float w = gn_weight<T>(a, u, c);
    sm.col[c] = make_float2(w * s.x, w * s.y);
  });
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int lg = threadIdx.x >> 5; lg < u.ng; lg += kGnThreads / 32) {
    const int cs = max((u.g0 + lg) * a.cpg - u.c0, 0);
    const int ce = min((u.g0 + lg + 1) * a.cpg - u.c0, u.nc);
    float2 s = make_float2(0.f, 0.f);
    for (int c = cs + lane; c < ce; c += 32) s = add2(s, sm.col[c]);
    s = group_sum2<32>(s);
    if (lane == 0) out[(int64_t)lg * stride] = s;
  }
  __syncthreads();
}

// dx of one unit.
template <typename T, int VEC, int ACT, bool FINE, typename W>
__device__ __forceinline__ void gn_bwd_apply_unit(const GnArgs& a, const GnUnit& u, GnSmem& sm,
                                                  Rows<T, VEC, 2, FINE>& rows, W&& walk) {
  constexpr int NP = Pack<T, VEC>::NP;
  gn_bwd_params<T>(a, u, sm);
  for (int c = threadIdx.x; c < u.tc; c += kGnThreads) {
    const int lg = a.by_cpg.div(u.c0 + min(c, u.nc - 1)) - u.g0;
    sm.par[4][c] = -sm.g0[lg];
    sm.par[5][c] = -sm.g1[lg];
  }
  __syncthreads();
  float2 m[NP], rs[NP], w[NP], b[NP], c1[NP], c2[NP], v[NP], d[NP];
  get_pairs<VEC>(sm.par[0] + u.tx * VEC, m);
  get_pairs<VEC>(sm.par[1] + u.tx * VEC, rs);
  get_pairs<VEC>(sm.par[2] + u.tx * VEC, w);
  get_pairs<VEC>(sm.par[3] + u.tx * VEC, b);
  get_pairs<VEC>(sm.par[4] + u.tx * VEC, c1);
  get_pairs<VEC>(sm.par[5] + u.tx * VEC, c2);
  T* o = static_cast<T*>(a.out) + gn_at<T, VEC>(u, a.out_sample, a.out_row);
  const int64_t ostep = (int64_t)u.TY * a.out_row;
  // The product w dz is rounded before c1 is taken off (no fma): in a group
  // of one value c1 is that very product and dx is exactly 0.
  auto body = [&](int j, T* to) {
    rows.v[0][j].get(v);
    rows.v[1][j].get(d);
    float2 z[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      v[i] = mul2(add2(v[i], m[i]), rs[i]);
      z[i] = fma2(v[i], w[i], b[i]);
    }
    through<ACT, NP>(d, z);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float2 g = make_float2(__fmul_rn(w[i].x, d[i].x), __fmul_rn(w[i].y, d[i].y));
      v[i] = mul2(rs[i], fma2(v[i], c2[i], add2(g, c1[i])));
    }
    Pack<T, VEC> y;
    y.set(v);
    y.template store<FINE>(to, a.grain, u.valid);
  };
  walk(o, ostep, body);
}

// ---- kernels ----------------------------------------------------------------------
__device__ __forceinline__ float2* gn_part(const GnArgs& a, const GnUnit& u) {
  return a.part + ((int64_t)u.n * a.tiles + u.tile) * a.max_groups * a.slices + u.slice;
}
// Dynamic shared memory: GnSmem, a cluster's partials, then the slots.
extern __shared__ __align__(16) unsigned char gn_dynamic[];
struct GnParts {
  float2 part[2][kGnMaxTileCh];
};
constexpr size_t gn_smem_bytes(int tensors, bool cluster) {
  return sizeof(GnSmem) + (cluster ? sizeof(GnParts) : 0) +
         (size_t)tensors * kGnRing * kGnThreads * 16;
}

// Where a unit's first rows are.
template <typename T, int VEC>
__device__ __forceinline__ void gn_fwd_rows(const GnArgs& a, const GnUnit& u, const T** p) {
  p[0] = static_cast<const T*>(a.x) + gn_at<T, VEC>(u, a.x_sample, a.x_row);
}
template <typename T, int VEC>
__device__ __forceinline__ void gn_bwd_rows(const GnArgs& a, const GnUnit& u, const T** p) {
  p[0] = static_cast<const T*>(a.x) + gn_at<T, VEC>(u, a.x_sample, a.x_row);
  p[1] = static_cast<const T*>(a.dy) + gn_at<T, VEC>(u, a.dy_sample, a.dy_row);
}

// One launch takes the statistics of the panels [stat0, stat1) and applies
// those of [app0, app1), which an earlier launch gathered.
template <typename T, int VEC, int ACT, bool FINE>
__global__ void __launch_bounds__(kGnThreads, 3)
    gn_fwd_kernel(GnArgs a, int stat0, int stat1, int app0, int app1) {
  GnSmem& sm = *reinterpret_cast<GnSmem*>(gn_dynamic);
  void* const ring = gn_dynamic + sizeof(GnSmem);
  const int p = a.by_slices.div(blockIdx.x), s = blockIdx.x - p * a.slices;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Rows<T, VEC, 1, FINE> rows;
  if (stat0 + p < stat1) {
    const GnUnit u = gn_unit<VEC>(a, stat0 + p, s);
    gn_fwd_rows<T, VEC>(a, u, rows.p);
    rows.step[0] = (int64_t)u.TY * a.x_row;
    rows.start(a, u, ring);
    gn_stats_unit<T, VEC>(a, u, sm, rows, gn_part(a, u), a.slices);
  }
  if (app0 + p < app1) {
    const GnUnit u = gn_unit<VEC>(a, app0 + p, s);
    gn_fwd_rows<T, VEC>(a, u, rows.p);
    rows.step[0] = (int64_t)u.TY * a.x_row;
    rows.start(a, u, ring);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    gn_combine<false>(a, u, sm);
    gn_apply_unit<T, VEC, ACT>(a, u, sm, rows, [&](T* o, int64_t ostep, auto& body) {
      rows.pass(o, ostep, body);
    });
  }
}

template <typename T, int VEC, int ACT, bool FINE>
__global__ void __launch_bounds__(kGnThreads, 2)
    gn_bwd_kernel(GnArgs a, int stat0, int stat1, int app0, int app1) {
  GnSmem& sm = *reinterpret_cast<GnSmem*>(gn_dynamic);
  void* const ring = gn_dynamic + sizeof(GnSmem);
  const int p = a.by_slices.div(blockIdx.x), s = blockIdx.x - p * a.slices;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Rows<T, VEC, 2, FINE> rows;
  if (stat0 + p < stat1) {
    const GnUnit u = gn_unit<VEC>(a, stat0 + p, s);
    gn_bwd_rows<T, VEC>(a, u, rows.p);
    rows.step[0] = (int64_t)u.TY * a.x_row;
    rows.step[1] = (int64_t)u.TY * a.dy_row;
    rows.start(a, u, ring);
    gn_bwd_stats_unit<T, VEC, ACT>(a, u, sm, rows, gn_part(a, u), a.slices);
  }
  if (app0 + p < app1) {
    const GnUnit u = gn_unit<VEC>(a, app0 + p, s);
    gn_bwd_rows<T, VEC>(a, u, rows.p);
    rows.step[0] = (int64_t)u.TY * a.x_row;
    rows.step[1] = (int64_t)u.TY * a.dy_row;
    rows.start(a, u, ring);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    gn_combine<true>(a, u, sm);
    gn_bwd_apply_unit<T, VEC, ACT>(a, u, sm, rows, [&](T* o, int64_t ostep, auto& body) {
      rows.pass(o, ostep, body);
    });
  }
}

// A panel a cluster: the statistics, a barrier of the cluster, and the rows
// again: those still in the slots, then the others out of the L2 cache. A
// cluster takes one panel after another and has the first rows of the next
// one on their way while it finishes this one. The partials have two places
// in turn: one is written again only after the barrier of the panel between,
// which every CTA reaches after it has read them.
template <typename T, int VEC, int ACT, bool FINE>
__global__ void __launch_bounds__(kGnThreads, 3) gn_fwd_cluster_kernel(GnArgs a, int panels) {
  GnSmem& sm = *reinterpret_cast<GnSmem*>(gn_dynamic);
  auto& part = reinterpret_cast<GnParts*>(gn_dynamic + sizeof(GnSmem))->part;
  void* const ring = gn_dynamic + sizeof(GnSmem) + sizeof(GnParts);
  int p = a.by_slices.div(blockIdx.x), turn = 0;
  const int rank = blockIdx.x - p * a.slices, clusters = a.by_slices.div(gridDim.x);
  GnUnit u = gn_unit<VEC>(a, p, rank);
  Rows<T, VEC, 1, FINE> rows;
  gn_fwd_rows<T, VEC>(a, u, rows.p);
  rows.step[0] = (int64_t)u.TY * a.x_row;
  rows.start(a, u, ring);
  while (true) {
    gn_stats_unit<T, VEC>(a, u, sm, rows, part[turn], 1);
    cluster_arrive();
    cluster_wait();
    gn_combine_cluster(a, u, sm, part[turn]);
    p += clusters;
    const GnUnit v = gn_unit<VEC>(a, p < panels ? p : 0, rank);
    const T* q[1];
    gn_fwd_rows<T, VEC>(a, v, q);
    gn_apply_unit<T, VEC, ACT>(a, u, sm, rows, [&](T* o, int64_t ostep, auto& body) {
      rows.again(o, ostep, body, q, p < panels ? v.rows : 0, v.valid);
    });
    if (p >= panels) break;
    u = v;
    turn ^= 1;
    __syncthreads();   // the parameters give way to the next sums
  }
  cluster_arrive();    // no CTA leaves while another reads its partials
  cluster_wait();
}

}  // namespace nf
