// The fused block's forward (bias + residual addition, LayerNorm or RMSNorm)
// with its result in 8 or 4 bits and scales (mx_formats.cuh).
//
// A row stays in registers from its one read to its codes, as in the 16-bit
// forward: sum and its rounding, mean, centred squares, then y in fp32, which
// is quantised as it is (rounding it to the I/O type first would round twice).
// A block's values lie in 2 to 32 neighbouring lanes, so its largest magnitude
// takes 1 to 5 shuffles; a row's goes through the CTA as the sums do.
//
// What bounds it: HBM (x and residual read, the sum and 0.5 to 1 bytes a value
// written) and, with block scales, the instructions: 16384 x 8192 bf16 RMSNorm
// with a residual takes 137 us to fp8_row (6.9 TB/s), 142 to mxfp8 (6.7), 153 to
// nvfp4 (5.8 TB/s, 82% of the issue slots).
#pragma once

#include "bulk.cuh"
#include "common.cuh"
#include "mx_formats.cuh"

namespace nf {

struct MxNormArgs {
  FwdArgs f;       // y may be null; amax and y_fp8 are not used
  QuantOut q;
  int64_t padded_rows;   // rows whose scales are written: a multiple of 128 in tiles
  int order_lanes;       // few rows: lanes or threads of a row, and vectors of each,
  int order_n;           // in the plan for many, whose order of sums they keep; else 0
};

// Few rows are spread over more threads than many. So that a row's result does not
// depend on how many others there are, both add in the order of the plan for many:
// each vector's values as a pair, the vectors of one of its order_lanes threads one
// after the other, the pair, the lanes, the warps. That costs many rows nothing
// (16384 x 8192 bf16 to nvfp4 152 us with and without) and few some 0.1 to 0.5 us; one
// tree over the vectors, a shuffle more for each, cost many rows 2 to 4%.

// In a warp that has N vectors a lane, where order_lanes is a power of two: the order_n
// vectors of a lane in the plan for many come by shuffles, from one of N places each.
template <int N> __device__ __forceinline__ float ordered_warp_sum(const MxNormArgs& a, const float2* part) {
  const int L = a.order_lanes, lane = threadIdx.x & 31;
  float2 t = splat2(0.f);
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    if (k >= a.order_n || k * L >= 32 * N) break;      // what is behind are zeros
    const float2 from = N == 2 && k * L >= 32 ? part[N - 1] : part[0];
    const int at = (k * L + (lane & (L - 1))) & 31;
    const float2 v = {__shfl_sync(0xffffffffu, from.x, at), __shfl_sync(0xffffffffu, from.y, at)};
    t = k == 0 ? v : add2(t, v);
  }
  float sum = t.x + t.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < L) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// The vectors of thread u in the plan for many, out of shared memory with `room` for
// them.
__device__ __forceinline__ float ordered_thread_sum(const MxNormArgs& a, const float2* parts, int u, int room) {
  float2 t = parts[u];
#pragma unroll
  for (int k = 1; k < 8; ++k) {
    const int v = k * a.order_lanes + u;
    if (k < a.order_n) t = add2(t, v < room ? parts[v] : splat2(0.f));
  }
  return t.x + t.y;
}
// In a CTA of `room` vectors; `parts` and `red`, each one of two in turn. Where a lane
// group has a row in the plan for many, each warp adds all of it.
__device__ __forceinline__ float ordered_cta_sum(const MxNormArgs& a, float2* parts, int room, float* red) {
  const int L = a.order_lanes;
  __syncthreads();
  if (L <= 32) {
    float v = ordered_thread_sum(a, parts, threadIdx.x & (L - 1), room);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < L) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  if ((int)threadIdx.x < L) {                           // whole warps
    const float v = group_sum<32>(ordered_thread_sum(a, parts, threadIdx.x, room));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  }
  __syncthreads();
  float t = 0.f;
#pragma unroll 4
  for (int i = 0; i < (L >> 5); ++i) t += red[i];       // as cta_sum_db_fit
  return t;
}

// Rows in registers. CLS: 0 a scale a row, 1 blocks of E4M3, 2 blocks of E2M1.
// G0 > 0: a group of G0 lanes a row; 0: the CTA.
template <typename T, int G0, int N, int CLS, typename Sum, typename Max>
__device__ __forceinline__ void mx_norm_row(const MxNormArgs& a, int64_t row, int t, Sum reduce,
                                            Max row_max) {
  constexpr int VEC = Vec<T>::N;
  constexpr int P = VEC / 2;
  const FwdArgs& f = a.f;
  const int G = G0 > 0 ? G0 : (int)blockDim.x;
  const bool row_ok = G0 == 0 || row < f.rows;     // a CTA without a row does not come here
  const int H = f.hidden;
  const int V = H / VEC;
  const int64_t off = row * (int64_t)H;
  const T* x = static_cast<const T*>(f.x) + off;
  const T* res = f.residual ? static_cast<const T*>(f.residual) + off : nullptr;
  uint4 xr[N], rr[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int v = k * G + t;
    if (row_ok && v < V) {
      xr[k] = ld_behind(x + v * VEC);
      if (res) rr[k] = ld_behind(res + v * VEC);
    }
  }
  if (CLS != 0 && mx_tiled(a.q.fmt) && row < a.padded_rows) put_padding(a.q, row, t, G);

  float2 s[N][P];
  float2 part[N], all;             // sums of the vectors and of the thread
  T* sum_row = f.out_sum ? static_cast<T*>(f.out_sum) + off : nullptr;
  const ParamRow<T> w_row = {nullptr, static_cast<const T*>(f.gamma), H, f.zero_centered != 0};
  const ParamRow<T> bias_row = {nullptr, static_cast<const T*>(f.bias), H, false};
  const ParamRow<T> beta_row = {nullptr, static_cast<const T*>(f.beta), H, false};
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int v = k * G + t;
#pragma unroll
    for (int i = 0; i < P; ++i) s[k][i] = splat2(0.f);
    part[k] = splat2(0.f);
    if (row_ok && v < V) {
      unpack2<T>(xr[k], s[k]);
      if (bias_row.g) {
        float2 b[P];
        bias_row.template load2<false>(v, b);
#pragma unroll
        for (int i = 0; i < P; ++i) s[k][i] = add2(s[k][i], b[i]);
      }
      if (res) {
        float2 r[P];
        unpack2<T>(rr[k], r);
#pragma unroll
        for (int i = 0; i < P; ++i) s[k][i] = add2(s[k][i], r[i]);
      }
      const uint4 packed = pack2<T>(s[k]);
      if (sum_row) st_vec(sum_row + v * VEC, packed);
      unpack2<T>(packed, s[k]);
      part[k] = s[k][0];
#pragma unroll
      for (int i = 1; i < P; ++i) part[k] = add2(part[k], s[k][i]);
    }
    all = k > 0 ? add2(all, part[k]) : part[k];
  }
  const float mean = f.rms ? 0.f : reduce(all.x + all.y, part) / (float)H;
  const float2 neg_mean = splat2(-mean);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    part[k] = splat2(0.f);
    if (row_ok && (k * G + t) < V) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        s[k][i] = add2(s[k][i], neg_mean);
        part[k] = i == 0 ? mul2(s[k][i], s[k][i]) : fma2(s[k][i], s[k][i], part[k]);
      }
    }
    all = k > 0 ? add2(all, part[k]) : part[k];
  }
  const float rstd = 1.0f / sqrtf(reduce(all.x + all.y, part) / (float)H + f.eps);
  if (row_ok && t == 0) {
    if (f.mean) f.mean[row] = mean;
    if (f.rstd) f.rstd[row] = rstd;
  }

  const float2 r2 = splat2(rstd);
  const float mul = CLS == 2 ? mul_of(a.q) : 1.0f;
  const int wide = (int)a.q.pitch * (CLS == 2 ? 2 : 1);   // columns with room for codes
  unsigned m = 0;
  // y of slot k, in fp32
  const auto norm = [&](int k) {
    const int v = k * G + t;
    if (row_ok && v < V) {
      float2 w[P], o[P];
      w_row.template load2<false>(v, w);
      if (beta_row.g) {
        beta_row.template load2<false>(v, o);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = splat2(0.f);
      }
#pragma unroll
      for (int i = 0; i < P; ++i) s[k][i] = fma2(mul2(s[k][i], r2), w[i], o[i]);
      if (f.y) st_vec(static_cast<T*>(f.y) + off + v * VEC, pack2<T>(s[k]));
      if (CLS == 0) m = max(m, amax_of<P>(s[k]));
    }
  };
  if constexpr (CLS == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) norm(k);
  } else {
    const auto blocks = [&](auto fmt) {
      using F = decltype(fmt);
      unsigned char *scales = scales_of_row<F::value>(a.q, row), *codes = a.q.codes + row * a.q.pitch;
      // a lane is first in a block in each slot or in none: G * VEC columns are whole blocks
      const bool first = row_ok && t * VEC % F::width == 0;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        norm(k);
        const int col = (k * G + t) * VEC;
        put_block<VEC, F::value>(s[k], mul, codes + (F::four ? col / 2 : col), row_ok && col < wide,
                                 scales + scale_step<F::value>(col / F::width), first && col < H);
      }
    };
    // one format a loop: its shuffles and conversions are known then
    if (CLS == 1) {
      if (a.q.fmt == MX_MXFP8) blocks(Format<MX_MXFP8>());
      else blocks(Format<MX_FP8_BLOCK>());
    } else {
      if (a.q.fmt == MX_MXFP4) blocks(Format<MX_MXFP4>());
      else blocks(Format<MX_NVFP4>());
    }
  }
  if (CLS == 0) {
    const BlockScale b = scale_fp32(row_max(m));
    if (row_ok && t == 0) static_cast<float*>(a.q.scales)[row] = b.scale;
    unsigned char* codes = a.q.codes + off;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int v = k * G + t;
      if (row_ok && v < V) {
        unsigned c[VEC / 4];
        codes_e4m3<P>(s[k], b.factor, c);
        put_codes<VEC>(codes + v * VEC, c, false);
      }
    }
  }
}

// A tile of 8 * (32 / LANES) rows a CTA, a lane group a row.
template <typename T, int LANES, int N, int CLS>
__global__ void __launch_bounds__(kBulkThreads, N <= 3 ? 4 : 3) mx_norm_tile_kernel(const MxNormArgs a) {
  constexpr int RPW = 32 / LANES;
  const int lane = threadIdx.x & 31;
  const int64_t row =
      ((int64_t)blockIdx.x * kConsumerWarps + (threadIdx.x >> 5)) * RPW + lane / LANES;
  start_after_stream();
  mx_norm_row<T, LANES, N, CLS>(
      a, row, lane % LANES,
      [&](float all, const float2* part) {
        if constexpr (LANES == 32 && N <= 2) {         // may be the plan for few rows
          if (a.order_n) return ordered_warp_sum<N>(a, part);
        }
        return group_sum<LANES>(all);
      },
      [](unsigned v) { return lanes_max<LANES>(v); });
}

// A CTA a row, blockDim.x * N vectors.
template <typename T, int N, int CLS>
__global__ void __launch_bounds__(kMaxFitThreads) __maxnreg__(N <= 4 ? 64 : 128) mx_norm_cta_kernel(const MxNormArgs a) {
  __shared__ float red[2][kMaxFitWarps];
  __shared__ unsigned red_max[kMaxFitWarps];
  extern __shared__ float2 parts[];                    // few rows: 2 * N * blockDim.x
  start_after_stream();
  if (blockIdx.x >= a.f.rows) {    // the scales behind the last row
    if (CLS != 0) put_padding(a.q, blockIdx.x, threadIdx.x, blockDim.x);
    return;
  }
  int parity = 0;
  mx_norm_row<T, 0, N, CLS>(
      a, blockIdx.x, threadIdx.x,
      [&](float all, const float2* part) {
        if constexpr (N == 2) {                        // may be the plan for few rows
          if (a.order_n) {
            const int room = N * blockDim.x;
            float2* row = parts + parity * room;
#pragma unroll
            for (int k = 0; k < N; ++k) row[k * blockDim.x + threadIdx.x] = part[k];
            const float t = ordered_cta_sum(a, row, room, red[parity]);
            parity ^= 1;
            return t;
          }
        }
        return cta_sum_db_fit(all, red, parity);
      },
      [&](unsigned v) {
        v = __reduce_max_sync(0xffffffffu, v);
        if ((threadIdx.x & 31) == 0) red_max[threadIdx.x >> 5] = v;
        __syncthreads();
        unsigned m = 0;
        for (int i = 0; i < (int)(blockDim.x >> 5); ++i) m = max(m, red_max[i]);
        return m;
      });
}

// Rows that start anywhere, of any hidden size: element by element, a warp's lanes
// on neighbouring columns, so that it still reads and writes runs of its lanes. A
// warp has chunks of 128 columns, four columns 32 apart a lane, up to kChunks of
// them. For the blocks they change places through shared memory (512 floats a
// warp, dynamic), to 8 neighbouring columns a lane: with a scale worked out for
// each access, a column a lane, 8192 x 5121 bf16 to nvfp4 took 442 us.
// WARP: a warp a row (up to 512 columns), 8 rows a CTA; else a CTA a row.
constexpr int kChunks = 4;

template <typename T, bool WARP>
__global__ void __launch_bounds__(kMaxFitThreads) mx_norm_ragged_kernel(const MxNormArgs a) {
  extern __shared__ float turned[];
  __shared__ float red[2][kMaxFitWarps];
  __shared__ unsigned red_max[kMaxFitWarps];
  start_after_stream();
  const FwdArgs& f = a.f;
  const QuantOut& q = a.q;
  const int H = f.hidden, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = WARP ? 1 : (int)(blockDim.x >> 5), mine = WARP ? 0 : warp;
  const int64_t row = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + warp : blockIdx.x;
  if (mx_tiled(q.fmt) && row < a.padded_rows) put_padding(q, row, mine * 32 + lane, warps * 32);
  if (row >= f.rows) return;      // a whole warp, or a whole CTA
  const int64_t off = row * (int64_t)H;
  const T *x = static_cast<const T*>(f.x) + off, *res = f.residual ? static_cast<const T*>(f.residual) + off : nullptr;
  const T *bias = static_cast<const T*>(f.bias), *gamma = static_cast<const T*>(f.gamma), *beta = static_cast<const T*>(f.beta);
  T *out_sum = f.out_sum ? static_cast<T*>(f.out_sum) + off : nullptr, *y = f.y ? static_cast<T*>(f.y) + off : nullptr;
  int parity = 0;
  const auto reduce = [&](float v) { return WARP ? group_sum<32>(v) : cta_sum_db_fit(v, red, parity); };
  // column of slot i, s
  const auto column = [&](int i, int s) { return (i * warps + mine) * 128 + 32 * s + lane; };
  float v[kChunks][4], u[kChunks][4];
  float t = 0.f;
  // each of these loops has its loads on their way together: what is stored
  // could, as far as the compiler knows, be what is loaded next
  const auto load = [&](const T* p, float (*to)[4]) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int s = 0; s < 4; ++s) to[i][s] = column(i, s) < H ? to_f(ld_one_behind(p + column(i, s))) : 0.f;
  };
  load(x, v);
  if (res) load(res, u);
  if (bias) {
    float b[kChunks][4];
    load(bias, b);
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int s = 0; s < 4; ++s) v[i][s] += b[i][s];
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int j = column(i, s);
      const T stored = from_f<T>(res ? v[i][s] + u[i][s] : v[i][s]);
      if (out_sum && j < H) out_sum[j] = stored;
      v[i][s] = to_f(stored);
      t += v[i][s];
    }
  const float mean = f.rms ? 0.f : reduce(t) / (float)H;
  t = 0.f;
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (column(i, s) < H) {
        v[i][s] -= mean;
        t = fmaf(v[i][s], v[i][s], t);
      }
  const float rstd = 1.0f / sqrtf(reduce(t) / (float)H + f.eps);
  if (mine == 0 && lane == 0) {
    if (f.mean) f.mean[row] = mean;
    if (f.rstd) f.rstd[row] = rstd;
  }
  unsigned m = 0;
  load(gamma, u);
  if (f.zero_centered) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int s = 0; s < 4; ++s) u[i][s] += 1.0f;
  }
  float b[kChunks][4] = {};
  if (beta) load(beta, b);
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int j = column(i, s);
      v[i][s] = j < H ? fmaf(v[i][s] * rstd, u[i][s], b[i][s]) : 0.f;
      if (y && j < H) y[j] = from_f<T>(v[i][s]);
      m = max(m, abs_bits(v[i][s]));
    }
  if (q.fmt == MX_FP8_ROW) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (!WARP) {
      if (lane == 0) red_max[warp] = m;
      __syncthreads();
      for (int i = 0; i < warps; ++i) m = max(m, red_max[i]);
    }
    const BlockScale b = scale_fp32(m);
    if (mine == 0 && lane == 0) static_cast<float*>(q.scales)[row] = b.scale;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (column(i, s) < H) q.codes[off + column(i, s)] = b.factor == 0.f ? 0 : fp8_one(v[i][s], b.factor);
    return;
  }
  const float mul = mul_of(q);
  float* place = turned + warp * (kChunks * 128);
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s) place[i * 128 + 32 * s + lane] = v[i][s];
  __syncwarp();
  const auto blocks = [&](auto fmt) {
    using F = decltype(fmt);
    unsigned char *scales = scales_of_row<F::value>(q, row), *codes = q.codes + row * q.pitch;
    const int wide = (int)q.pitch * (F::four ? 2 : 1);
#pragma unroll
    for (int k = 0; k < kChunks / 2; ++k) {
      if ((2 * k * warps + mine) * 128 >= H) break;
      const int col = ((2 * k + lane / 16) * warps + mine) * 128 + lane % 16 * 8;
      float2 o[4];
      const float4* from = reinterpret_cast<const float4*>(place + k * 256 + lane * 8);
      const float4 lo = from[0], hi = from[1];
      o[0] = make_float2(lo.x, lo.y);
      o[1] = make_float2(lo.z, lo.w);
      o[2] = make_float2(hi.x, hi.y);
      o[3] = make_float2(hi.z, hi.w);
      put_block<8, F::value>(o, mul, codes + (F::four ? col / 2 : col), col < wide,
                             scales + scale_step<F::value>(col / F::width), col % F::width == 0 && col < H,
                             min(8, wide - col), true);
    }
  };
  if (q.fmt == MX_NVFP4) blocks(Format<MX_NVFP4>());
  else if (q.fmt == MX_MXFP4) blocks(Format<MX_MXFP4>());
  else if (q.fmt == MX_MXFP8) blocks(Format<MX_MXFP8>());
  else blocks(Format<MX_FP8_BLOCK>());
}

template <typename T, int LANES, int CLS> const void* mx_norm_tile_of(int n) {
  switch (n) {
    case 1: return (const void*)mx_norm_tile_kernel<T, LANES, 1, CLS>;
    case 2: return (const void*)mx_norm_tile_kernel<T, LANES, 2, CLS>;
    case 3: return (const void*)mx_norm_tile_kernel<T, LANES, 3, CLS>;
    case 4: return (const void*)mx_norm_tile_kernel<T, LANES, 4, CLS>;
    case 5: return (const void*)mx_norm_tile_kernel<T, LANES, 5, CLS>;
    default: return nullptr;
  }
}
template <typename T, int CLS> const void* mx_norm_cta_of(int n) {
  switch (n) {
    case 2: return (const void*)mx_norm_cta_kernel<T, 2, CLS>;
    case 3: return (const void*)mx_norm_cta_kernel<T, 3, CLS>;
    case 4: return (const void*)mx_norm_cta_kernel<T, 4, CLS>;
    case 5: return (const void*)mx_norm_cta_kernel<T, 5, CLS>;
    case 6: return (const void*)mx_norm_cta_kernel<T, 6, CLS>;
    case 8: return (const void*)mx_norm_cta_kernel<T, 8, CLS>;
    default: return nullptr;
  }
}
// lanes 8, 16, 32: a lane group a row; 0: a CTA a row; -1, -2: element by element,
// a warp or a CTA a row.
template <typename T, int CLS> const void* mx_norm_cls(int lanes, int n) {
  switch (lanes) {
    case 8: return mx_norm_tile_of<T, 8, CLS>(n);
    case 16: return mx_norm_tile_of<T, 16, CLS>(n);
    case 32: return mx_norm_tile_of<T, 32, CLS>(n);
    default: return mx_norm_cta_of<T, CLS>(n);
  }
}
template <typename T> const void* mx_norm_table(int cls, int lanes, int n) {
  if (lanes == -1) return (const void*)mx_norm_ragged_kernel<T, true>;
  if (lanes == -2) return (const void*)mx_norm_ragged_kernel<T, false>;
  return cls == 0 ? mx_norm_cls<T, 0>(lanes, n) : cls == 1 ? mx_norm_cls<T, 1>(lanes, n)
                                                          : mx_norm_cls<T, 2>(lanes, n);
}

}  // namespace nf
