// A matrix, or its transpose, in 8 or 4 bits with scales (mx_formats.cuh), and
// back to values.
//
// Bound by HBM: each value read once, 0.5 to 1 bytes of code written for it.
// The transpose goes through a tile in shared memory: 64 columns of x (rows of
// the result) by 128 rows, read along x's rows and written along the result's.
#pragma once

#include "common.cuh"
#include "mx_formats.cuh"

namespace nf {

struct QuantArgs {
  const void* x;
  int64_t x_row;         // elements from one row of x to the next
  QuantOut q;            // rows, cols: of the result
  int vec;               // x can be read 16 bytes at a time
  int vec_codes;         // codes can be written 16 bytes at a time (rows: where the pitch allows)
  int64_t padded_rows;
};

constexpr int kQuantThreads = 256;

// Eight neighbouring values of a row as fp32, 0 from column `n` on.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int64_t col, int64_t n, bool vec, float2* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = splat2(0.f);
  if (vec && col + 8 <= n) {
#pragma unroll
    for (int i = 0; i < 8 / Vec<T>::N; ++i)
      unpack2<T>(ld_vec(row + col + i * Vec<T>::N), v + i * Vec<T>::N / 2);
  } else {
    float* f = reinterpret_cast<float*>(v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < n) f[i] = to_f(row[col + i]);
  }
}

// Blocks of 16, 32 or 128 columns: 8 columns a lane, `kTiles` warps' worth (256
// columns each) a warp. CLS: 1 E4M3, 2 E2M1.
template <typename T, int CLS>
__global__ void __launch_bounds__(kQuantThreads) quant_block_kernel(const QuantArgs a, int64_t chunks) {
  const QuantOut& q = a.q;
  const int lane = threadIdx.x & 31;
  const float mul = CLS == 2 ? mul_of(q) : 1.0f;
  const int64_t wide = q.pitch * (CLS == 2 ? 2 : 1);
  const int64_t all = a.padded_rows * chunks;
  for (int64_t i = (int64_t)blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5); i < all;
       i += (int64_t)gridDim.x * (kQuantThreads / 32)) {
    const int64_t row = i / chunks, chunk = i - row * chunks;
    if (chunk == 0 && mx_tiled(q.fmt)) put_padding(q, row, lane, 32);
    if (row >= q.rows) continue;
    const int64_t col = chunk * 256 + lane * 8;
    float2 v[4];
    load8<T>(static_cast<const T*>(a.x) + row * a.x_row, col, q.cols, a.vec != 0, v);
    put_block<8, CLS>(q, row, col, col < wide, v, mul, CLS == 1 && (q.pitch % 8 != 0 || !a.vec_codes));
  }
}

// A scale a row: a CTA a row, which it reads twice (the second time out of the caches).
template <typename T>
__global__ void __launch_bounds__(kQuantThreads) quant_row_kernel(const QuantArgs a) {
  __shared__ unsigned red[kQuantThreads / 32];
  const QuantOut& q = a.q;
  for (int64_t row = blockIdx.x; row < q.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_row;
    unsigned m = 0;
    for (int64_t col = threadIdx.x * 8; col < q.cols; col += kQuantThreads * 8) {
      float2 v[4];
      load8<T>(x, col, q.cols, a.vec != 0, v);
      m = max(m, amax_of<4>(v));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int i = 0; i < kQuantThreads / 32; ++i) m = max(m, red[i]);
    const BlockScale s = scale_fp32(m);
    if (threadIdx.x == 0) static_cast<float*>(q.scales)[row] = s.scale;
    unsigned char* codes = q.codes + row * q.pitch;
    for (int64_t col = threadIdx.x * 8; col < q.cols; col += kQuantThreads * 8) {
      float2 v[4];
      unsigned c[2];
      load8<T>(x, col, q.cols, a.vec != 0, v);
      codes_e4m3<4>(v, s.factor, c);
      if (q.pitch % 8 == 0 && a.vec_codes && col + 8 <= q.cols) {
        put_codes<8>(codes + col, c, false);
      } else {
        for (int i = 0; i < 8 && col + i < q.cols; ++i) codes[col + i] = (unsigned char)(c[i / 4] >> (8 * (i % 4)));
      }
    }
  }
}

// The transpose. A CTA has 64 rows of the result (columns of x) and, for the
// block formats, 128 columns of it (rows of x) a tile; with a scale a row it
// goes over all tiles of its rows twice.
constexpr int kTrRows = 64;     // columns of x
constexpr int kTrCols = 128;    // rows of x

template <typename T>
__device__ __forceinline__ void load_tile(const QuantArgs& a, int64_t row0, int64_t col0,
                                          T (*tile)[kTrRows + 2]) {
  const int64_t rows = a.q.rows, cols = a.q.cols;
  for (int i = threadIdx.x; i < kTrCols * (kTrRows / 8); i += kQuantThreads) {
    const int c = i / (kTrRows / 8), r = i % (kTrRows / 8) * 8;
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = splat2(0.f);
    if (col0 + c < cols) load8<T>(static_cast<const T*>(a.x) + (col0 + c) * a.x_row, row0 + r, rows, a.vec != 0, v);
    const float* f = reinterpret_cast<const float*>(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) tile[c][r + j] = from_f<T>(f[j]);   // what was read: exact
  }
}

// CLS: 0 a scale a row, 1 blocks of E4M3, 2 blocks of E2M1.
template <typename T, int CLS>
__global__ void __launch_bounds__(kQuantThreads) quant_transpose_kernel(const QuantArgs a) {
  __shared__ T tile[kTrCols][kTrRows + 2];
  __shared__ unsigned red[kTrRows][4];
  const QuantOut& q = a.q;
  const int64_t row0 = (int64_t)blockIdx.x * kTrRows;
  const int r = threadIdx.x & (kTrRows - 1), part = threadIdx.x / kTrRows;   // 32 columns each
  const int64_t row = row0 + r;
  const float mul = CLS == 2 ? mul_of(q) : 1.0f;
  const int64_t tiles = (q.cols + kTrCols - 1) / kTrCols;
  if (CLS != 0 && mx_tiled(q.fmt) && blockIdx.y == 0 && row < a.padded_rows) put_padding(q, row, part, 4);
  unsigned m = 0;
  if (CLS == 0) {
    for (int64_t t = 0; t < tiles; ++t) {
      __syncthreads();
      load_tile<T>(a, row0, t * kTrCols, tile);
      __syncthreads();
      for (int i = 0; i < 32; ++i) m = max(m, abs_bits(to_f(tile[part * 32 + i][r])));
    }
    red[r][part] = m;
    __syncthreads();
    m = max(max(red[r][0], red[r][1]), max(red[r][2], red[r][3]));
  }
  BlockScale s = scale_fp32(m);
  if (CLS == 0 && part == 0 && row < q.rows) static_cast<float*>(q.scales)[row] = s.scale;
  for (int64_t t = blockIdx.y; t < tiles; t += gridDim.y) {
    __syncthreads();
    load_tile<T>(a, row0, t * kTrCols, tile);
    __syncthreads();
    const int64_t col = t * kTrCols + part * 32;
    float2 v[16];
    m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v[i] = make_float2(to_f(tile[part * 32 + 2 * i][r]), to_f(tile[part * 32 + 2 * i + 1][r]));
      if (CLS == 2 && q.fmt == MX_NVFP4) v[i] = mul2(v[i], splat2(mul));
    }
    if (CLS == 1) {
      m = amax_of<16>(v);
      if (q.fmt == MX_FP8_BLOCK) {
        red[r][part] = m;
        __syncthreads();
        m = max(max(red[r][0], red[r][1]), max(red[r][2], red[r][3]));
        s = scale_fp32(m);
      } else {
        s = scale_e8m0<false>(m);
      }
    }
    if (row >= q.rows || col >= q.cols) continue;    // the barriers are at the loop's head
    if (CLS == 2) {
      unsigned w[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s = q.fmt == MX_NVFP4 ? scale_e4m3(amax_of<8>(v + 8 * h)) : scale_e8m0<true>(amax_of<16>(v));
        w[2 * h] = codes_e2m1<4>(v + 8 * h, s, q.fmt == MX_NVFP4);
        w[2 * h + 1] = codes_e2m1<4>(v + 8 * h + 4, s, q.fmt == MX_NVFP4);
        const int64_t b = q.fmt == MX_NVFP4 ? col / 16 + h : col / 32;
        if (b < q.blocks) static_cast<unsigned char*>(q.scales)[scale_at(row, b, q.blocks)] = (unsigned char)s.byte;
      }
      *reinterpret_cast<uint4*>(q.codes + row * q.pitch + col / 2) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      unsigned w[8];
      codes_e4m3<16>(v, s.factor, w);
      unsigned char* p = q.codes + row * q.pitch + col;
      if (a.vec_codes && q.pitch % 16 == 0 && col + 32 <= q.pitch) {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (col + i < q.pitch) p[i] = (unsigned char)(w[i / 4] >> (8 * (i % 4)));
      }
      if (CLS == 1 && q.fmt == MX_FP8_BLOCK) {
        if (part == 0) static_cast<float*>(q.scales)[row * q.blocks + t] = s.scale;
      } else if (CLS == 1) {
        static_cast<unsigned char*>(q.scales)[scale_at(row, col / 32, q.blocks)] = (unsigned char)s.byte;
      }
    }
  }
}

// Values of 8 columns a thread.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads) dequant_kernel(const QuantOut q, T* y, int64_t y_row,
                                                                bool vec, int64_t chunks) {
  const int64_t all = q.rows * chunks;
  for (int64_t i = (int64_t)blockIdx.x * kQuantThreads + threadIdx.x; i < all;
       i += (int64_t)gridDim.x * kQuantThreads) {
    const int64_t row = i / chunks, col = (i - row * chunks) * 8;
    const unsigned char* codes = q.codes + row * q.pitch;
    float2 v[4];
    if (mx_four(q.fmt)) {
      const unsigned w = *reinterpret_cast<const unsigned*>(codes + col / 2);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = __half22float2(__half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(w >> (8 * j)), __NV_E2M1)));
    } else {
      float* f = reinterpret_cast<float*>(v);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[j] = __half2float(__half(__nv_cvt_fp8_to_halfraw(col + j < q.pitch ? codes[col + j] : (unsigned char)0, __NV_E4M3)));
    }
    float s;
    if (q.fmt == MX_FP8_ROW) {
      s = static_cast<const float*>(q.scales)[row];
    } else if (q.fmt == MX_FP8_BLOCK) {
      s = static_cast<const float*>(q.scales)[row * q.blocks + col / 128];
    } else {
      const unsigned b = static_cast<const unsigned char*>(q.scales)[scale_at(row, col / mx_block(q.fmt), q.blocks)];
      if (q.fmt == MX_NVFP4)
        s = __half2float(__half(__nv_cvt_fp8_to_halfraw((unsigned char)b, __NV_E4M3)));
      else
        s = b == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float(b ? b << 23 : 1u << 22);
    }
    const float mul = mul_of(q);
    float* f = reinterpret_cast<float*>(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = f[j] * s;
    if (q.fmt == MX_NVFP4 && q.mul != nullptr) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] / mul;
    }
    T* out = y + row * y_row + col;
    if (vec && col + 8 <= q.cols) {
#pragma unroll
      for (int j = 0; j < 8 / Vec<T>::N; ++j) st_vec(out + j * Vec<T>::N, pack2<T>(v + j * Vec<T>::N / 2));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < q.cols) out[j] = from_f<T>(f[j]);
    }
  }
}

}  // namespace nf
