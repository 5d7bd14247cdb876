// The product of two microscaled matrices, simplest form: 64 x 64 results a
// CTA, values of 32 columns at a time in shared memory, 4 x 4 results a thread.
#pragma once

#include "common.cuh"
#include "mx_formats.cuh"

namespace nf {

struct ProductArgs {
  QuantOut a, b;
  float alpha;
  const void* bias;
  const void* residual;
  int64_t residual_row;
  void* out;
  int64_t out_row;
  float *psum, *psq;
};

__device__ __forceinline__ float mx_value(const QuantOut& q, int64_t row, int64_t col) {
  if (row >= q.rows || col >= q.cols) return 0.f;
  const unsigned b = static_cast<const unsigned char*>(q.scales)[scale_at(row, col / mx_block(q.fmt), q.blocks)];
  const float s = q.fmt == MX_NVFP4 ? __half2float(__half(__nv_cvt_fp8_to_halfraw((unsigned char)b, __NV_E4M3)))
                  : b == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float(b ? b << 23 : 1u << 22);
  const unsigned char* codes = q.codes + row * q.pitch;
  if (q.fmt == MX_MXFP8) return s * __half2float(__half(__nv_cvt_fp8_to_halfraw(codes[col], __NV_E4M3)));
  const __half2 h = __half2(__nv_cvt_fp4x2_to_halfraw2(codes[col / 2], __NV_E2M1));
  return s * __half2float(col & 1 ? __high2half(h) : __low2half(h));
}

template <typename T>
__global__ void __launch_bounds__(256) product_simple_kernel(const ProductArgs p) {
  __shared__ float as[32][65], bs[32][65];
  const int64_t m0 = (int64_t)blockIdx.x * 64, n0 = (int64_t)blockIdx.y * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < p.a.cols; k0 += 32) {
    for (int i = threadIdx.x; i < 64 * 32; i += 256) {
      as[i & 31][i >> 5] = mx_value(p.a, m0 + (i >> 5), k0 + (i & 31));
      bs[i & 31][i >> 5] = mx_value(p.b, n0 + (i >> 5), k0 + (i & 31));
    }
    __syncthreads();
    for (int k = 0; k < 32; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[k][ty * 4 + i], bs[k][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  const float f = p.alpha / (mul_of(p.a) * mul_of(p.b));
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= p.a.rows || n >= p.b.rows) continue;
      float v = acc[i][j] * f;
      if (p.bias) v += to_f(static_cast<const T*>(p.bias)[n]);
      if (p.residual) v += to_f(static_cast<const T*>(p.residual)[m * p.residual_row + n]);
      static_cast<T*>(p.out)[m * p.out_row + n] = from_f<T>(v);
    }
}

// Sums of the stored rows over 128 columns, a warp a tile.
template <typename T>
__global__ void __launch_bounds__(256) product_partials_kernel(const ProductArgs p) {
  const int64_t tiles = (p.b.rows + 127) / 128, i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= p.a.rows * tiles) return;
  const int64_t m = i / tiles, n0 = i % tiles * 128;
  const int n = (int)min((int64_t)128, p.b.rows - n0), lane = threadIdx.x & 31;
  const T* row = static_cast<const T*>(p.out) + m * p.out_row + n0;
  float s = 0.f, q = 0.f;
  for (int j = lane; j < n; j += 32) s += to_f(row[j]);
  s = group_sum<32>(s);
  for (int j = lane; j < n; j += 32) {
    const float d = to_f(row[j]) - s / (float)n;
    q = fmaf(d, d, q);
  }
  q = group_sum<32>(q);
  if (lane == 0) p.psum[i] = s, p.psq[i] = q;
}

template <typename T>
cudaError_t product_launch(const ProductArgs& p, cudaStream_t st) {
  const dim3 grid((unsigned)((p.a.rows + 63) / 64), (unsigned)((p.b.rows + 63) / 64));
  product_simple_kernel<T><<<grid, 256, 0, st>>>(p);
  if (p.psum) {
    const int64_t tiles = p.a.rows * ((p.b.rows + 127) / 128);
    product_partials_kernel<T><<<(unsigned)((tiles + 7) / 8), 256, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace nf
