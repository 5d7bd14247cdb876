// Norms with quantised results, the quantiser and its inverse: C entry points,
// argument checks and launch plan.
#include <math.h>

#include <algorithm>

#include "../../include/normfuse.h"
#include "launch.h"
#include "mx_check.h"
#include "mx_norm_kernels.cuh"
#include "mx_quantize_kernels.cuh"
#include "tensor_map.h"
#include "validate.h"

namespace nf {

cudaError_t take_error_quantize(cudaStream_t st, unsigned* out) { return take_tu_error(st, out); }

const void* mx_norm_table_f32(int cls, int lanes, int n);
const void* mx_norm_table_bf16(int cls, int lanes, int n);
const void* mx_norm_table_f16(int cls, int lanes, int n);

namespace {

ln_status cuda_fail(cudaError_t e) {
  nf_set_last_cuda_error((int)e);
  return LN_ERR_CUDA;
}

int class_of(int fmt) { return fmt == MX_FP8_ROW ? 0 : mx_four(fmt) ? 2 : 1; }

// Lanes a row (0: a CTA), vectors a lane and threads for rows of `slots` 16-byte
// vectors, room for codes included. As in the 16-bit forward: lane groups up to
// 160 vectors, four vectors a lane where the row splits evenly, then a CTA
// fitted to the row (8192 x 5120 bf16 LayerNorm to mxfp4 49.7 us with four
// vectors a thread, 53.4 with three, 55.2 with six, 65.6 with eight). A block of 128
// columns needs 16 lanes (32 for fp32).
struct NormPlan {
  int lanes = -1, n = 0, block = 256;
};
NormPlan norm_plan(int slots, int least_lanes) {
  NormPlan p;
  if (slots <= 160) {
    for (int n : {4, 3, 5, 2, 1}) {
      const int lanes = slots / n;
      if (slots % n == 0 && (lanes == 8 || lanes == 16 || lanes == 32) && lanes >= least_lanes)
        return {lanes, n, kBulkThreads};
    }
    int idle = 1 << 30;
    for (int lanes : {32, 16, 8}) {
      const int n = (slots + lanes - 1) / lanes;
      if (lanes < least_lanes || n > 5 || lanes * n - slots >= idle) continue;
      idle = lanes * n - slots;
      p = {lanes, n, kBulkThreads};
    }
    return p;
  }
  int idle = 1 << 30;
  for (int n : {4, 5, 3, 6, 8, 2}) {
    const int nt = std::max(64, (slots + 32 * n - 1) / (32 * n) * 32);
    if (nt > kMaxFitThreads || nt * n - slots >= idle) continue;
    idle = nt * n - slots;
    p = {0, n, nt};
  }
  return p;
}

// Few rows leave threads idle anyway, so a row is spread over as many as there are,
// two vectors each, and its sums are put in the order of the plan above (on the GPU
// 64 x 1280 bf16 to mxfp8 2.6 us against 3.8, 1 x 4096 to mxfp4 2.5 against 3.1, 1024 x
// 320 fp16 to mxfp8 3.3 against 4.1; 8192 x 320, which is not few, 7.3 against 6.1; a
// CTA's longer row gains or loses 0.2 us where a CTA an SM is not enough, 512 x 1000
// fp32 4.2 against 4.4, 300 x 2560 bf16 4.65 against 4.45). n = 0: rows are not few, or
// too wide.
NormPlan few_plan(int slots, int64_t rows, int sms) {
  const bool few = slots <= 160 ? rows * slots <= (int64_t)sms * 1024 : rows <= sms;
  if (!few || slots > 2 * kMaxFitThreads) return {-1, 0, 0};
  if (slots <= 64) return {32, (slots + 31) / 32, kBulkThreads};
  return {0, 2, std::max(64, (slots + 63) / 64 * 32)};
}

int64_t padded_rows(const QuantOut& q) { return mx_tiled(q.fmt) ? (q.rows + 127) / 128 * 128 : q.rows; }

// Lanes a row of `cols` columns takes at 8 a lane (`least` at least), as a power
// of two, and the grid of CTAs that deal rows to them: about 12 an SM, so that a
// lane has rows enough to have one on its way.
int row_shift(int64_t cols, int least) {
  int shift = 0;
  while (shift < 5 && ((1 << shift) < least || (8 << shift) < cols)) ++shift;
  return shift;
}
dim3 row_grid(int64_t rows, int64_t cols, int shift, int sms) {
  const int64_t x = (cols + 255) / 256, per = (int64_t)(kQuantThreads / 32) << (5 - shift);
  const int64_t most = std::max<int64_t>(1, (int64_t)sms * 12 / x);
  return dim3((unsigned)x, (unsigned)std::min<int64_t>(std::min<int64_t>((rows + per - 1) / per, most), 65535));
}

// The transpose by tensor maps: x on 16 bytes, its rows a multiple of them apart
// and not in one another.
template <typename T, int FMT>
cudaError_t launch_transpose_tma(const QuantArgs& a, int64_t x, int64_t tiles, int sms, cudaStream_t st) {
  const void* fn;
  if constexpr (FMT == MX_FP8_ROW) fn = (const void*)quant_transpose_row_tma_kernel<T>;
  else fn = (const void*)quant_transpose_tma_kernel<T, FMT>;
  constexpr size_t kSmem = kTrStages * kTrBytes + 1024;
  Encode encode;
  CUtensorMap map;
  cudaError_t e = encoder(&encode);
  if (e == cudaSuccess) e = (cudaError_t)allow_dyn_smem(fn, kSmem);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[2] = {(cuuint64_t)a.q.rows, (cuuint64_t)a.q.cols}, strides[1] = {(cuuint64_t)a.x_row * sizeof(T)};
  const cuuint32_t box[2] = {(cuuint32_t)TrRows<T>::N, (cuuint32_t)kTrCols}, step[2] = {1, 1};
  const CUresult r = encode(&map, sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
                            const_cast<void*>(a.x), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
  int64_t all = FMT == MX_FP8_ROW ? x : x * tiles;
  QuantArgs args = a;
  void* params[] = {&map, &args, &all};
  return launch_overlapped(fn, dim3((unsigned)std::min<int64_t>(all, 2 * sms)), dim3(kQuantThreads), params, kSmem, st);
}

template <typename T, int FMT>
cudaError_t launch_quantize(const QuantArgs& a, int transpose, int sms, cudaStream_t st) {
  const QuantOut& q = a.q;
  if (transpose) {
    const int64_t x = (a.padded_rows + TrRows<T>::N - 1) / TrRows<T>::N, tiles = (q.cols + kTrCols - 1) / kTrCols;
    // a copy each 16 bytes of x's rows: the tensor map's, from where the loop over
    // tiles has more than one round
    if (a.vec && a.x_row >= q.rows && a.x_row * (int64_t)sizeof(T) % 16 == 0 && a.x_row < (1ll << 37) &&
        x * tiles > 2 * sms)
      return launch_transpose_tma<T, FMT>(a, x, tiles, sms, st);
    const dim3 grid((unsigned)x, FMT == MX_FP8_ROW ? 1u : (unsigned)std::min<int64_t>(tiles, 65535));
    void* args[] = {const_cast<QuantArgs*>(&a)};
    return launch_overlapped((const void*)quant_transpose_kernel<T, FMT>, grid, dim3(kQuantThreads), args, 0, st);
  } else if constexpr (FMT == MX_FP8_ROW) {
    void* args[] = {const_cast<QuantArgs*>(&a)};
    return launch_overlapped((const void*)quant_row_kernel<T>, dim3((unsigned)std::min<int64_t>(q.rows, 1 << 20)),
                             dim3(kQuantThreads), args, 0, st);
  } else {
    // room for codes included
    int shift = row_shift(mx_tiled(FMT) ? (q.cols + 31) / 32 * 32 : q.cols, mx_block(FMT) / 8);
    const void* fn = a.vec ? (const void*)quant_block_kernel<T, FMT, false> : (const void*)quant_block_kernel<T, FMT, true>;
    void* args[] = {const_cast<QuantArgs*>(&a), &shift};
    return launch_overlapped(fn, row_grid(a.padded_rows, q.cols, shift, sms), dim3(kQuantThreads), args, 0, st);
  }
}

}  // namespace
}  // namespace nf

using namespace nf;

extern "C" {

ln_status mx_matrix_bytes(mx_format format, int64_t rows, int64_t cols, size_t* codes,
                          size_t* scales) {
  if (codes == nullptr || scales == nullptr) return LN_ERR_NULL;
  if (!known_format(format)) return LN_ERR_UNSUPPORTED;
  if (!fits(rows, cols)) return LN_ERR_SHAPE;
  *codes = code_bytes(format, rows, cols);
  *scales = scale_bytes(format, rows, cols);
  return LN_OK;
}

ln_status mx_norm_fwd(const void* x, const void* bias, const void* residual, const void* gamma,
                      const void* beta, float eps, ln_mode mode, int zero_centered_gamma,
                      void* out_sum, void* y, float* mean, float* rstd, const mx_matrix* q,
                      cudaStream_t stream, ln_dtype dtype) {
  if (q == nullptr) return LN_ERR_NULL;
  if (!known_dtype(dtype) || !known_format(q->format)) return LN_ERR_UNSUPPORTED;
  if (mode != LN_LAYERNORM && mode != LN_RMSNORM) return LN_ERR_UNSUPPORTED;
  const int64_t rows = q->rows, hidden = q->cols;
  if (rows < 0 || hidden < 1 || rows > INT32_MAX - 128) return LN_ERR_SHAPE;
  if (!(eps >= 0.0f) || !isfinite(eps)) return LN_ERR_INVALID;
  const bool rms = mode == LN_RMSNORM;
  if (rms) {
    beta = nullptr;
    mean = nullptr;
  }
  if (gamma == nullptr) return LN_ERR_NULL;
  if (rows > 0 && x == nullptr) return LN_ERR_NULL;
  ln_status st = check_matrix(*q);
  if (st != LN_OK) return st;
  const size_t es = elem_size(dtype);
  const void* tensors[] = {x, bias, residual, gamma, beta, out_sum, y};
  for (const void* p : tensors)
    if (!aligned(p, es)) return LN_ERR_ALIGN;
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return LN_ERR_ALIGN;
  bool vec = (hidden * (int64_t)es) % 16 == 0;
  for (const void* p : tensors)
    if (!aligned(p, 16)) vec = false;
  if (!aligned(q->codes, 16)) vec = false;
  if (vec && hidden > (int64_t)(16 / es) * kMaxVecSlots) vec = false;
  if (!vec && hidden > kMaxHiddenScalar) return LN_ERR_SHAPE;
  const size_t mat = (size_t)rows * (size_t)hidden * es, vecb = (size_t)hidden * es;
  const Range outs[] = {{out_sum, mat}, {y, mat}, {mean, (size_t)rows * 4}, {rstd, (size_t)rows * 4},
                        codes_range(*q), scales_range(*q)};
  const Range ins[] = {{x, mat}, {residual, mat}, {bias, vecb}, {gamma, vecb}, {beta, vecb},
                       mul_range(*q)};
  if (any_overlap(outs, 6, ins, 6)) return LN_ERR_INVALID;
  if (rows == 0) return LN_OK;

  MxNormArgs a = {};
  a.f.x = x;
  a.f.bias = bias;
  a.f.residual = residual;
  a.f.gamma = gamma;
  a.f.beta = beta;
  a.f.out_sum = out_sum;
  a.f.y = y;
  a.f.mean = mean;
  a.f.rstd = rstd;
  a.f.rows = rows;
  a.f.hidden = (int)hidden;
  a.f.eps = eps;
  a.f.rms = rms ? 1 : 0;
  a.f.zero_centered = zero_centered_gamma ? 1 : 0;
  a.q = quant_out(*q);
  a.padded_rows = padded_rows(a.q);
  const int cls = class_of(q->format), per = (int)(16 / es);
  NormPlan p;
  if (vec) {
    const int64_t wide = mx_tiled(q->format) ? (hidden + 31) / 32 * 32 : hidden;
    const int64_t slots = (wide + per - 1) / per;
    int sms = 0;
    const cudaError_t e = (cudaError_t)device_sm_count(&sms);
    if (e != cudaSuccess) return cuda_fail(e);
    p = norm_plan((int)slots, q->format == MX_FP8_BLOCK ? 128 / per : 8);
    const NormPlan few = few_plan((int)slots, rows, sms);
    if (few.n > 0 && few.n < p.n) {
      a.order_lanes = p.lanes > 0 ? p.lanes : p.block;
      a.order_n = p.n;
      p = few;
    }
  }
  if (!vec && hidden > 128 * kChunks) {
    p.lanes = -2;
    p.block = (int)((hidden + 128 * kChunks - 1) / (128 * kChunks)) * 32;
  }
  const void* fn = dtype == LN_F32 ? mx_norm_table_f32(cls, p.lanes, p.n)
                   : dtype == LN_BF16 ? mx_norm_table_bf16(cls, p.lanes, p.n)
                                      : mx_norm_table_f16(cls, p.lanes, p.n);
  int64_t grid = a.padded_rows;
  if (p.lanes > 0) grid = (a.padded_rows + 256 / p.lanes - 1) / (256 / p.lanes);
  if (p.lanes == -1) grid = (a.padded_rows + 7) / 8;
  size_t smem = 0;
  if (p.lanes < 0 && cls != 0) smem = (size_t)p.block / 32 * kChunks * 128 * sizeof(float);
  if (p.lanes == 0 && a.order_n > 0) smem = 2 * (size_t)p.n * p.block * sizeof(float2);
  void* args[] = {&a};
  const cudaError_t e = launch_overlapped(fn, dim3((unsigned)grid), dim3(p.block), args, smem, stream);
  return e == cudaSuccess ? LN_OK : cuda_fail(e);
}

ln_status mx_quantize(const void* x, int64_t x_row, int transpose, const mx_matrix* q,
                      cudaStream_t stream, ln_dtype dtype) {
  if (q == nullptr) return LN_ERR_NULL;
  if (!known_dtype(dtype) || !known_format(q->format)) return LN_ERR_UNSUPPORTED;
  ln_status st = check_matrix(*q);
  if (st != LN_OK) return st;
  const int64_t rows = transpose ? q->cols : q->rows, cols = transpose ? q->rows : q->cols;
  const size_t es = elem_size(dtype);
  if (q->rows > 0 && x == nullptr) return LN_ERR_NULL;
  if (x_row < 0 || (rows > 1 && x_row > INT64_MAX / 16 / rows)) return LN_ERR_INVALID;
  if (!aligned(x, es)) return LN_ERR_ALIGN;
  const size_t span = q->rows > 0 ? (size_t)((rows - 1) * x_row + cols) * es : 0;
  const Range outs[] = {codes_range(*q), scales_range(*q)};
  const Range ins[] = {{x, span}, mul_range(*q)};
  if (any_overlap(outs, 2, ins, 2)) return LN_ERR_INVALID;
  if (q->rows == 0) return LN_OK;
  int sms = 0;
  cudaError_t e = (cudaError_t)device_sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  QuantArgs a = {};
  a.x = x;
  a.x_row = x_row;
  a.q = quant_out(*q);
  a.vec = aligned(x, 16) && (rows == 1 || (x_row * es) % 16 == 0);
  a.vec_codes = aligned(q->codes, 16);
  a.padded_rows = padded_rows(a.q);
  e = by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    switch (q->format) {
      case MX_FP8_ROW: return launch_quantize<T, MX_FP8_ROW>(a, transpose, sms, stream);
      case MX_FP8_BLOCK: return launch_quantize<T, MX_FP8_BLOCK>(a, transpose, sms, stream);
      case MX_MXFP8: return launch_quantize<T, MX_MXFP8>(a, transpose, sms, stream);
      case MX_MXFP4: return launch_quantize<T, MX_MXFP4>(a, transpose, sms, stream);
      default: return launch_quantize<T, MX_NVFP4>(a, transpose, sms, stream);
    }
  });
  return e == cudaSuccess ? LN_OK : cuda_fail(e);
}

ln_status mx_dequantize(const mx_matrix* q, void* y, int64_t y_row, cudaStream_t stream,
                        ln_dtype dtype) {
  if (q == nullptr) return LN_ERR_NULL;
  if (!known_dtype(dtype) || !known_format(q->format)) return LN_ERR_UNSUPPORTED;
  ln_status st = check_matrix(*q);
  if (st != LN_OK) return st;
  const size_t es = elem_size(dtype);
  if (q->rows > 0 && y == nullptr) return LN_ERR_NULL;
  if (y_row < q->cols || (q->rows > 1 && y_row > INT64_MAX / 16 / q->rows)) return LN_ERR_INVALID;
  if (!aligned(y, es)) return LN_ERR_ALIGN;
  const size_t span = q->rows > 0 ? (size_t)((q->rows - 1) * y_row + q->cols) * es : 0;
  const Range outs[] = {{y, span}};
  const Range ins[] = {codes_range(*q), scales_range(*q), mul_range(*q)};
  if (any_overlap(outs, 1, ins, 3)) return LN_ERR_INVALID;
  if (q->rows == 0) return LN_OK;
  int sms = 0;
  cudaError_t e = (cudaError_t)device_sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  QuantOut o = quant_out(*q);
  const bool vec = aligned(y, 16) && (q->rows == 1 || (y_row * es) % 16 == 0);
  bool vec_codes = o.pitch % 8 == 0 && aligned(q->codes, 8);
  int shift = row_shift(q->cols, 1);
  const dim3 grid = row_grid(q->rows, q->cols, shift, sms);
  e = by_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const auto run = [&](auto fmt) {
      constexpr int FMT = decltype(fmt)::value;
      const void* fn = vec ? (const void*)dequant_kernel<T, FMT, false> : (const void*)dequant_kernel<T, FMT, true>;
      void* args[] = {&o, &y, &y_row, &vec_codes, &shift};
      return launch_overlapped(fn, grid, dim3(kQuantThreads), args, 0, stream);
    };
    switch (q->format) {
      case MX_MXFP8: return run(Format<MX_MXFP8>());
      case MX_MXFP4: return run(Format<MX_MXFP4>());
      case MX_NVFP4: return run(Format<MX_NVFP4>());
      default: return run(Format<MX_FP8_ROW>());
    }
  });
  return e == cudaSuccess ? LN_OK : cuda_fail(e);
}

}  // extern "C"
