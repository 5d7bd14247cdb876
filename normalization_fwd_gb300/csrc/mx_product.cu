// The product of two microscaled matrices: C entry point, argument checks and
// launch plan.
#include <math.h>

#include "../../include/normfuse.h"
#include "launch.h"
#include "mx_check.h"
#include "mx_product_kernels.cuh"

namespace nf {
namespace {

ln_status cuda_fail(cudaError_t e) {
  nf_set_last_cuda_error((int)e);
  return LN_ERR_CUDA;
}

}  // namespace
}  // namespace nf

using namespace nf;

extern "C" {

ln_status mx_product(const mx_matrix* a, const mx_matrix* b, float alpha, const void* bias,
                     const void* residual, int64_t residual_row, void* out, int64_t out_row,
                     float* psum, float* psq, cudaStream_t stream, ln_dtype dtype) {
  if (a == nullptr || b == nullptr) return LN_ERR_NULL;
  if (!known_dtype(dtype) || !known_format(a->format)) return LN_ERR_UNSUPPORTED;
  if (a->format != b->format || !mx_tiled(a->format)) return LN_ERR_UNSUPPORTED;
  if (a->cols != b->cols) return LN_ERR_SHAPE;
  ln_status st = check_matrix(*a);
  if (st == LN_OK) st = check_matrix(*b);
  if (st != LN_OK) return st;
  const int64_t M = a->rows, N = b->rows;
  if (!isfinite(alpha)) return LN_ERR_INVALID;
  if (M > 0 && N > 0 && out == nullptr) return LN_ERR_NULL;
  if ((psum == nullptr) != (psq == nullptr)) return LN_ERR_NULL;
  const size_t es = elem_size(dtype);
  const auto spans = [&](int64_t row) { return row >= N && row <= INT64_MAX / 16 / (M > 0 ? M : 1); };
  if (!spans(out_row) || (residual != nullptr && !spans(residual_row))) return LN_ERR_INVALID;
  if (!aligned(bias, es) || !aligned(residual, es) || !aligned(out, es)) return LN_ERR_ALIGN;
  if (!aligned(psum, 4) || !aligned(psq, 4)) return LN_ERR_ALIGN;
  if (M == 0 || N == 0) return LN_OK;
  const size_t tiles = (size_t)M * (size_t)((N + 127) / 128) * 4;
  const Range outs[] = {{out, (size_t)((M - 1) * out_row + N) * es}, {psum, psum ? tiles : 0}, {psq, psq ? tiles : 0}};
  const bool in_place = residual == out && residual_row == out_row;
  const Range ins[] = {codes_range(*a), scales_range(*a), mul_range(*a), codes_range(*b), scales_range(*b),
                       mul_range(*b), {bias, (size_t)N * es},
                       {in_place ? nullptr : residual, (size_t)((M - 1) * residual_row + N) * es}};
  if (any_overlap(outs, 3, ins, 8)) return LN_ERR_INVALID;
  ProductArgs p = {};
  p.a = quant_out(*a);
  p.b = quant_out(*b);
  p.alpha = alpha;
  p.bias = bias;
  p.residual = residual;
  p.residual_row = residual_row;
  p.out = out;
  p.out_row = out_row;
  p.psum = psum;
  p.psq = psq;
  const cudaError_t e = by_dtype(dtype, [&](auto t) { return product_launch<decltype(t)>(p, stream); });
  return e == cudaSuccess ? LN_OK : cuda_fail(e);
}

}  // extern "C"
