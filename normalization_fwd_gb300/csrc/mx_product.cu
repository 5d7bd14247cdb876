// The product of two microscaled matrices: C entry point, argument checks,
// tensor maps and launch plan.
#include <math.h>

#include <algorithm>
#include <mutex>
#include <vector>

#include "../../include/normfuse.h"
#include "launch.h"
#include "mx_check.h"
#include "mx_product_kernels.cuh"
#include "tensor_map.h"

namespace nf {

cudaError_t take_error_product(cudaStream_t st, unsigned* out) { return take_tu_error(st, out); }

namespace {

ln_status cuda_fail(cudaError_t e) {
  nf_set_last_cuda_error((int)e);
  return LN_ERR_CUDA;
}

// Codes as rows of bytes, boxes of 128 bytes by `rows`, swizzled.
cudaError_t codes_map(Encode encode, const QuantOut& q, int rows, CUtensorMap* map) {
  const cuuint64_t dims[2] = {(cuuint64_t)q.pitch, (cuuint64_t)q.rows}, strides[1] = {(cuuint64_t)q.pitch};
  const cuuint32_t box[2] = {kChunkBytes, (cuuint32_t)rows}, step[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q.codes, dims, strides, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// Scales as tiles of 128 words, [row tiles, tiles of a row], boxes of
// `row_tiles` by `tiles`.
cudaError_t scales_map(Encode encode, const QuantOut& q, int tiles, int row_tiles, CUtensorMap* map) {
  const cuuint64_t across = (cuuint64_t)(q.blocks + 3) / 4;
  const cuuint64_t dims[3] = {128, across, (cuuint64_t)(q.rows + 127) / 128}, strides[2] = {512, across * 512};
  const cuuint32_t box[3] = {128, (cuuint32_t)tiles, (cuuint32_t)row_tiles}, step[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, q.scales, dims, strides, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Whether the device places clusters of so many CTAs; asked once for a kernel, a
// device, a size and the shared memory.
cudaError_t places(const void* fn, int block, size_t smem, int cluster, bool* yes) {
  struct Entry {
    const void* fn;
    int device, cluster;
    size_t smem;
    bool yes;
  };
  static std::mutex mu;
  static std::vector<Entry> kept;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  for (const Entry& k : kept)
    if (k.fn == fn && k.device == dev && k.cluster == cluster && k.smem == smem) {
      *yes = k.yes;
      return cudaSuccess;
    }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
  if (e != cudaSuccess) return e;
  *yes = n > 0;
  kept.push_back({fn, dev, cluster, smem, *yes});
  return cudaSuccess;
}

constexpr uint32_t kSmemTarget = 200 * 1024;
constexpr uint32_t kPairSmem = 225 * 1024;   // with 1 KB for alignment and the barriers: 226.2 of 227

template <typename T, int FMT, bool SWAP>
cudaError_t launch_tiles(ProductArgs p, int sms, cudaStream_t st) {
  const QuantOut &lanes = SWAP ? p.b : p.a, &columns = SWAP ? p.a : p.b;
  const void* fn = (const void*)product_tile_kernel<T, FMT, SWAP>;
  p.lane_tiles = (int)((lanes.rows + kTileLanes - 1) / kTileLanes);
  const int64_t tiles = p.lane_tiles * ((columns.rows + p.cols - 1) / p.cols);
  // K over so many CTAs as fill the SMs, each with two chunks at least.
  p.splits = 1;
  while (p.splits < 8 && tiles * p.splits * 2 <= sms && p.chunks >= p.splits * 4) p.splits *= 2;
  const uint32_t stage = stage_bytes<FMT>(p.cols);
  p.stages = (int)std::min<uint32_t>(kMaxStages, kSmemTarget / stage);
  static_assert(kScaleCol + kMaxStages * 8 * chunk_tiles<FMT>() <= kTmemCols, "scales' buffers");
  const size_t smem = std::max<size_t>((size_t)p.stages * stage, (SWAP ? p.cols : kTileLanes) * kResultPitch * 4) + 1024;
  p.idesc = instr_desc(FMT, kTileLanes, p.cols);
  if (tiles * p.splits > INT32_MAX) return cudaErrorInvalidValue;

  CUtensorMap maps[4];
  Encode encode;
  cudaError_t e = encoder(&encode);
  if (e == cudaSuccess) e = codes_map(encode, lanes, kTileLanes, &maps[0]);
  if (e == cudaSuccess) e = scales_map(encode, lanes, chunk_tiles<FMT>(), 1, &maps[1]);
  if (e == cudaSuccess) e = codes_map(encode, columns, p.cols, &maps[2]);
  if (e == cudaSuccess) e = scales_map(encode, columns, chunk_tiles<FMT>(), 1, &maps[3]);
  if (e == cudaSuccess) e = (cudaError_t)allow_dyn_smem(fn, smem);
  if (e != cudaSuccess) return e;

  // no larger clusters than the device places
  for (bool yes = false; p.splits > 1 && !yes;) {
    e = places(fn, kTileThreads, smem, p.splits, &yes);
    if (e != cudaSuccess) return e;
    if (!yes) p.splits /= 2;
  }
  void* args[] = {&maps[0], &maps[1], &maps[2], &maps[3], &p};
  return launch_overlapped(fn, dim3((unsigned)(tiles * p.splits)), dim3(kTileThreads), args, smem, st, p.splits);
}

// *placed: false where the device does not place a pair of CTAs of this size.
template <typename T, int FMT, int WN>
cudaError_t launch_pairs(ProductArgs p, int sms, cudaStream_t st, bool* placed) {
  const void* fn = (const void*)product_pair_kernel<T, FMT, WN>;
  p.tiles_m = (int)((p.a.rows + 255) / 256);
  p.tiles_n = (int)((p.b.rows + WN - 1) / WN);
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  constexpr uint32_t kStage = pair_stage_step<FMT>(WN);
  p.stages = (int)std::min<uint32_t>(kMaxStages, (kPairSmem - 8 * kPieceBytes) / kStage);
  static_assert(256 + std::min<uint32_t>(kMaxStages, (kPairSmem - 8 * kPieceBytes) / kStage) * 4 *
                          chunk_tiles<FMT>() * (1 + WN / 128) <= kTmemCols, "scales' buffers");
  const size_t smem = (size_t)p.stages * kStage + 8 * kPieceBytes + 1024;
  p.idesc = instr_desc(FMT, 256, WN);
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  CUtensorMap maps[4];
  Encode encode;
  cudaError_t e = encoder(&encode);
  if (e == cudaSuccess) e = codes_map(encode, p.a, 128, &maps[0]);
  if (e == cudaSuccess) e = scales_map(encode, p.a, chunk_tiles<FMT>(), 1, &maps[1]);
  if (e == cudaSuccess) e = codes_map(encode, p.b, WN / 2, &maps[2]);
  if (e == cudaSuccess) e = scales_map(encode, p.b, chunk_tiles<FMT>(), WN / 128, &maps[3]);
  if (e == cudaSuccess) e = (cudaError_t)allow_dyn_smem(fn, smem);
  if (e != cudaSuccess) return e;
  e = places(fn, kPairThreads, smem, 2, placed);
  if (e != cudaSuccess || !*placed) return e;
  void* args[] = {&maps[0], &maps[1], &maps[2], &maps[3], &p};
  return launch_overlapped(fn, dim3((unsigned)std::min<int64_t>(2 * tiles, sms / 2 * 2)), dim3(kPairThreads), args,
                           smem, st, 2);
}

template <typename T, int FMT>
cudaError_t launch_format(ProductArgs p, int sms, cudaStream_t st) {
  p.chunks = (int)((p.a.pitch + kChunkBytes - 1) / kChunkBytes);
  p.steps = (int)((p.a.pitch + 31) / 32);
  if (p.a.rows <= 64) {
    p.cols = p.a.rows <= 16 ? 16 : p.a.rows <= 32 ? 32 : 64;
    return launch_tiles<T, FMT, true>(p, sms, st);
  }
  // Pairs of CTAs from where single tiles are more than the SMs (nvfp4 4096 x 4096
  // x 8192 49 us against 101 as single tiles, 512 x 8192 x 8192 18.5 against 29.5; 256
  // x 8192 x 8192, 128 tiles, 15.6 single, 14.9 as narrow pairs, 17.5 as wide ones).
  // Tiles of 256 columns unless they take more than 5 rounds for 8 of half the width
  // (the first 49 us against 71, mxfp8 2100 x 2300 x 800 19.0 against 18.3): a tile of
  // 128 takes some five eighths of one of 256, as its operands are copied for half the
  // results.
  const int64_t tm = (p.a.rows + 255) / 256, tn = (p.b.rows + 127) / 128, pairs = sms / 2;
  if (p.a.rows > 128 && pairs > 0 && tm * tn * 2 > sms) {
    const int64_t narrow = (tm * tn + pairs - 1) / pairs, wide = (tm * ((tn + 1) / 2) + pairs - 1) / pairs;
    bool placed = false;
    const cudaError_t e = wide * 8 <= narrow * 5 ? launch_pairs<T, FMT, 256>(p, sms, st, &placed)
                                                 : launch_pairs<T, FMT, 128>(p, sms, st, &placed);
    if (e != cudaSuccess || placed) return e;
  }
  p.cols = 128;
  return launch_tiles<T, FMT, false>(p, sms, st);
}

template <typename T>
cudaError_t launch_product(const ProductArgs& p, int sms, cudaStream_t st) {
  switch (p.a.fmt) {
    case MX_MXFP8: return launch_format<T, MX_MXFP8>(p, sms, st);
    case MX_MXFP4: return launch_format<T, MX_MXFP4>(p, sms, st);
    default: return launch_format<T, MX_NVFP4>(p, sms, st);
  }
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
  const auto rows_of = [&](const void* t, int64_t row) {
    return Strided{t, {M, 1, 1}, {row * (int64_t)es, 0, 0}, N * (int64_t)es};
  };
  const Strided results = rows_of(out, out_row), added = residual != nullptr ? rows_of(residual, residual_row) : Strided();
  const Range outs[] = {results.range(), {psum, psum ? tiles : 0}, {psq, psq ? tiles : 0}};
  const Range ins[] = {codes_range(*a), scales_range(*a), mul_range(*a), codes_range(*b), scales_range(*b),
                       mul_range(*b), {bias, (size_t)N * es}};
  const Range residual_range[] = {added.range()};
  if (any_overlap(outs, 3, ins, 7) || any_overlap(outs + 1, 2, residual_range, 1)) return LN_ERR_INVALID;
  // in place, or apart: two slices of one buffer are
  const bool in_place = residual == out && (residual_row == out_row || M == 1);
  if (!in_place && may_overlap(results, added)) return LN_ERR_INVALID;
  int sms = 0;
  cudaError_t e = (cudaError_t)device_sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
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
  const auto vec = [&](const void* t, int64_t row) { return aligned(t, 16) && (M == 1 || row * es % 16 == 0); };
  p.vec = vec(out, out_row) && (residual == nullptr || vec(residual, residual_row)) && aligned(bias, 16);
  e = by_dtype(dtype, [&](auto t) { return launch_product<decltype(t)>(p, sms, stream); });
  return e == cudaSuccess ? LN_OK : cuda_fail(e);
}

}  // extern "C"
