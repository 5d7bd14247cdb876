// Argument checks of quantised matrices, shared by the entry points that take them.
#pragma once

#include "mx_formats.cuh"
#include "validate.h"

namespace nf {

constexpr int64_t kMxMaxSide = 1ll << 31;   // rows and columns are below it

inline bool known_format(mx_format f) { return f >= MX_FP8_ROW && f <= MX_NVFP4; }
inline bool fits(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 1 && rows < kMxMaxSide - 128 && cols < kMxMaxSide - 128;
}
inline size_t code_bytes(int fmt, int64_t rows, int64_t cols) {
  return (size_t)rows * (size_t)mx_pitch(fmt, cols);
}
inline size_t scale_bytes(int fmt, int64_t rows, int64_t cols) {
  const int64_t blocks = mx_blocks(fmt, cols);
  if (!mx_tiled(fmt)) return (size_t)rows * (size_t)blocks * 4;
  return (size_t)((rows + 127) / 128) * (size_t)((blocks + 3) / 4) * 512;
}
inline Range codes_range(const mx_matrix& m) { return {m.codes, code_bytes(m.format, m.rows, m.cols)}; }
inline Range scales_range(const mx_matrix& m) { return {m.scales, scale_bytes(m.format, m.rows, m.cols)}; }
inline Range mul_range(const mx_matrix& m) {
  return {m.format == MX_NVFP4 ? m.mul : nullptr, m.format == MX_NVFP4 && m.mul ? 4u : 0u};
}
// Shape, pointers and their alignment: microscaled codes and scales on 16 bytes
// (the copies of the product start there), scales in fp32 on 4. The range of a
// matrix stays within 63 bits: 2^31 rows by 2^31 bytes.
inline ln_status check_matrix(const mx_matrix& m) {
  if (!known_format(m.format)) return LN_ERR_UNSUPPORTED;
  if (!fits(m.rows, m.cols)) return LN_ERR_SHAPE;
  if (m.rows > 0 && (m.codes == nullptr || m.scales == nullptr)) return LN_ERR_NULL;
  if (mx_tiled(m.format) ? !aligned(m.codes, 16) || !aligned(m.scales, 16) : !aligned(m.scales, 4))
    return LN_ERR_ALIGN;
  if (m.format == MX_NVFP4 && !aligned(m.mul, 4)) return LN_ERR_ALIGN;
  return LN_OK;
}
inline QuantOut quant_out(const mx_matrix& m) {
  QuantOut q;
  q.codes = static_cast<unsigned char*>(m.codes);
  q.scales = m.scales;
  q.mul = m.mul;
  q.rows = m.rows;
  q.cols = m.cols;
  q.pitch = mx_pitch(m.format, m.cols);
  q.blocks = mx_blocks(m.format, m.cols);
  q.fmt = m.format;
  return q;
}

}  // namespace nf
