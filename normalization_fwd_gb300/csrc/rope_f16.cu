// Rotary position kernels, f16.
#include "rope_table.cuh"

namespace nf {
const void* rope_table_f16(int vec, int ns, bool inter, bool aligned, bool full, bool bwd) {
  return rope_table<f16>(vec, ns, inter, aligned, full, bwd);
}
}  // namespace nf
