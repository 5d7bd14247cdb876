// Rotary position kernels, f32.
#include "rope_table.cuh"

namespace nf {
const void* rope_table_f32(int vec, int ns, bool inter, bool aligned, bool full, bool bwd) {
  return rope_table<float>(vec, ns, inter, aligned, full, bwd);
}
}  // namespace nf
