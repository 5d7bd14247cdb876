// Group norm kernels, f32.
#include "gn_table.cuh"

namespace nf {
const void* gn_table_f32(bool bwd, bool vec, int act) {
  return vec ? gn_table<float, Vec<float>::N>(bwd, act) : gn_table<float, 1>(bwd, act);
}
}  // namespace nf
