// Group norm kernels, f32.
#include "gn_table.cuh"

namespace nf {
const void* gn_table_f32(bool bwd, bool cluster, bool vec, int act) {
  return vec ? gn_table<float, Vec<float>::N>(bwd, cluster, act) : gn_table<float, 1>(bwd, cluster, act);
}
}  // namespace nf
