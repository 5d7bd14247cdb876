// Group norm kernels, f16.
#include "gn_table.cuh"

namespace nf {
const void* gn_table_f16(bool bwd, bool cluster, bool vec, int act) {
  return vec ? gn_table<f16, Vec<f16>::N>(bwd, cluster, act) : gn_table<f16, 1>(bwd, cluster, act);
}
}  // namespace nf
