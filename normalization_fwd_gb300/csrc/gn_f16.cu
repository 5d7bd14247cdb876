// Group norm kernels, f16.
#include "gn_table.cuh"

namespace nf {
const void* gn_table_f16(bool bwd, bool vec, int act) {
  return vec ? gn_table<f16, Vec<f16>::N>(bwd, act) : gn_table<f16, 1>(bwd, act);
}
}  // namespace nf
