// Group norm kernels, bf16.
#include "gn_table.cuh"

namespace nf {
const void* gn_table_bf16(bool bwd, bool cluster, bool vec, int act) {
  return vec ? gn_table<bf16, Vec<bf16>::N>(bwd, cluster, act) : gn_table<bf16, 1>(bwd, cluster, act);
}
}  // namespace nf
