// Group norm kernels, bf16.
#include "gn_table.cuh"

namespace nf {
const void* gn_table_bf16(bool bwd, bool vec, int act) {
  return vec ? gn_table<bf16, Vec<bf16>::N>(bwd, act) : gn_table<bf16, 1>(bwd, act);
}
}  // namespace nf
