// Group norm kernels, bf16.
#include "gn_table.cuh"

namespace nf {
const void* gn_table_bf16(bool bwd, bool cluster, bool fine, int act) {
  return gn_table<bf16>(bwd, cluster, fine, act);
}
}  // namespace nf
