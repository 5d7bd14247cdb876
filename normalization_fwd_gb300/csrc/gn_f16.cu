// Group norm kernels, f16.
#include "gn_table.cuh"

namespace nf {
const void* gn_table_f16(bool bwd, bool cluster, bool fine, int act) {
  return gn_table<f16>(bwd, cluster, fine, act);
}
}  // namespace nf
