// Group norm kernels, f32.
#include "gn_table.cuh"

namespace nf {
const void* gn_table_f32(bool bwd, bool cluster, bool fine, int act) {
  return gn_table<float>(bwd, cluster, fine, act);
}
}  // namespace nf
