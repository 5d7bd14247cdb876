// Norms with quantised results, f32.
#include "mx_norm_kernels.cuh"

namespace nf {
const void* mx_norm_table_f32(int cls, int lanes, int n) { return mx_norm_table<float>(cls, lanes, n); }
}  // namespace nf
