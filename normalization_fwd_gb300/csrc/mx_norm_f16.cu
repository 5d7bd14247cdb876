// Norms with quantised results, f16.
#include "mx_norm_kernels.cuh"

namespace nf {
const void* mx_norm_table_f16(int cls, int lanes, int n) { return mx_norm_table<f16>(cls, lanes, n); }
}  // namespace nf
