// Norms with quantised results, bf16.
#include "mx_norm_kernels.cuh"

namespace nf {
const void* mx_norm_table_bf16(int cls, int lanes, int n) { return mx_norm_table<bf16>(cls, lanes, n); }
}  // namespace nf
