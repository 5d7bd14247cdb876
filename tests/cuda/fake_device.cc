// A device that is not there, for the group norm's and the rotary positions'
// entry points: everything that gn.cu and rope.cu call to ask about the device
// or to launch is defined here instead, and counted. Linked with those two
// sources, it shows on a machine without a GPU what a call would launch where
// there is one, and whether it would launch at all.
#include <cuda_runtime.h>
#include <stddef.h>

namespace {
int g_sms = 152, g_most_cluster = 16;
int g_launches, g_grid, g_cluster, g_finalizes, g_memsets;
const int kKernel = 0;   // stands for every kernel

cudaError_t launched(dim3 grid, int cluster) {
  ++g_launches;
  g_grid = (int)grid.x;
  g_cluster = cluster;
  return cudaSuccess;
}
}  // namespace

namespace nf {
int device_sm_count(int* sms) {
  *sms = g_sms;
  return (int)cudaSuccess;
}
int cluster_limit(const void*, int, size_t, int* out) {
  *out = g_most_cluster;
  return (int)cudaSuccess;
}
int allow_dyn_smem(const void*, size_t) { return (int)cudaSuccess; }
cudaError_t launch_bwd_finalize(const float*, int, int, int, bool, void*, void*, void*, int,
                                cudaStream_t, int) {
  ++g_finalizes;
  return cudaSuccess;
}
#define FAKE_TABLES(NAME)                                                              \
  const void* gn_table_##NAME(bool, bool, bool, int) { return &kKernel; }              \
  const void* rope_table_##NAME(int, int, bool, bool, bool, bool) { return &kKernel; }
FAKE_TABLES(f32)
FAKE_TABLES(bf16)
FAKE_TABLES(f16)
}  // namespace nf

extern "C" {
void nf_set_last_cuda_error(int) {}

// The CUDA runtime's part.
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void*, void**) {
  int cluster = 1;
  for (unsigned i = 0; i < cfg->numAttrs; ++i)
    if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension)
      cluster = (int)cfg->attrs[i].val.clusterDim.x;
  if (cluster > g_most_cluster) return cudaErrorInvalidClusterSize;
  return launched(cfg->gridDim, cluster);
}
cudaError_t cudaLaunchKernel(const void*, dim3 grid, dim3, void**, size_t, cudaStream_t) {
  return launched(grid, 1);
}
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) {
  ++g_memsets;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}

// The test's part. out: kernel launches, the last one's grid and cluster,
// finalize launches, memsets.
void fake_reset(int sms, int most_cluster) {
  g_sms = sms;
  g_most_cluster = most_cluster;
  g_launches = g_grid = g_cluster = g_finalizes = g_memsets = 0;
}
void fake_counts(int* out) {
  out[0] = g_launches;
  out[1] = g_grid;
  out[2] = g_cluster;
  out[3] = g_finalizes;
  out[4] = g_memsets;
}
}
