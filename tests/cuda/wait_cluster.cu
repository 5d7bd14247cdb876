// Test helper (built by tests/test_gpu_mx_wait.py): the wait of the product and of
// the tensor-map transposes, on a barrier of this kernel's own at which nothing
// arrives and on one at which everything has, with a short limit. Nothing is in
// flight when it returns.
#include <stdint.h>

#include "tcgen05.cuh"

namespace {

__global__ void waits(int* gave_up, int* came, long long* cycles, long long limit) {
  __shared__ __align__(8) uint64_t never, there;
  if (threadIdx.x == 0) {
    nf::mbar_init(&never, 1);   // expects one arrival that never comes
    nf::mbar_init(&there, 1);
    nf::fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) nf::mbar_arrive_cluster(nf::smem_addr(&there));
  if (nf::mbar_wait_cluster(&there, 0, limit)) atomicAdd(came, 1);
  if (nf::mbar_ready_cluster(nf::smem_addr(&there), 0) && !nf::mbar_ready_cluster(nf::smem_addr(&never), 0))
    atomicAdd(came, 1);
  const long long t0 = clock64();
  if (!nf::mbar_wait_cluster(&never, 0, limit)) {
    atomicAdd(gave_up, 1);
    atomicOr(&nf::g_tu_error, nf::kErrWaitTimeout);
  }
  if (threadIdx.x == 0) *cycles = clock64() - t0;
}

}  // namespace

extern "C" int wait_cluster_launch(int* gave_up, int* came, long long* cycles, long long limit, int threads) {
  waits<<<1, threads>>>(gave_up, came, cycles, limit);
  return (int)cudaGetLastError();
}
extern "C" int wait_cluster_error(unsigned* flags) { return (int)nf::take_tu_error(0, flags); }
