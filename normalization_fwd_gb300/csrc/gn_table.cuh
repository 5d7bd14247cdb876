// (direction, form, width, threads, activation) -> group norm kernel of one dtype.
#pragma once

#include "gn_kernels.cuh"

namespace nf {

template <typename T, int VEC, int TH, int ACT> const void* gn_form(bool bwd, bool cluster) {
  if (cluster)
    return bwd ? (const void*)gn_bwd_cluster_kernel<T, VEC, TH, ACT>
               : (const void*)gn_fwd_cluster_kernel<T, VEC, TH, ACT>;
  // More than one launch: large calls, for which 256 threads are enough.
  if constexpr (TH > 256)
    return nullptr;
  else
    return bwd ? (const void*)gn_bwd_kernel<T, VEC, TH, ACT>
               : (const void*)gn_fwd_kernel<T, VEC, TH, ACT>;
}
template <typename T, int VEC, int TH> const void* gn_act(bool bwd, bool cluster, int act) {
  if (act == kActSilu) return gn_form<T, VEC, TH, kActSilu>(bwd, cluster);
  if (act == kActGelu) return gn_form<T, VEC, TH, kActGelu>(bwd, cluster);
  return gn_form<T, VEC, TH, kActNone>(bwd, cluster);
}
template <typename T> const void* gn_table(bool bwd, bool cluster, bool vec, int threads, int act) {
  if (!vec) return gn_act<T, 1, 256>(bwd, cluster, act);
  return threads == 512 ? gn_act<T, Vec<T>::N, 512>(bwd, cluster, act)
                        : gn_act<T, Vec<T>::N, 256>(bwd, cluster, act);
}

}  // namespace nf
