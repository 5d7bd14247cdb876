// (direction, form, width, activation) -> group norm kernel of one dtype.
#pragma once

#include "gn_kernels.cuh"

namespace nf {

template <typename T, int VEC, int ACT> const void* gn_form(bool bwd, bool cluster) {
  if (cluster)
    return bwd ? (const void*)gn_bwd_cluster_kernel<T, VEC, ACT>
               : (const void*)gn_fwd_cluster_kernel<T, VEC, ACT>;
  return bwd ? (const void*)gn_bwd_kernel<T, VEC, ACT> : (const void*)gn_fwd_kernel<T, VEC, ACT>;
}
template <typename T, int VEC> const void* gn_act(bool bwd, bool cluster, int act) {
  if (act == kActSilu) return gn_form<T, VEC, kActSilu>(bwd, cluster);
  if (act == kActGelu) return gn_form<T, VEC, kActGelu>(bwd, cluster);
  return gn_form<T, VEC, kActNone>(bwd, cluster);
}
template <typename T> const void* gn_table(bool bwd, bool cluster, bool vec, int act) {
  return vec ? gn_act<T, Vec<T>::N>(bwd, cluster, act) : gn_act<T, 1>(bwd, cluster, act);
}

}  // namespace nf
