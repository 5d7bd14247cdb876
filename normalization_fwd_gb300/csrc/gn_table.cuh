// (direction, form, activation) -> group norm kernel of one dtype and vector width.
#pragma once

#include "gn_kernels.cuh"

namespace nf {

template <typename T, int VEC, int ACT> const void* gn_form(bool bwd, bool cluster) {
  if (cluster)
    return bwd ? (const void*)gn_bwd_cluster_kernel<T, VEC, ACT>
               : (const void*)gn_fwd_cluster_kernel<T, VEC, ACT>;
  return bwd ? (const void*)gn_bwd_kernel<T, VEC, ACT> : (const void*)gn_fwd_kernel<T, VEC, ACT>;
}
template <typename T, int VEC> const void* gn_table(bool bwd, bool cluster, int act) {
  if (act == kActSilu) return gn_form<T, VEC, kActSilu>(bwd, cluster);
  if (act == kActGelu) return gn_form<T, VEC, kActGelu>(bwd, cluster);
  return gn_form<T, VEC, kActNone>(bwd, cluster);
}

}  // namespace nf
