// (direction, form, alignment, activation) -> group norm kernel of one dtype.
#pragma once

#include "gn_kernels.cuh"

namespace nf {

template <typename T, int ACT, bool FINE> const void* gn_form(bool bwd, bool cluster) {
  constexpr int V = Vec<T>::N;
  if (bwd) return (const void*)gn_bwd_kernel<T, V, ACT, FINE>;
  return cluster ? (const void*)gn_fwd_cluster_kernel<T, V, ACT, FINE>
                 : (const void*)gn_fwd_kernel<T, V, ACT, FINE>;
}
template <typename T, bool FINE> const void* gn_act(bool bwd, bool cluster, int act) {
  if (act == kActSilu) return gn_form<T, kActSilu, FINE>(bwd, cluster);
  if (act == kActGelu) return gn_form<T, kActGelu, FINE>(bwd, cluster);
  return gn_form<T, kActNone, FINE>(bwd, cluster);
}
template <typename T> const void* gn_table(bool bwd, bool cluster, bool fine, int act) {
  return fine ? gn_act<T, true>(bwd, cluster, act) : gn_act<T, false>(bwd, cluster, act);
}

}  // namespace nf
