// (direction, activation) -> group norm kernel of one dtype and vector width.
#pragma once

#include "gn_kernels.cuh"

namespace nf {

template <typename T, int VEC> const void* gn_table(bool bwd, int act) {
  if (act == kActSilu)
    return bwd ? (const void*)gn_bwd_kernel<T, VEC, kActSilu>
               : (const void*)gn_fwd_kernel<T, VEC, kActSilu>;
  if (act == kActGelu)
    return bwd ? (const void*)gn_bwd_kernel<T, VEC, kActGelu>
               : (const void*)gn_fwd_kernel<T, VEC, kActGelu>;
  return bwd ? (const void*)gn_bwd_kernel<T, VEC, kActNone>
             : (const void*)gn_fwd_kernel<T, VEC, kActNone>;
}

}  // namespace nf
