// (vector width, slots a lane, layout, direction) -> rotary kernel of one
// dtype. A lane holds at most 8 pairs, so a head of up to 512 elements takes
// 1, 2, ... or 8 / VEC slots of VEC pairs a lane (backward in vectors: 1 or 8 / VEC).
#pragma once

#include "rope_kernels.cuh"

namespace nf {

template <typename T, int VEC, int NS, bool INTER, bool ALIGNED, bool FULL>
const void* rope_dir(bool bwd) {
  if (!bwd) return (const void*)rope_kernel<T, VEC, NS, INTER, ALIGNED, FULL, false>;
  if constexpr (NS == 1 || NS == 8 / VEC || VEC == 1)
    return (const void*)rope_kernel<T, VEC, NS, INTER, ALIGNED, FULL, true>;
  return nullptr;
}
template <typename T, int VEC, bool INTER, bool ALIGNED>
const void* rope_ns(int ns, bool full, bool bwd) {
  // Heads of 64, 128 and 256 elements that are rotated whole, in vectors.
  if constexpr (VEC == Vec<T>::N && ALIGNED)
    if (ns == 1 && full) return rope_dir<T, VEC, 1, INTER, ALIGNED, true>(bwd);
  if (ns == 1) return rope_dir<T, VEC, 1, INTER, ALIGNED, false>(bwd);
  if constexpr (VEC <= 4)
    if (ns == 2) return rope_dir<T, VEC, 2, INTER, ALIGNED, false>(bwd);
  if constexpr (VEC <= 2)
    if (ns == 4) return rope_dir<T, VEC, 4, INTER, ALIGNED, false>(bwd);
  if constexpr (VEC == 1)
    if (ns == 8) return rope_dir<T, VEC, 8, INTER, ALIGNED, false>(bwd);
  return nullptr;
}
template <typename T, bool INTER> const void* rope_vec(int vec, int ns, bool aligned, bool full, bool bwd) {
  if (vec == Vec<T>::N) return rope_ns<T, Vec<T>::N, INTER, true>(ns, full, bwd);
  if (Vec<T>::N == 8 && vec == 4) return rope_ns<T, 4, INTER, true>(ns, full, bwd);
  if (vec == 2 && aligned) return rope_ns<T, 2, INTER, true>(ns, full, bwd);
  if (INTER) return vec == 2 ? rope_ns<T, 2, INTER, false>(ns, full, bwd) : nullptr;
  return vec == 1 ? rope_ns<T, 1, false, false>(ns, full, bwd) : nullptr;
}
template <typename T>
const void* rope_table(int vec, int ns, bool inter, bool aligned, bool full, bool bwd) {
  return inter ? rope_vec<T, true>(vec, ns, aligned, full, bwd)
               : rope_vec<T, false>(vec, ns, aligned, full, bwd);
}

}  // namespace nf
