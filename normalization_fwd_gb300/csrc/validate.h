// Host-side argument checks shared by the C entry points.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/normfuse.h"
#include "common.cuh"

namespace nf {

inline size_t elem_size(ln_dtype dt) { return dt == LN_F32 ? 4 : 2; }

inline bool known_dtype(ln_dtype dt) { return dt == LN_F32 || dt == LN_BF16 || dt == LN_F16; }

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Byte ranges for the overlap check.
struct Range {
  const void* p;
  size_t bytes;
};
inline bool overlap(const Range& a, const Range& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = (uintptr_t)a.p, a1 = a0 + a.bytes;
  const uintptr_t b0 = (uintptr_t)b.p, b1 = b0 + b.bytes;
  return a0 < b1 && b0 < a1;
}
inline bool any_overlap(const Range* outs, int n_out, const Range* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(outs[i], ins[j])) return true;
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

// A strided tensor: up to three outer dimensions around runs of `width`
// bytes. Strides in bytes, >= 0.
struct Strided {
  const void* p = nullptr;
  int64_t n[3] = {1, 1, 1};
  int64_t stride[3] = {0, 0, 0};
  int64_t width = 0;
  bool empty() const {
    return p == nullptr || width == 0 || n[0] == 0 || n[1] == 0 || n[2] == 0;
  }
  // Bytes from the first to past the last one.
  int64_t span() const {
    int64_t s = width;
    for (int i = 0; i < 3; ++i) s += (n[i] - 1) * stride[i];
    return s;
  }
  Range range() const { return {p, empty() ? 0 : (size_t)span()}; }
};

// Whether two runs of a tensor share a byte (a stride of 0, or one shorter
// than what it steps over): an output must not.
inline bool self_overlaps(const Strided& a) {
  if (a.empty()) return false;
  int64_t n[3], st[3];
  int d = 0;
  for (int i = 0; i < 3; ++i)
    if (a.n[i] > 1) {
      n[d] = a.n[i];
      st[d++] = a.stride[i];
    }
  for (int i = 0; i < d; ++i)
    for (int j = i + 1; j < d; ++j)
      if (st[j] < st[i]) {
        const int64_t t = st[i], m = n[i];
        st[i] = st[j];
        n[i] = n[j];
        st[j] = t;
        n[j] = m;
      }
  int64_t span = a.width;
  for (int i = 0; i < d; ++i) {
    if (st[i] < span) return true;
    span += (n[i] - 1) * st[i];
  }
  return false;
}

// The bytes of `a` taken modulo `period` as one interval: its length, or -1
// when it is longer than the period. Dimensions whose stride is a multiple
// of the period fall away.
inline int64_t residue_span(const Strided& a, int64_t period) {
  int64_t s = a.width;
  for (int i = 0; i < 3; ++i)
    if (a.n[i] > 1 && a.stride[i] % period != 0) s += (a.n[i] - 1) * a.stride[i];
  return s <= period ? s : -1;
}

// Whether two tensors may share a byte. Exact for disjoint address ranges
// and for slices that repeat with a common period (the queries and keys of
// one packed projection, channel slices of one activation); anything it
// cannot prove disjoint counts as shared.
inline bool may_overlap(const Strided& a, const Strided& b) {
  if (a.empty() || b.empty()) return false;
  if (!overlap(a.range(), b.range())) return false;
  for (int i = 0; i < 3; ++i) {
    const int64_t period = a.stride[i];
    if (a.n[i] <= 1 || period <= 0) continue;
    const int64_t sa = residue_span(a, period), sb = residue_span(b, period);
    if (sa < 0 || sb < 0) continue;
    // b's interval starts `delta` bytes after a's, on a circle of `period` bytes
    const int64_t pa = (int64_t)((uintptr_t)a.p % (uintptr_t)period);
    const int64_t pb = (int64_t)((uintptr_t)b.p % (uintptr_t)period);
    const int64_t delta = (pb - pa + period) % period;
    if (delta >= sa && delta + sb <= period) return false;
  }
  return true;
}

template <typename F>
cudaError_t by_dtype(ln_dtype dt, F&& f) {
  switch (dt) {
    case LN_F32: return f(float{});
    case LN_BF16: return f(bf16{});
    default: return f(f16{});
  }
}

}  // namespace nf
