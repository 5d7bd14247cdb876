// 8- and 4-bit formats with scales: layouts, and the device functions that
// turn fp32 values into codes and scales and back.
//
//   format      code   scale              covers        value
//   MX_FP8_ROW   E4M3  fp32               a row         code * scale
//   MX_FP8_BLOCK E4M3  fp32               128 columns   code * scale
//   MX_MXFP8     E4M3  E8M0 (2^(b - 127)) 32 columns    code * scale
//   MX_MXFP4     E2M1  E8M0               32 columns    code * scale
//   MX_NVFP4     E2M1  E4M3               16 columns    code * scale / mul
//
// The last three are the microscaled ones. Their rows of codes are padded with
// zeros to 32 columns (so that a row starts on 16 bytes), and their scales lie
// in tiles of 128 rows by 4 blocks, 512 bytes each: the scale of row r, block
// b of a tile is byte (r % 32) * 16 + (r / 32) * 4 + b. That is how the tensor
// cores take them (32 lanes of 16 bytes), so a tile goes there as it lies.
// Tiles run along a row first; what lies behind the last row or block is 0.
#pragma once

#include <cuda_fp8.h>

#include "../../include/normfuse.h"
#include "common.cuh"

namespace nf {

constexpr unsigned kInfBits = 0x7f800000u;
constexpr float kLeastAmax = 0x1p-100f;   // fp8_row, fp8_block: smaller ones count as this

inline __host__ __device__ bool mx_tiled(int fmt) { return fmt >= MX_MXFP8; }
inline __host__ __device__ bool mx_four(int fmt) { return fmt >= MX_MXFP4; }
// Columns of a block; a row's (MX_FP8_ROW) is given as 0.
inline __host__ __device__ int mx_block(int fmt) {
  return fmt == MX_NVFP4 ? 16 : fmt == MX_FP8_BLOCK ? 128 : fmt == MX_FP8_ROW ? 0 : 32;
}
inline __host__ __device__ int64_t mx_pitch(int fmt, int64_t cols) {   // bytes of a row of codes
  if (!mx_tiled(fmt)) return cols;
  const int64_t padded = (cols + 31) / 32 * 32;
  return mx_four(fmt) ? padded / 2 : padded;
}
inline __host__ __device__ int64_t mx_blocks(int fmt, int64_t cols) {
  const int b = mx_block(fmt);
  return b == 0 ? 1 : (cols + b - 1) / b;
}

// Kernels launched by launch_overlapped() call both of these. Behind the first, what
// was before this kernel on the stream has ended and its writes are visible: every
// thread calls it before it touches memory that another kernel reads or writes, so
// that whoever waits for this grid has waited for that one. After the second, the
// next kernel on the stream may be scheduled.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// The beginning of a kernel without tensor memory. One that takes some does so
// between the two, with a barrier behind it: it holds none while it waits for a
// kernel in front, which might still have to take its own on this SM, and the next
// one cannot take any, and wait with it for this one, before this one has its own.
__device__ __forceinline__ void start_after_stream() {
  let_next_start();
  wait_for_stream();
}

// 16 bytes, or one value, of a tensor that the kernel in front may have written. Such
// a kernel's lifetime begins before that one's writes, so the non-coherent loads
// of the other kernels (ld_vec, __ldg) are not for it: they hold only where memory
// does not change as long as the kernel lives, and the compiler may move them
// ahead of the wait. An ordinary load is coherent and stays behind it.
__device__ __forceinline__ uint4 ld_behind(const void* p) { return *reinterpret_cast<const uint4*>(p); }
template <typename T> __device__ __forceinline__ T ld_one_behind(const T* p) { return *p; }

// A format as a type.
template <int F> struct Format {
  static constexpr int value = F;
  static constexpr bool four = F >= MX_MXFP4;
  static constexpr int width = F == MX_NVFP4 ? 16 : F == MX_FP8_BLOCK ? 128 : 32;
};

// Where a call writes a quantised matrix.
struct QuantOut {
  unsigned char* codes;
  void* scales;          // float, or bytes in tiles
  const float* mul;      // MX_NVFP4: factor of the values before, null = 1
  int64_t rows;
  int64_t cols;
  int64_t pitch;         // bytes of a row of codes
  int64_t blocks;        // of a row
  int fmt;
};

// Offset of a block's scale byte in the tiles: a row's part and a block's.
__host__ __device__ __forceinline__ int64_t scale_row(int64_t row, int64_t blocks) {
  return (row >> 7) * ((blocks + 3) >> 2) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}
__host__ __device__ __forceinline__ int64_t scale_block(int64_t block) { return (block >> 2) * 512 + (block & 3); }
__host__ __device__ __forceinline__ int64_t scale_at(int64_t row, int64_t block, int64_t blocks) {
  return scale_row(row, blocks) + scale_block(block);
}

// A scale and the factor that goes with it: codes are those of v * factor
// (for MX_NVFP4: v / scale, see quotient2). `bits` of a block's largest |v|;
// infinite or NaN makes the scale NaN and the codes 0.
struct BlockScale {
  float factor;          // 0: all codes are 0
  float scale;           // MX_NVFP4: the scale's value; fp32 formats: the scale
  unsigned byte;         // microscaled formats
};

// E8M0: the least power of two 2^e, e >= -127, with amax <= MOST * 2^e, by the
// bits of amax: its exponent less that of MOST (8 or 2), one more where its
// fraction is larger than that of MOST (448 = 1.75 * 2^8, 6 = 1.5 * 2^2). No
// value saturates.
template <bool FOUR>
__device__ __forceinline__ BlockScale scale_e8m0(unsigned bits) {
  constexpr unsigned kRound = FOUR ? 0x3fffffu : 0x1fffffu;
  constexpr int kTop = FOUR ? 2 : 8;
  BlockScale s;
  const int e = max((int)((bits + kRound) >> 23) - kTop, 0);
  const bool odd = bits >= kInfBits;
  s.byte = odd ? 0xffu : (unsigned)e;
  s.factor = odd ? 0.f : __uint_as_float((unsigned)(254 - e) << 23);
  s.scale = 0.f;
  return s;
}

// v / d for a constant d, correctly rounded: see quotient2.
template <int D> __device__ __forceinline__ float over(float v) {
  constexpr float kInv = 1.0f / (float)D;
  const float q = v * kInv;
  return fmaf(fmaf(-q, (float)D, v), kInv, q);
}

// E4M3 scale of a block of MX_NVFP4: amax / 6, rounded to E4M3 (448 at most), and
// 1 / scale, correctly rounded: one Newton step from the approximation, which
// the eight fractions that E4M3 has all reach (the tests see every one).
__device__ __forceinline__ BlockScale scale_e4m3(unsigned bits) {
  BlockScale s;
  const bool odd = bits >= kInfBits;
  const float t = over<6>(__uint_as_float(bits));
  s.byte = odd ? 0x7fu : fp8x2(make_float2(t, 0.f), splat2(1.0f)) & 0xffu;
  s.scale = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s.byte, __NV_E4M3)));
  const float r = __fdividef(1.0f, s.scale);
  s.factor = s.byte && !odd ? fmaf(fmaf(-s.scale, r, 1.0f), r, r) : 0.f;
  return s;
}

// fp32 scale: amax / 448, with amax no less than 2^-100 (so that 448 / amax is
// finite and the scale normal).
__device__ __forceinline__ BlockScale scale_fp32(unsigned bits) {
  const bool odd = bits >= kInfBits;
  const float a = fmaxf(__uint_as_float(odd ? 0u : bits), kLeastAmax);
  return {odd ? 0.f : 448.0f / a, odd ? __uint_as_float(0x7fffffffu) : over<448>(a), 0u};
}

// v / s, correctly rounded, from r = 1 / s rounded to nearest: q = v r is
// within a rounding or two, and the remainder v - q s, exact in one fma, gives
// the correction (Markstein 1990). E2M1 has only eight magnitudes, 16-bit
// values often lie on the middle between two of them, and a quotient that is
// off by a rounding would fall to the wrong side.
__device__ __forceinline__ float2 quotient2(float2 v, float s, float r) {
  const float2 q = mul2(v, splat2(r));
  const float2 rem = fma2(q, splat2(-s), v);
  return fma2(rem, splat2(r), q);
}

// Codes of 2P values. FOUR: 2P / 2 bytes, else 2P bytes, the first value lowest.
template <int P>
__device__ __forceinline__ void codes_e4m3(const float2* v, float factor, unsigned* out) {
  const float2 f = splat2(factor);
#pragma unroll
  for (int i = 0; i < P; i += 2) out[i / 2] = (unsigned)fp8x2(v[i], f) | ((unsigned)fp8x2(v[i + 1], f) << 16);
  if (factor == 0.f) {   // an infinity times 0 is not 0
#pragma unroll
    for (int i = 0; i < P; i += 2) out[i / 2] = 0u;
  }
}
// E2M1 codes of four or eight values, to nearest even, 6 at most.
__device__ __forceinline__ unsigned fp4x4(float2 a, float2 b) {
  unsigned o;
  asm("{\n\t.reg .b8 b0, b1, z;\n\tmov.b16 {z, z}, 0;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "mov.b32 %0, {b0, b1, z, z};\n\t}"
      : "=r"(o)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return o;
}
__device__ __forceinline__ unsigned fp4x8(const float2* v) {
  unsigned o;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(o)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x),
        "f"(v[3].y));
  return o;
}
// The eight values of four bytes of E2M1 codes.
__device__ __forceinline__ void fp4_values(unsigned w, float2* v) {
  unsigned h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f16x2_to_f2(h[i]);
}
// 2P / 2 bytes in the low end of the result (P = 2, 4).
template <int P>
__device__ __forceinline__ unsigned codes_e2m1(const float2* v, const BlockScale& s, bool nvfp4) {
  float2 q[P];
#pragma unroll
  for (int i = 0; i < P; ++i) q[i] = nvfp4 ? quotient2(v[i], s.scale, s.factor) : mul2(v[i], splat2(s.factor));
  unsigned out;
  if constexpr (P == 4) out = fp4x8(q);
  else out = fp4x4(q[0], q[1]);
  return s.factor == 0.f ? 0u : out;
}

// Larger magnitude of two values as a magnitude; NaN wins.
__device__ __forceinline__ float abs_max(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(fabsf(a)), "f"(fabsf(b)));
  return m;
}
// Largest |v| of 2P values as bits (NaN wins: its bits are above those of inf).
template <int P>
__device__ __forceinline__ unsigned amax_of(const float2* v) {
  float m = abs_max(v[0].x, v[0].y);
#pragma unroll
  for (int i = 1; i < P; ++i) m = abs_max(m, abs_max(v[i].x, v[i].y));
  return __float_as_uint(m);
}
// Largest over aligned groups of LANES lanes, by all lanes of the warp.
template <int LANES> __device__ __forceinline__ unsigned lanes_max(unsigned m) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Store VEC codes of the columns from `col` on (col a multiple of VEC).
template <int VEC>
__device__ __forceinline__ void put_codes(unsigned char* p, const unsigned* c, bool four) {
  if (four) {
    if (VEC == 8) *reinterpret_cast<unsigned*>(p) = c[0];
    else *reinterpret_cast<unsigned short*>(p) = (unsigned short)c[0];
  } else {
    if (VEC == 8) *reinterpret_cast<uint2*>(p) = make_uint2(c[0], c[1]);
    else *reinterpret_cast<unsigned*>(p) = c[0];
  }
}

// Scale and codes of a block whose values lie in neighbouring lanes, VEC each (0
// behind the last column). All lanes of the warp call it; a lane's codes go to
// `codes` where it is `live`, the block's scale (fp32 or a byte) to `scale` where
// it is the `first` of its block. `bytes` (MX_FP8_BLOCK): a byte at a time,
// `most` of them.
template <int VEC, int FMT>
__device__ __forceinline__ void put_block(float2* v, float mul, unsigned char* codes, bool live, void* scale,
                                          bool first, int most = VEC, bool bytes = false) {
  constexpr int P = VEC / 2;
  constexpr bool FOUR = FMT >= MX_MXFP4;
  constexpr int kWidth = FMT == MX_NVFP4 ? 16 : FMT == MX_FP8_BLOCK ? 128 : 32;
  if (FMT == MX_NVFP4) {
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = mul2(v[i], splat2(mul));
  }
  const unsigned m = lanes_max<kWidth / VEC>(amax_of<P>(v));
  unsigned c[VEC / 4];
  const BlockScale s = FMT == MX_NVFP4 ? scale_e4m3(m) : FMT == MX_FP8_BLOCK ? scale_fp32(m) : scale_e8m0<FOUR>(m);
  if (FOUR) c[0] = codes_e2m1<P>(v, s, FMT == MX_NVFP4);
  else codes_e4m3<P>(v, s.factor, c);
  if (live) {
    if (FMT != MX_FP8_BLOCK || !bytes) {
      put_codes<VEC>(codes, c, FOUR);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < most) codes[i] = (unsigned char)(c[i / 4] >> (8 * (i % 4)));
    }
  }
  if (first) {
    if (FMT == MX_FP8_BLOCK) *static_cast<float*>(scale) = s.scale;
    else *static_cast<unsigned char*>(scale) = (unsigned char)s.byte;
  }
}

// Where the scales of a row begin, and how far from there a block's is, in bytes.
template <int FMT> __device__ __forceinline__ unsigned char* scales_of_row(const QuantOut& q, int64_t row) {
  return static_cast<unsigned char*>(q.scales) + (FMT == MX_FP8_BLOCK ? row * q.blocks * 4 : scale_row(row, q.blocks));
}
template <int FMT, typename I> __device__ __forceinline__ I scale_step(I block) {
  return FMT == MX_FP8_BLOCK ? block * 4 : (block >> 2) * 512 + (block & 3);
}

// The scale bytes behind a row's last block, and all of a row behind the last
// row, are 0. `t` of `n` threads.
__device__ __forceinline__ void put_padding(const QuantOut& q, int64_t row, int t, int n) {
  const int64_t first = row < q.rows ? q.blocks : 0;
  for (int64_t b = first + t; b < (q.blocks + 3) / 4 * 4; b += n)
    static_cast<unsigned char*>(q.scales)[scale_at(row, b, q.blocks)] = 0;
}

__device__ __forceinline__ float mul_of(const QuantOut& q) {
  return q.fmt == MX_NVFP4 && q.mul != nullptr ? *q.mul : 1.0f;
}

}  // namespace nf
