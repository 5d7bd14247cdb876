// Rotary positions (Su et al., 2021) of attention heads, with the RMSNorm of
// each head before the rotation where a gamma is given:
//   u = x * rstd * w, rstd = 1/sqrt(sum x^2 / D + eps)      (or u = x)
//   y0 = s (u0 cos t - u1 sin t), y1 = s (u1 cos t + u0 sin t)
// for the pairs (j, j + rot/2) or (2j, 2j + 1) of the first `rot` elements;
// the others pass through. The backward applies the transposed rotation to
// dy, then the RMSNorm's: with g' the rotated-back gradient, dgamma sums
// g' * xhat over tokens and heads, g = g' * w,
//   dx = rstd (g - xhat * sum(g * xhat) / D).
// The statistics are taken anew from x, whose head is in registers anyway.
//
// Angles: a position times a frequency passes fp32's precision at a few
// thousand radians. A frequency is turned into a 64-bit fraction of a turn,
// the product with the integer position is taken modulo 2^64, which is
// modulo one turn exactly, and its top 32 bits give sine and cosine. The error
// is that of the frequency itself times the position, plus 2^-33 turns.
//
// Every tensor is read and written once. The forward reaches 0.80 of the copy
// rate; neither DRAM (61 % of its peak) nor the FMA pipe (34 %, its heavy half
// 44 %) is full: norm, rotation, conversions and addresses issue in half of the
// cycles, and 24 warps an SM, which its 80 registers allow, have too few loads
// in flight to cover the rest. Measured, back to back, with norm:
//   forward  1 x 16384 tokens, 32 + 8 heads of 128, bf16   62 us, 5.4 TB/s
//            64 x 1 token                                   3.9 us (latency)
//   backward 4 x 4096 tokens, 16 + 4 heads of 64, bf16      36 us, 3.5 TB/s:
//            two CTAs an SM (120 registers with dgamma's sums)
#pragma once

#include "common.cuh"

namespace nf {

constexpr int kRopeThreads = 256;
// Heads that a thread has on their way. Forward: with one 1 x 16384 tokens take
// 69 us for 62, with three 77. Backward: two do not pay for their registers
// (37.4 us for 36.8 over 4 x 4096 tokens, 22.8 for 21.1 over 2 x 4096 with two
// axes).
constexpr int kRopeAheadFwd = 2, kRopeAheadBwd = 1;
constexpr int kRopeMaxDim = 512;
constexpr int kRopeMaxTable = 2048;   // floats of a tile's cosines, and of its sines
constexpr int kRopeMaxAxes = 4;

// One of the tensors a call takes (queries or keys).
struct RopeSide {
  const void* in;        // x, or dy in the backward
  const void* x;         // backward: the forward's x, when gamma is given
  void* out;             // y, or dx
  const void* gamma;     // nullable: no norm
  int heads;             // 0: absent
  int head_lanes;        // heads that a CTA works on at a time
  int token_lanes;       // tokens, each by head_lanes groups of threads
  int tile;              // tokens of a tile
  int64_t row_tiles;     // tiles of a sequence, ceil(tokens / tile)
  int64_t tiles;         // of all sequences
  int64_t in_s[3], x_s[3], out_s[3];   // strides of batch, token, head (elements)
};

struct RopeArgs {
  RopeSide side[2];
  const void* pos;
  const double* freqs;   // [axes][rot / 2] radians a position
  int64_t pos_s[3];      // strides of axis, batch, token (elements)
  int64_t batch, tokens; // sequences, and the tokens of one
  float* ws;             // backward: [max of blocks][2 * dim] partials, or null
  int blocks[2];         // CTAs of each side, the queries' first
  int pos64, axes;
  int dim, rot;
  int lanes;             // threads of one head, a power of two <= 32
  int row;               // floats of a token's row in the table, a multiple of 4
  int wide;              // threads that work out a token's angles, a power of two
  float scale_c, scale_s;  // of the cosines and the sines; the sines' sign turns it round
  float eps, inv_dim;
  int zero_centered;
};

// VEC elements as they are in memory; ALIGNED: one access of all of them.
template <typename T, int VEC, bool ALIGNED> struct RopeRaw {
  static constexpr int B = VEC * (int)sizeof(T);
  union {
    uint4 q;
    uint2 d;
    unsigned w;
    T t[VEC];
  } u;
  __device__ __forceinline__ RopeRaw() {}
  __device__ __forceinline__ void load(const T* p) {
    if (ALIGNED && B == 16) u.q = *reinterpret_cast<const uint4*>(p);
    else if (ALIGNED && B == 8) u.d = *reinterpret_cast<const uint2*>(p);
    else if (ALIGNED && B == 4) u.w = *reinterpret_cast<const unsigned*>(p);
    else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) u.t[i] = p[i];
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < VEC; ++i) u.t[i] = from_f<T>(0.f);
  }
  // As pairs of fp32 (one element: a pair with an idle second half), and back.
  __device__ __forceinline__ void get(float2* f) const {
    if constexpr (B == 16) {
      unpack2<T>(u.q, f);
    } else if constexpr (VEC == 1) {
      f[0] = make_float2(to_f(u.t[0]), 0.f);
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) f[i] = make_float2(to_f(u.t[2 * i]), to_f(u.t[2 * i + 1]));
    }
  }
  __device__ __forceinline__ void set(const float2* f) {
    if constexpr (B == 16) {
      u.q = pack2<T>(f);
    } else if constexpr (VEC == 1) {
      u.t[0] = from_f<T>(f[0].x);
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        u.t[2 * i] = from_f<T>(f[i].x);
        u.t[2 * i + 1] = from_f<T>(f[i].y);
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if (ALIGNED && B == 16) *reinterpret_cast<uint4*>(p) = u.q;
    else if (ALIGNED && B == 8) *reinterpret_cast<uint2*>(p) = u.d;
    else if (ALIGNED && B == 4) *reinterpret_cast<unsigned*>(p) = u.w;
    else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = u.t[i];
    }
  }
};

// A frequency in radians as a 64-bit fraction of a turn: f * 2^64 / (2 pi)
// modulo 2^64, by integers (double arithmetic is slow on this part). With
// f = m * 2^e, m of 53 bits, and K = 2^130 / (2 pi), rounded to 128 bits, it
// is (m * K) >> (66 - e), bits 64 and up of which fall away. Off by less than
// 2^-64 turns for frequencies up to 2^60.
__device__ __forceinline__ unsigned long long turns_of(double f) {
  const unsigned long long k1 = 0xa2f9836e4e441529ull, k0 = 0xfc2757d1f534ddc1ull;
  const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
  const int ex = (int)(bits >> 52) & 0x7ff;
  if (ex == 0 || ex == 0x7ff) return 0;   // zero, below 2^-1022, or not finite (see finite_turns)
  const unsigned long long m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
  // m * K = (w2, w1, w0)
  const unsigned long long w0 = m * k0, w1 = m * k1 + __umul64hi(m, k0);
  const unsigned long long w2 = __umul64hi(m, k1) + (w1 < m * k1 ? 1 : 0);
  const int sh = 1077 - ex;               // t = (w2, w1, w0) >> (64 + sh)
  unsigned long long t;
  if (sh >= 128) t = 0;
  else if (sh >= 64) t = w2 >> (sh - 64);
  else if (sh > 0) t = (w1 >> sh) | (w2 << (64 - sh));
  else if (sh == 0) t = w1;
  else t = sh > -64 ? (w1 << -sh) | (w0 >> (64 + sh)) : 0;
  return (long long)bits < 0 ? 0ull - t : t;
}

// An infinity or a NaN has no fraction of a turn: its pair's cosines and sines
// are NaN, as the definition gives them for any position.
__device__ __forceinline__ bool finite_turns(double f) {
  return ((unsigned long long)__double_as_longlong(f) >> 52 & 0x7ff) != 0x7ff;
}

// Sine and cosine of t 2^-32 turns: the nearest quarter turn, then the Taylor
// series of the rest, at most pi / 4, to x^9 and x^10 (the next terms are
// below 2^-29 and 2^-31); about 1 ulp in all.
__device__ __forceinline__ void sincos_turns(unsigned t, float* sine, float* cosine) {
  const unsigned q = (t + 0x20000000u) >> 30;
  const float x = (float)(int)(t - (q << 30)) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float z = x * x;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -1.6666667e-1f);
  s = fmaf(x * z, s, x);
  float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  c = fmaf(z, c, -1.3888889e-3f);
  c = fmaf(z, c, 4.1666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  const float a = q & 1 ? c : s, b = q & 1 ? s : c;
  *sine = __uint_as_float(__float_as_uint(a) ^ (q & 2) << 30);
  *cosine = __uint_as_float(__float_as_uint(b) ^ ((q + 1) & 2) << 30);
}

// Which vectors a head's lane slot s holds. The first `rot` elements make
// rot / 2 pairs; HALF: vectors (s, s + rv) of the rotated part, then pairs
// of vectors of what passes through; INTER: vectors s and s + ceil(nv / 2),
// each holding VEC / 2 neighbouring pairs.
struct RopeSlot {
  int a, b;              // first elements of the two vectors
  bool on, on_b;
  unsigned turned;       // bit i: pair i of the slot is rotated
};
// Pair number of a slot's pair i (HALF: that of the vectors' elements i;
// INTER: VEC / 2 pairs of the first vector, then those of the second).
template <int VEC, bool INTER> __device__ __forceinline__ int rope_pair(const RopeSlot& r, int i) {
  if (!INTER) return r.a + i;
  return i < VEC / 2 ? r.a / 2 + i : r.b / 2 + i - VEC / 2;
}
// FULL: every slot is there and all of it is rotated.
template <int VEC, bool INTER, bool FULL>
__device__ __forceinline__ RopeSlot rope_slot(int s, int dim, int rot) {
  RopeSlot r;
  const int nv = dim / VEC;
  if (FULL) {
    r.on = r.on_b = true;
    r.turned = (1u << VEC) - 1;
    r.a = s * VEC;
    r.b = r.a + dim / 2;
    return r;
  }
  if (INTER) {
    const int n2 = (nv + 1) / 2;
    r.on = s < n2;
    r.on_b = r.on && s + n2 < nv;
    r.a = s * VEC;
    r.b = (s + n2) * VEC;
    r.turned = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (r.on && rope_pair<VEC, true>(r, i) < rot / 2) r.turned |= 1u << i;
  } else {
    const int rv = rot / 2 / VEC;
    if (s < rv) {
      r.on = r.on_b = true;
      r.turned = (1u << VEC) - 1;
      r.a = s * VEC;
      r.b = (s + rv) * VEC;
    } else {
      const int np = nv - 2 * rv, n2 = (np + 1) / 2, p = s - rv;
      r.on = p < n2;
      r.on_b = r.on && p + n2 < np;
      r.turned = 0;
      r.a = (2 * rv + p) * VEC;
      r.b = (2 * rv + p + n2) * VEC;
    }
  }
  return r;
}

// Rotate a slot's pairs in place by (cos, sin); INV: the transposed
// rotation. v: the slot's two vectors as pairs of neighbours. Pairs that pass
// through are not touched (an infinity times a sine of 0 would be a NaN in
// its neighbour).
template <int VEC, bool INTER, bool INV, int NP>
__device__ __forceinline__ void rope_rotate(float2 (&v)[2][NP], const float2 (&cs)[NP],
                                            const float2 (&sn)[NP], unsigned turned) {
  if (INTER) {
    // cs, sn: of the first vector's pairs, then of the second's
    constexpr int H = VEC > 1 ? VEC / 2 : 1;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float2& p = v[i / H][i % H];
      const float c = i % 2 ? cs[i / 2].y : cs[i / 2].x;
      const float t = i % 2 ? sn[i / 2].y : sn[i / 2].x, s = INV ? -t : t;
      const float2 r = make_float2(p.x * c - p.y * s, p.y * c + p.x * s);
      if (turned >> i & 1) p = r;
    }
  } else if (turned) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float2 a = v[0][i], b = v[1][i];
      const float2 as = mul2(a, sn[i]), bs = mul2(b, sn[i]);
      const float2 ac = mul2(a, cs[i]), bc = mul2(b, cs[i]);
      v[0][i] = INV ? add2(ac, bs) : fma2(bs, splat2(-1.f), ac);
      v[1][i] = INV ? fma2(as, splat2(-1.f), bc) : add2(bc, as);
    }
  }
}

// Sum over aligned groups of `lanes` lanes; the same branches in every lane.
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// N consecutive floats of the table, from pair `at` of f on.
template <int N, int NP>
__device__ __forceinline__ void rope_table_get(const float* t, float2 (&f)[NP], int at) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 v = reinterpret_cast<const float4*>(t)[i];
      f[at + 2 * i] = make_float2(v.x, v.y);
      f[at + 2 * i + 1] = make_float2(v.z, v.w);
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) f[at + i] = reinterpret_cast<const float2*>(t)[i];
  } else {
    f[at] = make_float2(t[0], 0.f);
  }
}

// A CTA takes the queries or the keys of a tile of one sequence's tokens. It
// works out the cosines and sines of those tokens once, into shared memory.
// A group of `lanes` threads has a head and goes through the tile's tokens
// with it, so that it steps its pointers and does little else; the next rows
// of a group are always on their way. A CTA takes tile after tile; in the
// backward it keeps its share of dgamma in registers. FULL: each lane has a
// whole slot and all of the head is rotated.
template <typename T, int VEC, int NS, bool INTER, bool ALIGNED, bool FULL, bool BWD>
__global__ void __launch_bounds__(kRopeThreads, BWD ? 2 : 3) rope_kernel(RopeArgs A) {
  using Raw = RopeRaw<T, VEC, ALIGNED>;
  constexpr int kAhead = BWD ? kRopeAheadBwd : kRopeAheadFwd;
  // Cosines and sines, of two tiles in turn: a warp may write the next tile's
  // while others still read, so a tile takes one barrier.
  __shared__ __align__(16) float tab[2][2][kRopeMaxTable];
  __shared__ unsigned long long tab_t[kRopeMaxAxes * kRopeMaxDim / 2];   // several axes only
  const int L = A.lanes, per_cta = kRopeThreads / L;
  const int l = threadIdx.x & (L - 1), grp = threadIdx.x / L;
  const int side = (int)blockIdx.x >= A.blocks[0] ? 1 : 0;
  const int blk = blockIdx.x - (side ? A.blocks[0] : 0), blks = A.blocks[side];
  const RopeSide &q0 = A.side[0], &k0 = A.side[1];
  // Taken once: a side indexed at run time would be read anew at every use.
#define NF_SIDE(field) (side ? k0.field : q0.field)
  const bool norm = NF_SIDE(gamma) != nullptr;
  const T* const in = static_cast<const T*>(NF_SIDE(in));
  const T* const xin = static_cast<const T*>(NF_SIDE(x));
  T* const out = static_cast<T*>(NF_SIDE(out));
  const int heads = NF_SIDE(heads), head_lanes = NF_SIDE(head_lanes);
  const int token_lanes = NF_SIDE(token_lanes), tile_rows = NF_SIDE(tile);
  const int64_t row_tiles = NF_SIDE(row_tiles), tiles = NF_SIDE(tiles);
  const int64_t in_b = NF_SIDE(in_s[0]), in_t = NF_SIDE(in_s[1]), in_h = NF_SIDE(in_s[2]);
  const int64_t out_b = NF_SIDE(out_s[0]), out_t = NF_SIDE(out_s[1]), out_h = NF_SIDE(out_s[2]);
  const int64_t x_b = BWD ? NF_SIDE(x_s[0]) : 0, x_t = BWD ? NF_SIDE(x_s[1]) : 0,
                x_h = BWD ? NF_SIDE(x_s[2]) : 0;
  const T* const gm = static_cast<const T*>(NF_SIDE(gamma));
#undef NF_SIDE
  const int tl = grp / head_lanes, hl = grp - tl * head_lanes;
  RopeSlot slot[NS];
#pragma unroll
  for (int n = 0; n < NS; ++n) slot[n] = rope_slot<VEC, INTER, FULL>(l + n * L, A.dim, A.rot);
  constexpr int NP = (VEC + 1) / 2;
  RopeRaw<T, VEC, false> gamma[NS][2];   // as it is in memory, to save registers
  float2 acc[BWD ? NS : 1][2][NP];
  const float2 add = splat2(A.zero_centered ? 1.f : 0.f);
#pragma unroll
  for (int n = 0; n < NS; ++n)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      gamma[n][k].clear();
      if (norm && (k == 0 ? slot[n].on : slot[n].on_b))
        gamma[n][k].load(gm + (k == 0 ? slot[n].a : slot[n].b));
      if (BWD) {
#pragma unroll
        for (int i = 0; i < NP; ++i) acc[n][k][i] = splat2(0.f);
      }
    }
  const int j = threadIdx.x & (A.wide - 1);      // this thread's pair
  unsigned long long turns = 0;
  bool finite = true;                            // all of its frequencies are
  if (A.axes == 1) {
    if (j < A.rot / 2) {
      const double f = A.freqs[j];
      turns = turns_of(f);
      finite = finite_turns(f);
    }
  } else {
#pragma unroll
    for (int ax = 0; ax < kRopeMaxAxes; ++ax)
      if (j < A.rot / 2 && ax < A.axes) finite &= finite_turns(A.freqs[ax * (A.rot / 2) + j]);
    for (int i = threadIdx.x; i < A.axes * (A.rot / 2); i += kRopeThreads)
      tab_t[i] = turns_of(A.freqs[i]);
    __syncthreads();
  }

  const int64_t in_step = token_lanes * in_t, out_step = token_lanes * out_t,
                x_step = token_lanes * x_t;
  int turn = 0;
  for (int64_t tile = blk; tile < tiles; tile += blks, turn ^= 1) {
    float* const tab_c = tab[turn][0];
    float* const tab_s = tab[turn][1];
    const int64_t b = tile / row_tiles, tok0 = (tile - b * row_tiles) * tile_rows;
    const int toks = (int)min((int64_t)tile_rows, A.tokens - tok0);
    // Whole warps run the loops below, so that every lane reaches the shuffles.
    const int steps = (toks + token_lanes - 1) / token_lanes;
    const int mine = tl < token_lanes && toks > tl ? (toks - tl - 1) / token_lanes + 1 : 0;
    for (int h0 = 0; h0 < heads; h0 += head_lanes) {
      const int h = h0 + hl, n_rows = h < heads ? mine : 0;
      const T* p = in + b * in_b + (tok0 + tl) * in_t + h * in_h;
      const T* q = BWD ? xin + b * x_b + (tok0 + tl) * x_t + h * x_h : nullptr;
      T* dst = out + b * out_b + (tok0 + tl) * out_t + h * out_h;
      Raw v0[kAhead][NS][2], x0[BWD ? kAhead : 1][NS][2];
      const auto fetch = [&](int d, int r) {   // row r of the group
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          if (r < n_rows && slot[n].on) {
            v0[d][n][0].load(p + slot[n].a);
            if (slot[n].on_b) v0[d][n][1].load(p + slot[n].b);
            if (BWD && norm) {
              x0[d][n][0].load(q + slot[n].a);
              if (slot[n].on_b) x0[d][n][1].load(q + slot[n].b);
            }
          }
        }
        p += in_step;
        if (BWD) q += x_step;
      };
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            v0[d][n][k].clear();
            if (BWD) x0[d][n][k].clear();
          }
        fetch(d, d);
      }
      if (h0 == 0) {
        // The angles, while the first rows are on their way; positions are
        // loaded four at a time.
        if (j < A.rot / 2) {
          const int step = kRopeThreads / A.wide;
          for (int t0 = threadIdx.x / A.wide; t0 < toks; t0 += 4 * step) {
            unsigned long long sum[4] = {0, 0, 0, 0};
            for (int ax = 0; ax < A.axes; ++ax) {
              const int64_t at = ax * A.pos_s[0] + b * A.pos_s[1] + (tok0 + t0) * A.pos_s[2];
              long long pos[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                pos[i] = 0;
                const int64_t from = at + i * step * A.pos_s[2];
                if (t0 + i * step < toks)
                  pos[i] = A.pos64 ? static_cast<const long long*>(A.pos)[from]
                                   : (long long)static_cast<const int*>(A.pos)[from];
              }
              if (A.axes > 1) turns = tab_t[ax * (A.rot / 2) + j];
#pragma unroll
              for (int i = 0; i < 4; ++i) sum[i] += (unsigned long long)pos[i] * turns;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int t = t0 + i * step;
              if (t < toks) {
                const float kNaN = __int_as_float(0x7fffffff);
                float s, c;
                sincos_turns((unsigned)((sum[i] + 0x80000000ull) >> 32), &s, &c);
                tab_c[t * A.row + j] = finite ? c * A.scale_c : kNaN;
                tab_s[t * A.row + j] = finite ? s * A.scale_s : kNaN;
              }
            }
          }
        }
        __syncthreads();
      }
      const float* tc = tab_c + tl * A.row;
      const float* ts = tab_s + tl * A.row;
      for (int st = 0; st < steps; st += kAhead) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
          const bool act = st + d < n_rows;
          float2 v[NS][2][NP], cs[NS][NP], sn[NS][NP], sum = splat2(0.f);
#pragma unroll
          for (int n = 0; n < NS; ++n) {
            v0[d][n][0].get(v[n][0]);
            v0[d][n][1].get(v[n][1]);
            if constexpr (INTER) {
              constexpr int H = VEC / 2;
              const int sb = slot[n].on_b ? slot[n].b / 2 : 0;
              if constexpr (H == 1) {
                cs[n][0] = make_float2(tc[slot[n].a / 2], tc[sb]);
                sn[n][0] = make_float2(ts[slot[n].a / 2], ts[sb]);
              } else {
                rope_table_get<H>(tc + slot[n].a / 2, cs[n], 0);
                rope_table_get<H>(ts + slot[n].a / 2, sn[n], 0);
                rope_table_get<H>(tc + sb, cs[n], H / 2);
                rope_table_get<H>(ts + sb, sn[n], H / 2);
              }
            } else {
              const int at = slot[n].turned ? slot[n].a : 0;
              rope_table_get<VEC>(tc + at, cs[n], 0);
              rope_table_get<VEC>(ts + at, sn[n], 0);
            }
          }
          if (!BWD) {
            fetch(d, st + d + kAhead);
            if (norm) {
#pragma unroll
              for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                  for (int i = 0; i < NP; ++i) sum = fma2(v[n][k][i], v[n][k][i], sum);
              const float ss = lanes_sum(sum.x + sum.y, L);
              const float2 rstd = splat2(rsqrtf(fmaf(ss, A.inv_dim, A.eps)));
#pragma unroll
              for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  float2 w[NP];
                  gamma[n][k].get(w);
#pragma unroll
                  for (int i = 0; i < NP; ++i)
                    v[n][k][i] = mul2(mul2(v[n][k][i], rstd), add2(w[i], add));
                }
            }
#pragma unroll
            for (int n = 0; n < NS; ++n)
              rope_rotate<VEC, INTER, false>(v[n], cs[n], sn[n], slot[n].turned);
          } else {
            float2 xv[NS][2][NP];
#pragma unroll
            for (int n = 0; n < NS; ++n) {
              x0[d][n][0].get(xv[n][0]);
              x0[d][n][1].get(xv[n][1]);
            }
            fetch(d, st + d + kAhead);
#pragma unroll
            for (int n = 0; n < NS; ++n)
              rope_rotate<VEC, INTER, true>(v[n], cs[n], sn[n], slot[n].turned);
            if (norm) {
              float2 dot = splat2(0.f), vx[NS][2][NP];   // g' x, then v = g
#pragma unroll
              for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  float2 w[NP];
                  gamma[n][k].get(w);
#pragma unroll
                  for (int i = 0; i < NP; ++i) {
                    w[i] = add2(w[i], add);
                    sum = fma2(xv[n][k][i], xv[n][k][i], sum);
                    vx[n][k][i] = mul2(v[n][k][i], xv[n][k][i]);
                    dot = fma2(vx[n][k][i], w[i], dot);
                    v[n][k][i] = mul2(v[n][k][i], w[i]);
                  }
                }
              // sum g xhat = rstd sum g x, so one round of shuffles serves both
              const float ss = lanes_sum(sum.x + sum.y, L), gs = lanes_sum(dot.x + dot.y, L);
              const float rstd = rsqrtf(fmaf(ss, A.inv_dim, A.eps));
              const float2 rs = splat2(rstd), mean = splat2(-gs * rstd * A.inv_dim);
#pragma unroll
              for (int n = 0; n < NS; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                  for (int i = 0; i < NP; ++i) {
                    if (act) acc[n][k][i] = fma2(vx[n][k][i], rs, acc[n][k][i]);
                    v[n][k][i] = mul2(rs, fma2(mul2(xv[n][k][i], rs), mean, v[n][k][i]));
                  }
            }
          }
          if (act) {
#pragma unroll
            for (int n = 0; n < NS; ++n) {
              Raw r;
              if (slot[n].on) {
                r.set(v[n][0]);
                r.store(dst + slot[n].a);
              }
              if (slot[n].on_b) {
                r.set(v[n][1]);
                r.store(dst + slot[n].b);
              }
            }
          }
          dst += out_step;
          if (st + d + 1 < n_rows) {   // stay inside the table behind the last row
            tc += token_lanes * A.row;
            ts += token_lanes * A.row;
          }
        }
      }
    }
  }
  if (BWD && A.ws != nullptr) {
    // The groups' sums, added in their order, into this CTA's partial row, by
    // way of the tables' memory (a group's head each: 4096 floats at most). The
    // side with fewer CTAs has its other rows zeroed by the other side.
    float* const red = tab[0][0];
    // The finalize may be scheduled while the last CTAs work; it waits for them.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();   // the tables give way
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float2 p = acc[n][0][i / 2], q = acc[n][1][i / 2];
        if (slot[n].on) red[grp * A.dim + slot[n].a + i] = i % 2 ? p.y : p.x;
        if (slot[n].on_b) red[grp * A.dim + slot[n].b + i] = i % 2 ? q.y : q.x;
      }
    __syncthreads();
    float* row = A.ws + (int64_t)blk * 2 * A.dim;
    for (int d = threadIdx.x; d < A.dim; d += kRopeThreads) {
      float t = 0.f;
#pragma unroll 4
      for (int g = 0; g < per_cta; ++g) t += red[g * A.dim + d];
      row[side * A.dim + d] = t;
      if (blk >= A.blocks[1 - side]) row[(1 - side) * A.dim + d] = 0.f;
    }
  }
}

}  // namespace nf
