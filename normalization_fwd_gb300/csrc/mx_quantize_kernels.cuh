// A matrix, or its transpose, in 8 or 4 bits with scales (mx_formats.cuh), and
// back to values.
//
// Bound by HBM: each value read once, 0.5 to 1 bytes of code written for it.
// 8192 x 8192 bf16 transposed to mxfp8 41 us (4.9 TB/s); 1280 x 8192 fp32 to nvfp4
// 11 us and back to bf16 10 us, of which 2 are the launch.
// The transpose goes through a tile in shared memory: 128 bytes of 256 rows of
// x, read along x's rows and written along the result's.
#pragma once

#include "common.cuh"
#include "mx_formats.cuh"
#include "tcgen05.cuh"

namespace nf {

struct QuantArgs {
  const void* x;
  int64_t x_row;         // elements from one row of x to the next
  QuantOut q;            // rows, cols: of the result
  int vec;               // x can be read 16 bytes at a time
  int vec_codes;         // codes can be written 16 bytes at a time (rows: where the pitch allows)
  int64_t padded_rows;
};

constexpr int kQuantThreads = 256;

// Eight neighbouring values of a row as fp32, 0 from column `n` on.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int64_t col, int64_t n, bool vec, float2* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = splat2(0.f);
  if (vec && col + 8 <= n) {
#pragma unroll
    for (int i = 0; i < 8 / Vec<T>::N; ++i)
      unpack2<T>(ld_behind(row + col + i * Vec<T>::N), v + i * Vec<T>::N / 2);
  } else {
    float* f = reinterpret_cast<float*>(v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < n) f[i] = to_f(row[col + i]);
  }
}

// Rows are dealt to lanes: 2^shift lanes a row, 8 columns each, so that narrow
// matrices leave few of a warp idle; the grid's x covers columns, y rows, which
// go on a grid apart.
struct LaneRows {
  int64_t row, step, col;
  __device__ __forceinline__ LaneRows(int shift) {
    const int per = 5 - shift, lane = threadIdx.x & 31;      // rows of a warp, as a power of two
    row = (((int64_t)blockIdx.y * (kQuantThreads / 32) + (threadIdx.x >> 5)) << per) + (lane >> shift);
    step = ((int64_t)gridDim.y * (kQuantThreads / 32)) << per;
    col = (int64_t)blockIdx.x * 256 + (lane & ((1 << shift) - 1)) * 8;
  }
};

// Rows that start anywhere: a warp's 256 values, lane after lane from one element
// to the next, through shared memory to or from the 8 of each lane (8 elements a
// lane, each of them 16 bytes from the next lane's, take 16 sectors an access).
// f(row, col, place) for each of a lane's eight elements in that order.
template <typename F>
__device__ __forceinline__ void each_element(int64_t row, int64_t col, int shift, F f) {
  const int lane = threadIdx.x & 31;
  const int64_t row0 = row - (lane >> shift), col0 = col - (lane & ((1 << shift) - 1)) * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = i * 32 + lane;
    f(row0 + (e >> (shift + 3)), col0 + (e & ((8 << shift) - 1)), e);
  }
}

// Blocks of 16, 32 or 128 columns. A warp's rows end together (the loop's test is
// by all of them), as its lanes work on blocks together. Two rows at a time, so
// that one is on its way while the other is worked on.
template <typename T, int FMT, bool RAGGED>
__global__ void __launch_bounds__(kQuantThreads) quant_block_kernel(const QuantArgs a, int shift) {
  start_after_stream();
  using F = Format<FMT>;
  __shared__ __align__(16) T buffer[RAGGED ? kQuantThreads / 32 : 1][RAGGED ? 256 : 8];
  T* buf = buffer[RAGGED ? threadIdx.x >> 5 : 0];
  const QuantOut& q = a.q;
  const float mul = FMT == MX_NVFP4 ? mul_of(q) : 1.0f;
  const LaneRows at(shift);
  const int64_t col = at.col, wide = q.pitch * (F::four ? 2 : 1);
  const bool room = col < wide, first = col % F::width == 0 && col < q.cols;
  const bool pads = FMT != MX_FP8_BLOCK && blockIdx.x == 0;
  const bool bytes = FMT == MX_FP8_BLOCK && (q.pitch % 8 != 0 || !a.vec_codes);
  const int most = (int)min((int64_t)8, q.cols - col);
  const bool vec = col + 8 <= q.cols;
  const int64_t step = scale_step<FMT>(col / F::width);
  const int64_t x_step = at.step * a.x_row, code_step = at.step * q.pitch;
  int64_t row = at.row;
  const T* x = static_cast<const T*>(a.x) + row * a.x_row + col;
  unsigned char* codes = q.codes + row * q.pitch + (F::four ? col / 2 : col);
  const auto load = [&](int64_t r, const T* p, float2* v) {
    if constexpr (RAGGED) {
      __syncwarp();
      each_element(r, col, shift, [&](int64_t er, int64_t ec, int e) {
        buf[e] = er < q.rows && ec < q.cols ? static_cast<const T*>(a.x)[er * a.x_row + ec] : from_f<T>(0.f);
      });
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8 / Vec<T>::N; ++i)
        unpack2<T>(reinterpret_cast<const uint4*>(buf + (threadIdx.x & 31) * 8)[i], v + i * Vec<T>::N / 2);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = splat2(0.f);
      if (r >= q.rows) return;
      if (vec) {
#pragma unroll
        for (int i = 0; i < 8 / Vec<T>::N; ++i) unpack2<T>(ld_behind(p + i * Vec<T>::N), v + i * Vec<T>::N / 2);
      } else {
        float* f = reinterpret_cast<float*>(v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < most) f[i] = to_f(p[i]);
      }
    }
  };
  const auto put = [&](int64_t r, unsigned char* c, float2* v) {
    const bool ok = r < q.rows;
    put_block<8, FMT>(v, mul, c, ok && room, scales_of_row<FMT>(q, r) + step, ok && first, most, bytes);
    if (pads && r < a.padded_rows) put_padding(q, r, (threadIdx.x & 31) & ((1 << shift) - 1), 1 << shift);
  };
  for (; __any_sync(0xffffffffu, row < a.padded_rows); row += 2 * at.step) {
    float2 v[4], w[4];
    load(row, x, v);
    load(row + at.step, x + x_step, w);
    put(row, codes, v);
    if (__any_sync(0xffffffffu, row + at.step < a.padded_rows)) put(row + at.step, codes + code_step, w);
    x += 2 * x_step;
    codes += 2 * code_step;
  }
}

// A scale a row: a CTA a row. The first 8192 columns stay in registers, those
// behind them are read again (out of the caches).
constexpr int kRowKept = 4;
template <typename T>
__global__ void __launch_bounds__(kQuantThreads) quant_row_kernel(const QuantArgs a) {
  start_after_stream();
  __shared__ unsigned red[2][kQuantThreads / 32];
  const QuantOut& q = a.q;
  const bool vec_codes = q.pitch % 8 == 0 && a.vec_codes;
  int parity = 0;
  for (int64_t row = blockIdx.x; row < q.rows; row += gridDim.x, parity ^= 1) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_row;
    unsigned m = 0;
    float2 v[kRowKept][4];
#pragma unroll
    for (int k = 0; k < kRowKept; ++k) {
      load8<T>(x, (k * kQuantThreads + (int)threadIdx.x) * 8, q.cols, a.vec != 0, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kRowKept; ++k) m = max(m, amax_of<4>(v[k]));
    for (int64_t col = ((int64_t)kRowKept * kQuantThreads + threadIdx.x) * 8; col < q.cols; col += kQuantThreads * 8) {
      float2 w[4];
      load8<T>(x, col, q.cols, a.vec != 0, w);
      m = max(m, amax_of<4>(w));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) red[parity][threadIdx.x >> 5] = m;
    __syncthreads();
    for (int i = 0; i < kQuantThreads / 32; ++i) m = max(m, red[parity][i]);
    const BlockScale s = scale_fp32(m);
    if (threadIdx.x == 0) static_cast<float*>(q.scales)[row] = s.scale;
    unsigned char* codes = q.codes + row * q.pitch;
    const auto put = [&](int64_t col, const float2* w) {
      unsigned c[2];
      if (col >= q.cols) return;
      codes_e4m3<4>(w, s.factor, c);
      if (vec_codes && col + 8 <= q.cols) {
        put_codes<8>(codes + col, c, false);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < q.cols) codes[col + i] = (unsigned char)(c[i / 4] >> (8 * (i % 4)));
      }
    };
#pragma unroll
    for (int k = 0; k < kRowKept; ++k) put((k * kQuantThreads + (int)threadIdx.x) * 8, v[k]);
    for (int64_t col = ((int64_t)kRowKept * kQuantThreads + threadIdx.x) * 8; col < q.cols; col += kQuantThreads * 8) {
      float2 w[4];
      load8<T>(x, col, q.cols, a.vec != 0, w);
      put(col, w);
    }
  }
}

// The transpose. A tile is 32 words (32 fp32 or 64 16-bit columns of x: rows of
// the result) by 256 rows of x; a lane has a word's one or two rows, a warp 32 of
// the result's columns. With a scale a row a CTA goes over all tiles of its rows
// twice.
constexpr int kTrCols = 256;
constexpr int kTrPitch = 33;
template <typename T> struct TrRows { static constexpr int N = 32 * 4 / sizeof(T); };

template <typename T>
__device__ __forceinline__ void load_tile(const QuantArgs& a, int64_t row0, int64_t col0, unsigned* tile) {
  constexpr int V = Vec<T>::N;                  // of 16 bytes, 8 of them a row of the tile
  const int64_t rows = a.q.rows, cols = a.q.cols;
  uint4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = i * kQuantThreads + threadIdx.x, c = at >> 3, r = (at & 7) * V;
    const T* x = static_cast<const T*>(a.x) + (col0 + c) * a.x_row + row0 + r;
    w[i] = make_uint4(0, 0, 0, 0);
    if (col0 + c < cols) {
      if (a.vec && row0 + r + V <= rows) {
        w[i] = ld_behind(x);
      } else {
        T t[V];
#pragma unroll
        for (int j = 0; j < V; ++j) t[j] = row0 + r + j < rows ? x[j] : from_f<T>(0.f);
        w[i] = *reinterpret_cast<const uint4*>(t);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = i * kQuantThreads + threadIdx.x;
    unsigned* p = tile + (at >> 3) * kTrPitch + (at & 7) * 4;
    p[0] = w[i].x;
    p[1] = w[i].y;
    p[2] = w[i].z;
    p[3] = w[i].w;
  }
}

// Value h (0, or 1 of 16-bit types) of a word.
template <typename T> __device__ __forceinline__ float word_value(unsigned w, int h);
template <> __device__ __forceinline__ float word_value<float>(unsigned w, int) { return __uint_as_float(w); }
template <> __device__ __forceinline__ float word_value<bf16>(unsigned w, int h) {
  return __uint_as_float(h ? w & 0xffff0000u : w << 16);
}
template <> __device__ __forceinline__ float word_value<f16>(unsigned w, int h) {
  return __half2float(__ushort_as_half((unsigned short)(h ? w >> 16 : w & 0xffffu)));
}

// Largest |value| of n words, of each of a word's rows, as fp32 bits. 16-bit
// values are compared as they lie, two at a time.
template <typename T, int N> __device__ __forceinline__ void words_amax(const unsigned* w, unsigned* m) {
  if (sizeof(T) == 4) {
    m[0] = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m[0] = max(m[0], w[i] & 0x7fffffffu);
  } else {
    unsigned b = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) b = __vmaxu2(b, w[i] & 0x7fff7fffu);
    m[0] = __float_as_uint(word_value<T>(b, 0));
    m[sizeof(T) == 2] = __float_as_uint(word_value<T>(b, 1));
  }
}

// Codes and scales of a lane's rows row .. row + W - 1 of the result, columns col
// .. col + 31, out of 32 words. `s`: the rows' scales where they are known (fp32
// scales); `writes`: whether this warp has a block's first columns.
template <typename T, int FMT>
__device__ __forceinline__ void put_columns(const QuantOut& q, int64_t row, int64_t col, const unsigned* w,
                                            float mul, BlockScale* s, bool writes, bool vec_codes) {
  constexpr int W = 4 / sizeof(T);
  constexpr bool FOUR = FMT >= MX_MXFP4, TILED = FMT >= MX_MXFP8;
  unsigned m[W], m2[W];
  if (FMT == MX_NVFP4) {
    words_amax<T, 16>(w, m);
    words_amax<T, 16>(w + 16, m2);
  } else if (TILED) {
    words_amax<T, 32>(w, m);
  }
#pragma unroll
  for (int h = 0; h < W; ++h) {
    if (row + h >= q.rows) break;
    unsigned char* scales = static_cast<unsigned char*>(q.scales);
    if (FOUR) {
      unsigned c[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        BlockScale b;
        if (FMT == MX_NVFP4) {
          // the largest product is that of the largest value: products round monotonically
          b = scale_e4m3(__float_as_uint(fabsf(__uint_as_float(k ? m2[h] : m[h]) * mul)));
          if (col / 16 + k < q.blocks) scales[scale_at(row + h, col / 16 + k, q.blocks)] = (unsigned char)b.byte;
        } else {
          b = scale_e8m0<true>(m[h]);
          if (k == 0) scales[scale_at(row + h, col / 32, q.blocks)] = (unsigned char)b.byte;
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float2 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = 16 * k + 8 * g + 2 * i;
            v[i] = make_float2(word_value<T>(w[at], h), word_value<T>(w[at + 1], h));
            if (FMT == MX_NVFP4) v[i] = mul2(v[i], splat2(mul));
          }
          c[2 * k + g] = codes_e2m1<4>(v, b, FMT == MX_NVFP4);
        }
      }
      *reinterpret_cast<uint4*>(q.codes + (row + h) * q.pitch + col / 2) = make_uint4(c[0], c[1], c[2], c[3]);
    } else {
      if (FMT == MX_MXFP8) {
        s[h] = scale_e8m0<false>(m[h]);
        scales[scale_at(row + h, col / 32, q.blocks)] = (unsigned char)s[h].byte;
      } else if (FMT == MX_FP8_BLOCK && writes) {
        static_cast<float*>(q.scales)[(row + h) * q.blocks + col / 128] = s[h].scale;
      }
      unsigned c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 v[2] = {make_float2(word_value<T>(w[4 * i], h), word_value<T>(w[4 * i + 1], h)),
                             make_float2(word_value<T>(w[4 * i + 2], h), word_value<T>(w[4 * i + 3], h))};
        codes_e4m3<2>(v, s[h].factor, c + i);
      }
      unsigned char* p = q.codes + (row + h) * q.pitch + col;
      if (TILED || (vec_codes && q.pitch % 16 == 0 && col + 32 <= q.pitch)) {
        *reinterpret_cast<uint4*>(p) = make_uint4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<uint4*>(p + 16) = make_uint4(c[4], c[5], c[6], c[7]);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (col + i < q.pitch) p[i] = (unsigned char)(c[i / 4] >> (8 * (i % 4)));
      }
    }
  }
}

// The scales of a 128-column block, whose words four warps have.
template <typename T>
__device__ __forceinline__ void join_blocks(const unsigned* w, unsigned (*red)[32][4 / sizeof(T)], BlockScale* s) {
  constexpr int W = 4 / sizeof(T);
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  unsigned m[W];
  words_amax<T, 32>(w, m);
#pragma unroll
  for (int h = 0; h < W; ++h) red[part][lane][h] = m[h];
  __syncthreads();
#pragma unroll
  for (int h = 0; h < W; ++h) {
    unsigned b = 0;
    for (int i = 0; i < 4; ++i) b = max(b, red[(part & 4) + i][lane][h]);
    s[h] = scale_fp32(b);
  }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kQuantThreads, 3) quant_transpose_kernel(const QuantArgs a) {
  start_after_stream();
  __shared__ unsigned tile[kTrCols * kTrPitch];
  constexpr int W = 4 / sizeof(T);             // rows of a lane
  __shared__ unsigned red[8][32][W];
  const QuantOut& q = a.q;
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * TrRows<T>::N, row = row0 + lane * W;
  const float mul = FMT == MX_NVFP4 ? mul_of(q) : 1.0f;
  const int64_t tiles = (q.cols + kTrCols - 1) / kTrCols;
  const unsigned* mine = tile + part * 32 * kTrPitch + lane;
  if (FMT >= MX_MXFP8 && blockIdx.y == 0)
    for (int h = 0; h < W; ++h)
      if (row + h < a.padded_rows) put_padding(q, row + h, part, 8);
  BlockScale s[W];
  unsigned w[32];
  if (FMT == MX_FP8_ROW) {
    unsigned m[W] = {};
    for (int64_t t = 0; t < tiles; ++t) {
      __syncthreads();
      load_tile<T>(a, row0, t * kTrCols, tile);
      __syncthreads();
      unsigned b[W];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = mine[i * kTrPitch];
      words_amax<T, 32>(w, b);
#pragma unroll
      for (int h = 0; h < W; ++h) m[h] = max(m[h], b[h]);
    }
#pragma unroll
    for (int h = 0; h < W; ++h) red[part][lane][h] = m[h];
    __syncthreads();
#pragma unroll
    for (int h = 0; h < W; ++h) {
      for (int i = 0; i < 8; ++i) m[h] = max(m[h], red[i][lane][h]);
      s[h] = scale_fp32(m[h]);
      if (part == 0 && row + h < q.rows) static_cast<float*>(q.scales)[row + h] = s[h].scale;
    }
  }
  for (int64_t t = blockIdx.y; t < tiles; t += gridDim.y) {
    __syncthreads();
    load_tile<T>(a, row0, t * kTrCols, tile);
    __syncthreads();
    const int64_t col = t * kTrCols + part * 32;
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = mine[i * kTrPitch];
    if (FMT == MX_FP8_BLOCK) join_blocks<T>(w, red, s);
    if (col < q.cols) put_columns<T, FMT>(q, row, col, w, mul, s, part % 4 == 0, a.vec_codes != 0);
  }
}

// The same with tiles that a tensor map copies, in a ring of kTrStages that stay
// in flight while the ones before are worked on (with loads through registers
// three CTAs an SM left HBM idle between them: 8192 x 8192 bf16 to mxfp8 49 us).
// The tile's rows of 128 bytes lie in the 128-byte swizzle: 16-byte part p of row
// c at p ^ (c % 8), so that a warp still reads a row's 32 words without conflict.
// CTAs take tiles a grid apart, those of one column of x after another.
constexpr int kTrStages = 3;
constexpr uint32_t kTrBytes = kTrCols * 128;

template <typename T, int FMT>
__global__ void __launch_bounds__(kQuantThreads, 2)
    quant_transpose_tma_kernel(const __grid_constant__ CUtensorMap map, const QuantArgs a, int64_t all) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t full[kTrStages];
  constexpr int W = 4 / sizeof(T);
  __shared__ unsigned red[8][32][W];
  const QuantOut& q = a.q;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int64_t tiles = (q.cols + kTrCols - 1) / kTrCols;      // along a row of the result
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTrStages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  start_after_stream();
  __syncthreads();
  const float mul = FMT == MX_NVFP4 ? mul_of(q) : 1.0f;
  const auto copy = [&](int64_t i, int st) {                   // by one thread
    const int64_t r = i / tiles, t = i - r * tiles;
    mbar_arrive_expect_tx(&full[st], kTrBytes);
    tma_load_2d(base + st * kTrBytes, &map, (int)(r * TrRows<T>::N), (int)(t * kTrCols), smem_addr(&full[st]));
  };
  if (threadIdx.x == 0)
    for (int k = 0; k < kTrStages; ++k)
      if (blockIdx.x + (int64_t)k * gridDim.x < all) copy(blockIdx.x + (int64_t)k * gridDim.x, k);
  int st = 0, round = 0;
  bool ok = true;
  for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
    // all threads go on, or none: a wait that gave up has the others give up too
    ok = __syncthreads_and(mbar_wait_cluster(&full[st], round & 1));
    if (!ok) break;
    const int64_t r = i / tiles, t = i - r * tiles;
    const int64_t row = r * TrRows<T>::N + lane * W, col = t * kTrCols + part * 32;
    if (FMT >= MX_MXFP8 && t == 0)
      for (int h = 0; h < W; ++h)
        if (row + h < a.padded_rows) put_padding(q, row + h, part, 8);
    unsigned w[32];
    const uint32_t tile = base + st * kTrBytes + part * 32 * 128;
#pragma unroll
    for (int k = 0; k < 32; ++k)
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[k]) : "r"(tile + k * 128 + (((lane >> 2) ^ (k & 7)) << 4) + (lane & 3) * 4));
    BlockScale s[W];
    if (FMT == MX_FP8_BLOCK) join_blocks<T>(w, red, s);
    __syncthreads();                                           // the stage is read
    if (threadIdx.x == 0 && i + (int64_t)kTrStages * gridDim.x < all) copy(i + (int64_t)kTrStages * gridDim.x, st);
    if (col < q.cols) put_columns<T, FMT>(q, row, col, w, mul, s, part % 4 == 0, a.vec_codes != 0);
    if (++st == kTrStages) {
      st = 0;
      ++round;
    }
  }
  if (!ok && threadIdx.x == 0) {      // copies in flight land before the CTA ends
    atomicOr(&g_tu_error, kErrWaitTimeout);
    for (int k = 0; k < kTrStages; ++k) {
      mbar_wait_cluster(&full[st], round & 1);
      if (++st == kTrStages) {
        st = 0;
        ++round;
      }
    }
  }
}

// The same with a scale a row: a CTA has its rows to itself and goes over their
// tiles twice, the second time mostly out of the L2 cache (9552 x 9344 fp16 166 us
// with loads through registers).
template <typename T>
__global__ void __launch_bounds__(kQuantThreads, 2)
    quant_transpose_row_tma_kernel(const __grid_constant__ CUtensorMap map, const QuantArgs a, int64_t all) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t full[kTrStages];
  constexpr int W = 4 / sizeof(T);
  __shared__ unsigned red[8][32][W];
  const QuantOut& q = a.q;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int64_t tiles = (q.cols + kTrCols - 1) / kTrCols;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTrStages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  start_after_stream();
  __syncthreads();
  // step i: tile i % tiles of pass i / tiles of a block of rows
  const auto copy = [&](int64_t r, int64_t i, int st) {
    mbar_arrive_expect_tx(&full[st], kTrBytes);
    tma_load_2d(base + st * kTrBytes, &map, (int)(r * TrRows<T>::N), (int)((i < tiles ? i : i - tiles) * kTrCols),
                smem_addr(&full[st]));
  };
  int st = 0, round = 0;
  bool ok = true;
  for (int64_t r = blockIdx.x; r < all && ok; r += gridDim.x) {
    const int64_t row = r * TrRows<T>::N + lane * W;
    if (threadIdx.x == 0)
      for (int k = 0; k < kTrStages && k < 2 * tiles; ++k) copy(r, k, (st + k) % kTrStages);
    unsigned m[W] = {};
    BlockScale s[W];
    for (int64_t i = 0; i < 2 * tiles; ++i) {
      ok = __syncthreads_and(mbar_wait_cluster(&full[st], round & 1));
      if (!ok) break;
      unsigned w[32];
      const uint32_t tile = base + st * kTrBytes + part * 32 * 128;
#pragma unroll
      for (int k = 0; k < 32; ++k)
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[k]) : "r"(tile + k * 128 + (((lane >> 2) ^ (k & 7)) << 4) + (lane & 3) * 4));
      if (i < tiles) {
        unsigned b[W];
        words_amax<T, 32>(w, b);
#pragma unroll
        for (int h = 0; h < W; ++h) m[h] = max(m[h], b[h]);
        if (i == tiles - 1) {
#pragma unroll
          for (int h = 0; h < W; ++h) red[part][lane][h] = m[h];
        }
      }
      __syncthreads();                                         // the stage is read, the maxima are there
      if (threadIdx.x == 0 && i + kTrStages < 2 * tiles) copy(r, i + kTrStages, st);
      if (i == tiles - 1) {
#pragma unroll
        for (int h = 0; h < W; ++h) {
          for (int k = 0; k < 8; ++k) m[h] = max(m[h], red[k][lane][h]);
          s[h] = scale_fp32(m[h]);
          if (part == 0 && row + h < q.rows) static_cast<float*>(q.scales)[row + h] = s[h].scale;
        }
      } else if (i >= tiles) {
        const int64_t col = (i - tiles) * kTrCols + part * 32;
        if (col < q.cols) put_columns<T, MX_FP8_ROW>(q, row, col, w, 1.0f, s, false, a.vec_codes != 0);
      }
      if (++st == kTrStages) {
        st = 0;
        ++round;
      }
    }
  }
  if (!ok && threadIdx.x == 0) {      // copies in flight land before the CTA ends
    atomicOr(&g_tu_error, kErrWaitTimeout);
    for (int k = 0; k < kTrStages; ++k) {
      mbar_wait_cluster(&full[st], round & 1);
      if (++st == kTrStages) {
        st = 0;
        ++round;
      }
    }
  }
}

// Values, 8 columns a lane. FMT 0: the formats with fp32 scales.
template <typename T, int FMT, bool RAGGED>
__global__ void __launch_bounds__(kQuantThreads) dequant_kernel(const QuantOut q, T* y, int64_t y_row,
                                                                bool vec_codes, int shift) {
  start_after_stream();
  constexpr bool FOUR = FMT >= MX_MXFP4;
  __shared__ __align__(16) T buffer[RAGGED ? kQuantThreads / 32 : 1][RAGGED ? 256 : 8];
  T* buf = buffer[RAGGED ? threadIdx.x >> 5 : 0];
  const LaneRows at(shift);
  const int64_t col = at.col;
  if (!RAGGED && col >= q.cols) return;
  const float mul = FMT == MX_NVFP4 ? mul_of(q) : 1.0f, r_mul = 1.0f / mul;
  const int64_t block = FMT == MX_FP8_ROW ? (q.fmt == MX_FP8_ROW ? 0 : col >> 7) : col / Format<FMT>::width;
  const int most = (int)max((int64_t)0, min((int64_t)8, q.cols - col));
#pragma unroll 2
  for (int64_t row = at.row; RAGGED ? __any_sync(0xffffffffu, row < q.rows) : row < q.rows; row += at.step) {
    const bool here = !RAGGED || (row < q.rows && most > 0);
    const unsigned char* codes = q.codes + row * q.pitch + (FOUR ? col / 2 : col);
    float2 v[4];
    float s = 0.f;
    if (!here) {
    } else if (FMT == MX_FP8_ROW) {
      s = static_cast<const float*>(q.scales)[row * q.blocks + block];
    } else {
      const unsigned b = static_cast<const unsigned char*>(q.scales)[scale_at(row, block, q.blocks)];
      if (FMT == MX_NVFP4)
        s = __half2float(__half(__nv_cvt_fp8_to_halfraw((unsigned char)b, __NV_E4M3)));
      else
        s = b == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float(b ? b << 23 : 1u << 22);
    }
    if (FOUR) {
      fp4_values(here ? *reinterpret_cast<const unsigned*>(codes) : 0u, v);
    } else {
      unsigned w[2] = {0, 0};
      if (!here) {
      } else if (vec_codes && most == 8) {
        const uint2 u = *reinterpret_cast<const uint2*>(codes);
        w[0] = u.x;
        w[1] = u.y;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < most) w[j / 4] |= (unsigned)codes[j] << (8 * (j % 4));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j / 2] >> (16 * (j % 2))), __NV_E4M3)));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], splat2(s));
    if (FMT == MX_NVFP4 && q.mul != nullptr) {
      float2 d[4];
      float all = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[j] = quotient2(v[j], mul, r_mul);
        all += d[j].x + d[j].y;
      }
      if (all != all || isinf(all)) {     // past the largest number the correction is inf - inf
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = make_float2(v[j].x / mul, v[j].y / mul);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = d[j];
      }
    }
    if (!RAGGED) {
      T* out = y + row * y_row + col;
      if (most == 8) {
#pragma unroll
        for (int j = 0; j < 8 / Vec<T>::N; ++j) st_vec(out + j * Vec<T>::N, pack2<T>(v + j * Vec<T>::N / 2));
      } else {
        const float* f = reinterpret_cast<const float*>(v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < most) out[j] = from_f<T>(f[j]);
      }
    } else {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8 / Vec<T>::N; ++j)
        reinterpret_cast<uint4*>(buf + (threadIdx.x & 31) * 8)[j] = pack2<T>(v + j * Vec<T>::N / 2);
      __syncwarp();
      each_element(row, col, shift, [&](int64_t er, int64_t ec, int e) {
        if (er < q.rows && ec < q.cols) y[er * y_row + ec] = buf[e];
      });
    }
  }
}

}  // namespace nf
