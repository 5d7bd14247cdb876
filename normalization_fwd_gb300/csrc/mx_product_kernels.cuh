// The product of two microscaled matrices on the tensor cores.
//
// A tile of results has 128 lanes of tensor memory by `cols` columns. One of the
// operands lies along the lanes (128 of its rows), the other along the columns.
// With few rows of A (SWAP) the lanes are B's rows (a projection's output
// features) and the columns A's: 16, 32 or 64 tokens cost a tile of that width
// and not one of 128. Otherwise lanes are A's rows and the 128 columns B's.
//
// K goes by in chunks of 128 bytes of codes a row (256 E2M1 or 128 E4M3): one
// thread copies a chunk's codes and scales to a ring of stages (tensor maps;
// the codes in the swizzle that the matrix instructions read, the scales as
// they lie, which is how tensor memory wants them), another one moves the scales
// on to tensor memory and issues four instructions of 32 bytes of K. Scales
// have a buffer there for each stage: a stage that is full again says that the
// instructions on what it held before are done, and so are those that read that
// buffer. The issuing warp asks for the next stage before it issues, by a test that
// returns at once (with one that may hold it back 16384 x 8192 x 8192 took 335 us).
//
// What bounds it: few rows of A, the weights' bytes and the fixed 4 us of a launch,
// a ring's first round and the join (16 x 8192 x 8192 nvfp4 10.7 us: 38 MB, 5.6 us of
// HBM's time, on 128 SMs). Many rows, the tensor cores: a chunk's four instructions take a
// pair of CTAs 512 cycles, moving its scales 10 cycles for each of their 12 (nvfp4),
// 6 (mxfp4) or 3 (mxfp8) tiles, and data is always there (16384 x 8192 x 8192
// nvfp4 314 us, 7.0 PFLOP/s, alone; 356 us in a loop, under the power limit; tensor
// pipe 74% active on a smaller case).
//
// Few tiles: K is split over the CTAs of a cluster. Each gets the tile's rows
// of results that it is to finish from all others through distributed shared
// memory and adds them in the order of the ranks.
//
// Every wait gives up after a second, reports it (ln_device_error) and lets the
// kernel end; barriers of the cluster are passed by every thread in any case.
#pragma once

#include "common.cuh"
#include "mx_formats.cuh"
#include "tcgen05.cuh"

namespace nf {

struct ProductArgs {
  QuantOut a, b;         // A [M, K], B [N, K]
  float alpha;
  const void* bias;
  const void* residual;
  int64_t residual_row;
  void* out;
  int64_t out_row;
  float *psum, *psq;
  int cols;              // columns of a tile
  int lane_tiles;        // tiles along the lanes' operand; the grid's x is lane_tiles * column tiles
  int splits;            // CTAs of a cluster, each with its share of the chunks
  int chunks;            // of K
  int steps;             // instructions along all of K
  int stages;
  int vec;               // out, residual and bias can be accessed 16 bytes at a time
  uint32_t idesc;
  int tiles_m, tiles_n;  // pairs of CTAs: tiles of 256 rows of A, of 128 or 256 of B
};

constexpr int kTileLanes = 128;
constexpr int kTileThreads = 256;
constexpr int kChunkBytes = 128;
constexpr int kTmemCols = 512;      // 128 or 256 of results, then scales
constexpr int kScaleCol = 128;
constexpr int kResultPitch = 132;   // floats of a row of results in shared memory
constexpr int kMaxStages = 10;

// 512-byte tiles of scales that a chunk takes.
template <int FMT> __host__ __device__ constexpr int chunk_tiles() { return FMT == MX_NVFP4 ? 4 : FMT == MX_MXFP4 ? 2 : 1; }
template <int FMT> __host__ __device__ constexpr uint32_t stage_bytes(int cols) {
  return (uint32_t)(kTileLanes + cols) * kChunkBytes + 2u * chunk_tiles<FMT>() * 512u;
}

// What the sums are multiplied by, alpha / mul of A / mul of B: `first`, then `second`,
// a power of two and mostly 1. As one number it need not be an fp32 one, nor alpha /
// mul of A, where the result is (two matrices of values about 1e-19 have factors of
// some 1e22 each): quotients of the fractions, powers of two apart.
struct Factor {
  float first, second;
};
__device__ __forceinline__ Factor factor_of(const ProductArgs& p) {
  int e, ea, eb;
  const float m = frexpf(p.alpha, &e) / frexpf(mul_of(p.a), &ea) / frexpf(mul_of(p.b), &eb);   // below 4
  e -= ea + eb;
  const int near = min(max(e, -124), 124);     // m * 2^near is a normal number
  // past these powers the product is 0 or infinite anyway: sums are below 2^64, and
  // with a mul (MX_NVFP4) multiples of 2^-20
  return {ldexpf(m, near), ldexpf(1.0f, min(max(e - near, -126), 127))};
}

// Rounding of a row of up to 128 results, four a lane, and its statistics.
template <typename T>
__device__ __forceinline__ void finish_row(const ProductArgs& p, int64_t m, int64_t n0, float4 acc,
                                           Factor f) {
  const int lane = threadIdx.x & 31;
  const int64_t n = n0 + lane * 4;
  const int live = (int)max((int64_t)0, min((int64_t)4, p.b.rows - n));
  float v[4] = {acc.x * f.first * f.second, acc.y * f.first * f.second, acc.z * f.first * f.second,
                acc.w * f.first * f.second};
  const T* res = p.residual ? static_cast<const T*>(p.residual) + m * p.residual_row + n : nullptr;
  T* out = static_cast<T*>(p.out) + m * p.out_row + n;
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < live) v[i] += to_f(static_cast<const T*>(p.bias)[n + i]);
  }
  T o[4];
  if (p.vec && live == 4) {
    if (res) {
      T r[4];
      if (sizeof(T) == 4) *reinterpret_cast<uint4*>(r) = *reinterpret_cast<const uint4*>(res);
      else *reinterpret_cast<uint2*>(r) = *reinterpret_cast<const uint2*>(res);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += to_f(r[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = from_f<T>(v[i]);
    if (sizeof(T) == 4) *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(o);
    else *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(o);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = from_f<T>(0.f);
      if (i < live) {
        if (res) v[i] += to_f(res[i]);
        o[i] = from_f<T>(v[i]);
        out[i] = o[i];
      }
    }
  }
  if (p.psum) {
    const int n_tile = (int)min((int64_t)128, p.b.rows - n0);
    float s = 0.f, q = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s += i < live ? to_f(o[i]) : 0.f;
    s = group_sum<32>(s);
    const float mean = s / (float)n_tile;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float d = i < live ? to_f(o[i]) - mean : 0.f;
      q = fmaf(d, d, q);
    }
    q = group_sum<32>(q);
    if (lane == 0) {
      const int64_t at = m * ((p.b.rows + 127) / 128) + n0 / 128;
      p.psum[at] = s;
      p.psq[at] = q;
    }
  }
}

template <typename T, int FMT, bool SWAP>
__global__ void __launch_bounds__(kTileThreads, 1)
    product_tile_kernel(const __grid_constant__ CUtensorMap lane_codes,
                        const __grid_constant__ CUtensorMap lane_scales,
                        const __grid_constant__ CUtensorMap col_codes,
                        const __grid_constant__ CUtensorMap col_scales, const ProductArgs p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
  __shared__ uint32_t tmem_at;
  constexpr int kTiles = chunk_tiles<FMT>();
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cols = SWAP ? p.cols : 128;
  const uint32_t rank = p.splits > 1 ? cluster_rank() : 0u;
  const int tile = blockIdx.x / p.splits;
  const int lane_row = tile % p.lane_tiles * kTileLanes, col_row = tile / p.lane_tiles * cols;
  const int c0 = (int)((int64_t)p.chunks * rank / p.splits);
  const int c1 = (int)((int64_t)p.chunks * (rank + 1) / p.splits);
  const uint32_t stage_size = stage_bytes<FMT>(cols);

  // A chunk's copies, by one thread.
  const auto copy = [&](int c, int st) {
    const uint32_t at = base + st * stage_size, bar = smem_addr(&full[st]);
    const uint32_t sc = at + (kTileLanes + cols) * kChunkBytes;
    mbar_arrive_expect_tx(&full[st], stage_size);
    tma_load_2d(at, &lane_codes, c * kChunkBytes, lane_row, bar);
    tma_load_2d(at + kTileLanes * kChunkBytes, &col_codes, c * kChunkBytes, col_row, bar);
    tma_load_3d(sc, &lane_scales, 0, c * kTiles, lane_row / 128, bar);
    tma_load_3d(sc + kTiles * 512, &col_scales, 0, c * kTiles, col_row / 128, bar);
  };
  // The ring's first round needs no one else: its copies are on their way while
  // tensor memory is handed out.
  const int first = min(p.stages, c1 - c0);
  if (warp == 0 && elect_one()) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    fence_mbar_init();
  }
  wait_for_stream();
  if (warp == 0 && elect_one())
    for (int i = 0; i < first; ++i) copy(c0 + i, i);
  if (warp == 2) tmem_alloc<kTmemCols>(&tmem_at);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  let_next_start();
  const uint32_t tmem = tmem_at;

  if (warp == 0) {
    bool ok = true;
    int st = first == p.stages ? 0 : first, round = first == p.stages ? 1 : 0, c = c0 + first;
    for (; c < c1; ++c) {
      if (!mbar_wait_cluster(&empty[st], (round - 1) & 1)) {
        ok = false;
        break;
      }
      if (elect_one()) copy(c, st);
      __syncwarp();
      if (++st == p.stages) {
        st = 0;
        ++round;
      }
    }
    if (!ok) {   // copies in flight land before the CTA ends
      if (lane == 0) atomicOr(&g_tu_error, kErrWaitTimeout);
      for (int i = max(c0, c - p.stages); i < c; ++i)
        mbar_wait_cluster(&full[(i - c0) % p.stages], ((i - c0) / p.stages) & 1);
    }
  } else if (warp == 1) {
    bool ok = true, here = mbar_ready_cluster(smem_addr(&full[0]), 0);
    int st = 0, round = 0;
    for (int c = c0; c < c1; ++c) {
      const int i = c - c0;
      ok = here || mbar_wait_cluster(&full[st], round & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const int next = st + 1 == p.stages ? 0 : st + 1;
      here = c + 1 < c1 && mbar_ready_cluster(smem_addr(&full[next]), (next == 0 ? round + 1 : round) & 1);
      const uint32_t at = base + st * stage_size;
      const uint32_t sc = at + (kTileLanes + cols) * kChunkBytes;
      const uint32_t sa = tmem + kScaleCol + st * 8 * kTiles, sb = sa + 4 * kTiles;
      const uint64_t da = operand_desc(at), db = operand_desc(at + kTileLanes * kChunkBytes), ds = scales_desc(sc);
      const int steps = min(4, p.steps - 4 * c);
      if (elect_one()) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          tc_copy_scales(sa + 4 * t, ds + 32 * t);
          tc_copy_scales(sb + 4 * t, ds + 32 * (kTiles + t));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // scales of the step: a tile of 4 a row serves 1, 2 or 4 steps
          const uint32_t col = 4 * (k * kTiles / 4), id = FMT == MX_NVFP4 ? 0 : FMT == MX_MXFP4 ? (k & 1) * 2 : k;
          if (k < steps)
            tc_mma<FMT>(tmem, da + 2 * k, db + 2 * k, p.idesc | (id << 29) | (id << 4), sa + col, sb + col,
                        i > 0 || k > 0);
        }
        tc_commit(smem_addr(&empty[st]));
      }
      __syncwarp();
      st = next;
      if (next == 0) ++round;
    }
    if (!ok && lane == 0) atomicOr(&g_tu_error, kErrWaitTimeout);
    if (elect_one()) tc_commit(smem_addr(&done));
  }
  __syncwarp();
  if (!mbar_wait_cluster(&done, 0)) atomicOr(&g_tu_error, kErrWaitTimeout);
  __syncwarp();
  tc_fence_after();
  // The stages are read and become the place of the results: of all CTAs of the cluster.
  if (p.splits > 1) cluster_sync();
  else __syncthreads();

  const int tile_rows = SWAP ? cols : kTileLanes;          // rows of results
  const int rows_each = tile_rows / p.splits;              // that a CTA finishes
  const uint32_t lane_base = (uint32_t)(warp & 3) * 32;    // the warp's lanes of tensor memory
  const int half = warp >> 2;                              // of the columns
  for (int j = half * 16; j < cols; j += 32) {
    float v[16];
    tmem_load16(tmem + (lane_base << 16) + j, v);
    if (SWAP) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = j + i, to = r / rows_each;
        const uint32_t at = base + (((rank * rows_each + r - to * rows_each) * kResultPitch) + lane_base + lane) * 4;
        st_cluster(map_to_rank(at, to), v[i]);
      }
    } else {
      const int r = lane_base + lane, to = r / rows_each;
      const uint32_t at = map_to_rank(base + (((rank * rows_each + r - to * rows_each) * kResultPitch) + j) * 4, to);
#pragma unroll
      for (int i = 0; i < 16; i += 4) st_cluster4(at + 4 * i, make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
    }
  }
  tc_fence_before();
  if (p.splits > 1) cluster_sync();
  else __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_free<kTmemCols>(tmem);
  }

  const Factor f = factor_of(p);
  const int64_t m0 = (SWAP ? col_row : lane_row) + (int64_t)rank * rows_each, n0 = SWAP ? lane_row : col_row;
  for (int r = warp; r < rows_each; r += kTileThreads / 32) {
    if (m0 + r >= p.a.rows) break;
    float4 s = lds_f4(base + (r * kResultPitch + lane * 4) * 4);
    for (int q = 1; q < p.splits; ++q) {
      const float4 t = lds_f4(base + ((q * rows_each + r) * kResultPitch + lane * 4) * 4);
      s = make_float4(s.x + t.x, s.y + t.y, s.z + t.z, s.w + t.w);
    }
    finish_row<T>(p, m0 + r, n0, s, f);
  }
}

// ---- pairs of CTAs ------------------------------------------------------------
//
// Tiles of 256 by WN results (WN = 128 or 256) by pairs of CTAs that stay and
// take one tile after another. A step of the pair reads 128 rows of A and WN / 2
// of B from each CTA's shared memory, so that a chunk costs half the copies a
// result of two single tiles. Warps: 0 copies, 1 issues (in the first CTA of the
// pair) and has the tensor memory, 4 to 11 finish results. WN = 256: the results
// fill one half of tensor memory, the eight warps take 128 columns a thread into
// registers and hand it back at once; WN = 128: two buffers, four warps each.
constexpr int kPairThreads = 384;   // 168 registers a thread, of which 128 hold results

template <int FMT> __host__ __device__ constexpr uint32_t pair_stage_bytes(int wn) {
  return (uint32_t)(128 + wn / 2) * kChunkBytes + (uint32_t)(1 + wn / 128) * chunk_tiles<FMT>() * 512u;
}

// The same, up to where the next stage may begin.
template <int FMT> __host__ __device__ constexpr uint32_t pair_stage_step(int wn) {
  return (pair_stage_bytes<FMT>(wn) + 1023u) / 1024u * 1024u;
}

// Tile t in an order that keeps what runs at a time in few rows of A and B:
// groups of 8 tiles of A's rows, all of B's columns in each.
__device__ __forceinline__ void pair_tile(const ProductArgs& p, int t, int* tm, int* tn) {
  const int per = 8 * p.tiles_n, g = t / per, rest = t - g * per;
  const int rows = min(8, p.tiles_m - g * 8);
  *tn = rest / rows;
  *tm = g * 8 + rest - *tn * rows;
}

// A warp's 32 rows by 128 columns of results, a row a lane. A lane scales,
// rounds and sums its own row; 64 bytes of each row at a time change places
// through shared memory, so that rows of the residual and the output are read
// and written in runs of 64 bytes (straight from a row a lane, 4099 x 1165 x 1280,
// whose 16-bit rows start anywhere, took 78 us).
constexpr int kPiecePitch = 80;      // bytes: 16-byte accesses of 8 rows meet no bank twice
constexpr int kPieceBytes = 32 * kPiecePitch;

// The output is not read again by this kernel, the residual not twice: their
// lines make way in the L2 cache for those of the operands first. Volatile, so
// that the loads of later pieces are not moved ahead of the ones before and need
// registers all at once.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_bias(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
// Tiles of 32 rows and 128 columns that can be accessed 16 bytes at a time, so
// that nothing is asked along the way. `load` waits for the results and takes
// them into registers; false: they did not come. The residual's first piece is
// on its way before.
template <typename T, bool RES, bool SUMS, typename Load>
__device__ __forceinline__ bool finish_full(const ProductArgs& p, int64_t m0, int64_t n0, Factor f,
                                            unsigned char* piece, Load load) {
  constexpr int N = Vec<T>::N, kCols = 4 * N, kPieces = 128 / kCols;
  const int lane = threadIdx.x & 31, part = lane & 3, row = lane >> 2;
  uint4* own = reinterpret_cast<uint4*>(piece + lane * kPiecePitch);
  uint4* other = reinterpret_cast<uint4*>(piece + row * kPiecePitch + part * 16);
  constexpr int kStep = 8 * kPiecePitch / 16;
  const int64_t res_step = 8 * p.residual_row, out_step = 8 * p.out_row;
  const T* res = static_cast<const T*>(p.residual) + (m0 + row) * p.residual_row + n0 + part * N;
  T* out = static_cast<T*>(p.out) + (m0 + row) * p.out_row + n0 + part * N;
  const T* bias = p.bias ? static_cast<const T*>(p.bias) + n0 : nullptr;
  float sum = 0.f, m2 = 0.f;          // of the columns so far
  uint4 next[4];
  const auto fetch = [&](int col) {
#pragma unroll
    for (int i = 0; i < 4; ++i) next[i] = ld_stream(res + i * res_step + col);
  };
  if (RES) fetch(0);
  uint32_t v[128];
  if (!load(v)) return false;
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int col = j * kCols;
    if (RES) {
#pragma unroll
      for (int i = 0; i < 4; ++i) other[i * kStep] = next[i];
      __syncwarp();
    }
    uint4 mine[4];
    float2 s2 = splat2(0.f);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int at = col + c * N;
      float2 o[N / 2];
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        o[i] = mul2(mul2(make_float2(__uint_as_float(v[at + 2 * i]), __uint_as_float(v[at + 2 * i + 1])),
                         splat2(f.first)), splat2(f.second));
      if (bias) {
        float2 b[N / 2];
        unpack2<T>(ld_bias(bias + at), b);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) o[i] = add2(o[i], b[i]);
      }
      if (RES) {
        float2 r[N / 2];
        unpack2<T>(own[c], r);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) o[i] = add2(o[i], r[i]);
      }
      mine[c] = pack2<T>(o);
      own[c] = mine[c];
      if (SUMS) {
        unpack2<T>(mine[c], o);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) s2 = add2(s2, o[i]);
      }
    }
    if (RES && j + 1 < kPieces) fetch(col + kCols);     // into registers that are free now
    __syncwarp();
    uint4 t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = other[i * kStep];
#pragma unroll
    for (int i = 0; i < 4; ++i) __stcs(reinterpret_cast<uint4*>(out + i * out_step + col), t[i]);
    if (SUMS) {
      // the piece's sum and squares about its own mean, joined to those before
      // (the parallel-variance identity)
      const float s = s2.x + s2.y, mean = s * (1.0f / kCols);
      float2 q = splat2(0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float2 o[N / 2];
        unpack2<T>(mine[c], o);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float2 d = add2(o[i], splat2(-mean));
          q = fma2(d, d, q);
        }
      }
      m2 += q.x + q.y;
      if (j > 0) {
        const float d = mean - sum / (float)col;
        m2 = fmaf(d * d, (float)col * kCols / (float)(col + kCols), m2);
      }
      sum += s;
    }
    __syncwarp();
  }
  if (SUMS) {
    const int64_t at = (m0 + lane) * ((p.b.rows + 127) / 128) + n0 / 128;
    p.psum[at] = sum;
    p.psq[at] = m2;
  }
  return true;
}

// Any other tile (rows or columns that the matrix does not have, rows that start
// anywhere), 16 columns at a time as fp32 in shared memory: 16 lanes a row for
// what is read and written.
template <typename T, typename Load>
__device__ __forceinline__ bool finish_ragged(const ProductArgs& p, int64_t m0, int64_t n0, Factor f,
                                              unsigned char* piece, Load load) {
  const int lane = threadIdx.x & 31, c = lane & 15;
  const int rows = (int)max((int64_t)0, min((int64_t)32, p.a.rows - m0));
  const int width = (int)max((int64_t)0, min((int64_t)128, p.b.rows - n0));
  float4* own = reinterpret_cast<float4*>(piece + lane * kPiecePitch);
  float* there = reinterpret_cast<float*>(piece) + (lane >> 4) * (kPiecePitch / 4) + c;
  const T* res = p.residual ? static_cast<const T*>(p.residual) + (m0 + (lane >> 4)) * p.residual_row + n0 + c : nullptr;
  T* out = static_cast<T*>(p.out) + (m0 + (lane >> 4)) * p.out_row + n0 + c;
  const int64_t res_step = 2 * p.residual_row, out_step = 2 * p.out_row;
  float sum = 0.f, m2 = 0.f;
  uint32_t v[128];
  if (!load(v)) return false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int col = 16 * j;
    if (rows == 0 || col >= width) break;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      own[i] = make_float4(__uint_as_float(v[col + 4 * i]) * f.first * f.second,
                           __uint_as_float(v[col + 4 * i + 1]) * f.first * f.second,
                           __uint_as_float(v[col + 4 * i + 2]) * f.first * f.second,
                           __uint_as_float(v[col + 4 * i + 3]) * f.first * f.second);
    __syncwarp();
    const int live = col + c < width ? (rows - (lane >> 4) + 1) / 2 : 0;    // rows of this lane's column
    const float b = p.bias && live > 0 ? to_f(static_cast<const T*>(p.bias)[n0 + col + c]) : 0.f;
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = res && i < live ? to_f(res[i * res_step + col]) : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float* x = there + 2 * i * (kPiecePitch / 4);
      T o = from_f<T>(0.f);
      if (i < live) {
        o = from_f<T>(*x + b + y[i]);
        out[i * out_step + col] = o;
      }
      if (p.psum) *x = to_f(o);
    }
    __syncwarp();
    if (p.psum) {
      const int cnt = min(16, width - col);
      float s = 0.f, q = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) s += (own[i].x + own[i].y) + (own[i].z + own[i].w);   // 0 behind the last column
      const float mean = s / (float)cnt;
      for (int i = 0; i < cnt; ++i) {
        const float d = reinterpret_cast<const float*>(own)[i] - mean;
        q = fmaf(d, d, q);
      }
      m2 += q;
      if (j > 0) {
        const float d = mean - sum / (float)col;
        m2 = fmaf(d * d, (float)col * (float)cnt / (float)(col + cnt), m2);
      }
      sum += s;
    }
    __syncwarp();
  }
  if (p.psum && lane < rows && width > 0) {
    const int64_t at = (m0 + lane) * ((p.b.rows + 127) / 128) + n0 / 128;
    p.psum[at] = sum;
    p.psq[at] = m2;
  }
  return true;
}

// The lines of a warp's rows of the residual, on their way to the L2 cache while
// the tile's results are still being worked out.
template <typename T>
__device__ __forceinline__ void prefetch_residual(const ProductArgs& p, int64_t m0, int64_t n0) {
  const int64_t m = m0 + (threadIdx.x & 31);
  if (m >= p.a.rows || n0 >= p.b.rows) return;
  const char* at = reinterpret_cast<const char*>(static_cast<const T*>(p.residual) + m * p.residual_row + n0);
  const int bytes = (int)min((int64_t)128, p.b.rows - n0) * (int)sizeof(T);
  for (int b = 0; b < bytes; b += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + b));
}

template <typename T, int FMT, int WN>
__global__ void __launch_bounds__(kPairThreads, 1)
    product_pair_kernel(const __grid_constant__ CUtensorMap a_codes,
                        const __grid_constant__ CUtensorMap a_scales,
                        const __grid_constant__ CUtensorMap b_codes,
                        const __grid_constant__ CUtensorMap b_scales, const ProductArgs p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], ready[2], drained[2];
  __shared__ uint32_t tmem_at;
  constexpr int kTiles = chunk_tiles<FMT>();
  constexpr int kBufs = 256 / WN;                        // of results
  constexpr int kRowTiles = WN / 128;                    // of B's scales
  constexpr uint32_t kStage = pair_stage_step<FMT>(WN);
  constexpr int kScaleStep = 4 * kTiles * (1 + kRowTiles);   // columns of a stage's scales
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2, tiles = p.tiles_m * p.tiles_n;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ready[i], 1);
      mbar_init(&drained[i], 2 * (WN == 256 ? 8 : 4));   // warps of both CTAs
    }
    fence_mbar_init();
    tma_prefetch(&a_codes);
    tma_prefetch(&a_scales);
    tma_prefetch(&b_codes);
    tma_prefetch(&b_scales);
  }
  wait_for_stream();
  if (warp == 1) tmem_alloc_pair<kTmemCols>(&tmem_at);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  let_next_start();
  const uint32_t tmem = tmem_at;

  if (warp == 0) {
    bool ok = true;
    int i = 0, st = 0, round = 0;                        // chunks copied, stage and its use
    for (int t = pair; t < tiles && ok; t += pairs) {
      int tm, tn;
      pair_tile(p, t, &tm, &tn);
      const int a_row = tm * 256 + (int)rank * 128, b_row = tn * WN;
      for (int c = 0; c < p.chunks; ++c, ++i) {
        if (round > 0 && !mbar_wait_cluster(&empty[st], (round - 1) & 1)) {
          ok = false;
          break;
        }
        const uint32_t at = base + st * kStage, sc = at + (128 + WN / 2) * kChunkBytes;
        const uint32_t bar = map_to_rank(smem_addr(&full[st]), 0);
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * pair_stage_bytes<FMT>(WN));
          tma_load_2d_pair(at, &a_codes, c * kChunkBytes, a_row, bar);
          tma_load_2d_pair(at + 128 * kChunkBytes, &b_codes, c * kChunkBytes, b_row + (int)rank * (WN / 2), bar);
          tma_load_3d_pair(sc, &a_scales, 0, c * kTiles, a_row / 128, bar);
          tma_load_3d_pair(sc + kTiles * 512, &b_scales, 0, c * kTiles, b_row / 128, bar);
        }
        __syncwarp();
        if (++st == p.stages) {
          st = 0;
          ++round;
        }
      }
    }
    if (!ok && lane == 0) atomicOr(&g_tu_error, kErrWaitTimeout);
    // Copies in flight and arrivals from the other CTA land before this one ends:
    // a stage that is free again has had both. After a wait that gave up, the
    // first CTA waits a second more for what it asked for.
    for (int k = max(0, i - p.stages); k < i && ok; ++k)
      ok = mbar_wait_cluster(&empty[k % p.stages], (k / p.stages) & 1);
    if (!ok && rank == 0)
      for (int k = max(0, i - p.stages); k < i; ++k) mbar_wait_cluster(&full[k % p.stages], (k / p.stages) & 1);
  } else if (warp == 1 && rank == 0) {
    bool ok = true;
    int i = 0, n = 0;                                    // chunks and tiles so far
    int st = 0, round = 0;
    bool here = mbar_ready_cluster(smem_addr(&full[0]), 0);
    for (int t = pair; t < tiles && ok; t += pairs, ++n) {
      const int buf = n % kBufs;
      if (n >= kBufs) ok = __all_sync(0xffffffffu, mbar_wait_cluster(&drained[buf], (n / kBufs - 1) & 1));
      tc_fence_after();
      for (int c = 0; c < p.chunks && ok; ++c, ++i) {
        ok = here || mbar_wait_cluster(&full[st], round & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const int next = st + 1 == p.stages ? 0 : st + 1;
        here = (c + 1 < p.chunks || t + pairs < tiles) &&
               mbar_ready_cluster(smem_addr(&full[next]), (next == 0 ? round + 1 : round) & 1);
        const uint32_t at = base + st * kStage, sc = at + (128 + WN / 2) * kChunkBytes;
        const uint32_t sa = tmem + 256 + st * kScaleStep, sb = sa + 4 * kTiles;
        const uint64_t da = operand_desc(at), db = operand_desc(at + 128 * kChunkBytes), ds = scales_desc(sc);
        const int steps = min(4, p.steps - 4 * c);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kTiles; ++k) {
            tc_copy_scales_pair(sa + 4 * k, ds + 32 * k);
#pragma unroll
            for (int r = 0; r < kRowTiles; ++r)
              tc_copy_scales_pair(sb + 4 * (k * kRowTiles + r), ds + 32 * (kTiles * (1 + r) + k));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t tile = k * kTiles / 4, id = FMT == MX_NVFP4 ? 0 : FMT == MX_MXFP4 ? (k & 1) * 2 : k;
            if (k < steps)
              tc_mma_pair<FMT>(tmem + buf * WN, da + 2 * k, db + 2 * k, p.idesc | (id << 29) | (id << 4),
                               sa + 4 * tile, sb + 4 * tile * kRowTiles, c > 0 || k > 0);
          }
          tc_commit_pair(smem_addr(&empty[st]));
        }
        __syncwarp();
        st = next;
        if (next == 0) ++round;
      }
      if (elect_one()) tc_commit_pair(smem_addr(&ready[buf]));
      __syncwarp();
    }
    if (!ok && lane == 0) atomicOr(&g_tu_error, kErrWaitTimeout);
    // all that was issued is done before tensor memory goes back, and the other
    // CTA's arrivals have come before this one ends
    for (int e = max(0, i - p.stages); e < i; ++e) mbar_wait_cluster(&empty[e % p.stages], (e / p.stages) & 1);
    for (int e = max(0, n - kBufs); e < n && ok; ++e) mbar_wait_cluster(&drained[e % kBufs], (e / kBufs) & 1);
  } else if (warp >= 4) {
    const int quarter = warp & 3, group = (warp - 4) >> 2;
    const Factor f = factor_of(p);
    unsigned char* piece = smem_raw + (base - smem_addr(smem_raw)) + p.stages * kStage + (warp - 4) * kPieceBytes;
    int n = 0;
    for (int t = pair; t < tiles; t += pairs, ++n) {
      const int buf = n % kBufs;
      if (WN == 128 && buf != group) continue;
      int tm, tn;
      pair_tile(p, t, &tm, &tn);
      const int col = WN == 256 ? group * 128 : 0;
      const int64_t m0 = (int64_t)tm * 256 + rank * 128 + quarter * 32, n0 = (int64_t)tn * WN + col;
      if (p.residual) prefetch_residual<T>(p, m0, n0);
      const auto load = [&](uint32_t* v) {
        const bool here = __all_sync(0xffffffffu, mbar_wait_cluster(&ready[buf], (n / kBufs) & 1));
        if (!here) return false;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 4; ++j) tmem_load32(tmem + ((uint32_t)quarter << 21) + buf * WN + col + 32 * j, v + 32 * j);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_addr(&drained[buf]), 0));
        return true;
      };
      bool ok;
      if (!p.vec || m0 + 32 > p.a.rows || n0 + 128 > p.b.rows) ok = finish_ragged<T>(p, m0, n0, f, piece, load);
      else if (p.psum && p.residual) ok = finish_full<T, true, true>(p, m0, n0, f, piece, load);
      else if (p.psum) ok = finish_full<T, false, true>(p, m0, n0, f, piece, load);
      else if (p.residual) ok = finish_full<T, true, false>(p, m0, n0, f, piece, load);
      else ok = finish_full<T, false, false>(p, m0, n0, f, piece, load);
      if (!ok) {
        if (lane == 0) atomicOr(&g_tu_error, kErrWaitTimeout);
        break;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_free_pair<kTmemCols>(tmem);
  }
}

}  // namespace nf
