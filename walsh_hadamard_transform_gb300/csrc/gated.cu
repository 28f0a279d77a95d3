// Gated projections h = act(x Wg^T) * (x Wu^T) and their gradients, on tensor cores.
//
// Four products of 16-bit operands share one kernel:
//
//   forward    [g u] = x [Wg; Wu]^T     a tile holds the same columns of g and of u side by
//                                       side in tensor memory, so the epilogue has both:
//                                       h = act(g) * u, one rounding
//   gradients  the same, and dg = dh u act'(g), du = dh act(g)
//   dx         dg Wg + du Wu            one contraction of twice the length
//   dw         dg^T x and du^T x        the tiles of both in one launch
//
// CTAs are persistent, one an SM.  One warp fills a ring of operand stages by TMA (128 bytes
// of the contraction, 128-byte swizzle; operands that run across the contraction are read
// MN-major, so nothing is transposed in memory), one thread issues the products, and eight
// warps turn finished accumulators into output while the next tile's products run in the
// other half of tensor memory.  (With four warps the gradients' epilogue took longer than
// a tile's products: the whole backward pass of 8192 x 2048 x 8192 1086 us against 1027.)  Large products
// pair two CTAs on a tile of 256 x 256: each loads half of both operands, which halves the
// shared-memory traffic of the second.
//
// Bound, large: the tensor cores under the power limit.  8192 x 4096 x 8192 bf16 forward: 513
// to 530 us in bursts, 599 for seconds on end (1545 MHz), 2140 to 1840 TFLOP/s, the tensor pipe active
// 92% of the cycles; 8192 x 2048 x 8192 backward: 0.92 and 1.04 ms (1530 MHz), 1800 and 1590 TFLOP/s.
// Small: latency, some 3 us from launch to the last store and 0.2 to 0.3 us a stage; 333 x
// 1001 x 2731 forward 7.5 us, 517 x 1001 x 2731 backward 41 us in three launches, 50 us in
// float16 with the bounds' before them.  64 x 2048 x 8192 backward: 64 us, float16 84.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "feed_forward.cuh"
#include "ff_host.cuh"
#include "fwt.h"
#include "tcgen05.cuh"

namespace fwt {
namespace ff {
namespace {

enum Mode { kForward, kGradients, kDx, kDw };

struct GemmParams {
  int m, n;               // rows and columns of the output
  int k_blocks, phases;   // stages of 64 along the contraction, times over (two operand pairs)
  int tiles_m, tiles_n, outputs;
  const void* grad;       // gradients: dh
  int64_t ld_grad;
  void* out[2];
  int64_t ld_out[2];
  int act;
  int vec;                // output rows start on 16-byte boundaries
  Bounds bounds;          // gradients, dx and dw in float16
};

struct GemmMaps {
  CUtensorMap a[2], b[2];
};

constexpr int kTileK = 64;  // elements of the contraction in a stage: one swizzle row
constexpr int kRingBytes = 196608;
constexpr int kThreads = 320;  // a warp each for copies and products, eight for the epilogue
constexpr int kPieceBytes = 32 * 64;  // 32 columns of a warp's 32 rows, see store_rows

// CG: CTAs that share a tile.  BN: columns of its accumulator.  Each CTA holds 128 rows of
// the first operand and BN / CG lines of the second.
template <int CG, int BN>
struct Config {
  static constexpr int kABytes = 128 * 128, kBBytes = BN / CG * 128;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = kRingBytes / kStage;
  static constexpr size_t kSmem = (size_t)kStages * kStage + 8 * kPieceBytes + 1024;
};

struct Tile {
  int m0, n0, output;
};

// Tiles in groups of 16 rows of tiles, so that those in flight together share operands in L2
// (measured, us, at 8 and at 16: 4096 x 4096 x 8192 forward 306 and 290, 8192 x 4096 x 8192
// the same).
constexpr int kGroup = 16;
__device__ __forceinline__ Tile tile_at(const GemmParams& p, int index, int rows, int cols) {
  const int area = p.tiles_m * p.tiles_n;
  Tile t;
  t.output = index / area;
  index -= t.output * area;
  const int group = index / (kGroup * p.tiles_n);
  const int height = min(kGroup, p.tiles_m - group * kGroup);
  index -= group * kGroup * p.tiles_n;
  t.m0 = (group * kGroup + index % height) * rows;
  t.n0 = index / height * cols;
  return t;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 v = __floats2half2_rn(a, b);
    return *(const uint32_t*)&v;
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *(const uint32_t*)&v;
  }
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (std::is_same<T, __half>::value) return __half22float2(*(const __half2*)&v);
  else return __bfloat1622float2(*(const __nv_bfloat162*)&v);
}

// A warp's 32 rows from `row0` on, W columns from `col`, one row a thread as pairs: through
// the warp's piece of shared memory (16-byte chunks, swizzled by row), so that global memory
// sees whole runs of a row and not 16 bytes of each.  Outside m x n nothing is touched.
template <int W>
__device__ __forceinline__ uint4* piece_at(uint8_t* piece, int row, int chunk) {
  constexpr int kChunks = W / 8;
  return (uint4*)(piece + (row * kChunks + ((chunk ^ (row * kChunks / 8)) & (kChunks - 1))) * 16);
}
template <typename T, int W>
__device__ __forceinline__ void store_rows(T* out, int64_t ld, uint8_t* piece, int row0, int lane,
                                           int m, int col, int n, bool vec, const uint32_t (&v)[W / 2]) {
  constexpr int kChunks = W / 8;
  static_assert(kChunks > 0, "whole 16-byte chunks");
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
    *piece_at<W>(piece, lane, i) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int r = i * (32 / kChunks) + lane / kChunks, chunk = lane & (kChunks - 1);
    const uint4 q = *piece_at<W>(piece, r, chunk);
    const int at = col + 8 * chunk;
    if (row0 + r < m && at < n) {
      T* to = out + (int64_t)(row0 + r) * ld + at;
      if (vec && at + 8 <= n) {
        *(uint4*)to = q;
      } else {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at + j < n) *(unsigned short*)(to + j) = (unsigned short)(w[j / 2] >> (16 * (j & 1)));
      }
    }
  }
}
// (Rows of `in` start on 16-byte boundaries.)
template <typename T, int W>
__device__ __forceinline__ void load_rows(const T* in, int64_t ld, uint8_t* piece, int row0, int lane,
                                          int m, int col, int n, uint32_t (&v)[W / 2]) {
  constexpr int kChunks = W / 8;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int r = i * (32 / kChunks) + lane / kChunks, chunk = lane & (kChunks - 1);
    const int at = col + 8 * chunk;
    uint4 q = make_uint4(0, 0, 0, 0);
    if (row0 + r < m && at < n) {
      const T* from = in + (int64_t)(row0 + r) * ld + at;
      if (at + 8 <= n) {
        q = *(const uint4*)from;
      } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (at + j < n) w[j / 2] |= (uint32_t)((const unsigned short*)from)[j] << (16 * (j & 1));
        q = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    *piece_at<W>(piece, r, chunk) = q;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const uint4 q = *piece_at<W>(piece, lane, i);
    v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
  }
}

// ---- the range of dg and du in float16 -------------------------------------------------
//
// dg = dh u act'(g) and du = dh act(g) of a scaled loss pass 65504 long before the sums over them
// do, and the gradients at the end of training fall below 2^-24.  |u| <= |x_m| |w_up_f| (Euclidean
// norms), |act(g)| <= |g| <= |x_m| |w_gate_f| and |act'| < 1.13, so
//
//     |dg|, |du| <= 1.13 max_m (max_f |dh| |x_m|) max_f max(|w_gate_f|, |w_up_f|) = B,
//
// and both are held as 2^k dg and 2^k du with 2^14 <= 2^k B < 2^15 (kGradients), of which dx and
// dw take 2^k away from their fp32 sums.  Powers of two change no rounding; what lies below
// 2^-28 B is held in steps of 2^-38 B or less.  k is one for the whole call, as dx sums over the columns of dg and dw over its rows.  bfloat16 has fp32's range and needs
// none of it.  Elements that are not finite count as zero here: their rows and columns are not
// finite either way, and the others keep a scale of their own making.
//
// Bound: the latency of a row's few loads, then HBM, every input once: 9 us of the 50 that 517 x
// 1001 x 2731 takes (17 MB), 20 us for 64 x 2048 x 8192 (69 MB), where 24 were with half the warps.

// The largest magnitude (SQUARES: the sum of squares) of a row, over the lanes of a warp.
// Elements that are not finite are left out, in a second pass where there are any: no finite
// float16 takes either beyond fp32.
template <bool SQUARES, bool CHECKED>
__device__ __forceinline__ float row_pass(const __half* from, int cols, int lane) {
  float sums[8] = {};  // independent of one another: the additions' latency bounds this
  auto take = [](float& sum, float v) {
    if (CHECKED && !(fabsf(v) < INFINITY)) return;
    sum = SQUARES ? fmaf(v, v, sum) : fmaxf(sum, fabsf(v));
  };
  constexpr int kAhead = 4;
  const int whole = cols & ~7;
  for (int64_t c = 8 * lane; c < whole; c += 256 * kAhead) {
    uint4 q[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      q[i] = c + 256 * i < whole ? *(const uint4*)(from + c + 256 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = unpack2<__half>(w[j]);
        take(sums[2 * j], v.x), take(sums[2 * j + 1], v.y);
      }
    }
  }
  if (whole + lane < cols) take(sums[0], __half2float(from[whole + lane]));
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) sum = SQUARES ? sum + sums[j] : fmaxf(sum, sums[j]);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float other = __shfl_xor_sync(~0u, sum, o);
    sum = SQUARES ? sum + other : fmaxf(sum, other);
  }
  return sum;
}
template <bool SQUARES>
__device__ __forceinline__ float row_magnitude(CMat mat, int row, int cols, int lane) {
  const __half* from = (const __half*)mat.p + (int64_t)row * mat.ld;
  const float sum = row_pass<SQUARES, false>(from, cols, lane);
  return sum < INFINITY ? sum : row_pass<SQUARES, true>(from, cols, lane);
}

struct BoundParams {
  CMat grad, x, w_gate, w_up;
  float2* pairs;
  int m, f, d;
};
constexpr int kBoundWarps = 16;

__global__ void __launch_bounds__(kBoundWarps * 32, 3) bounds_kernel(const BoundParams p) {
  __shared__ float2 tops[kBoundWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rows = (int64_t)p.m + p.f;
  float2 most = make_float2(0.f, 0.f);
  pdl_begin();
  for (int64_t r = (int64_t)blockIdx.x * kBoundWarps + warp; r < rows; r += (int64_t)gridDim.x * kBoundWarps) {
    if (r < p.m) {
      const float dh = row_magnitude<false>(p.grad, (int)r, p.f, lane);
      const float x = row_magnitude<true>(p.x, (int)r, p.d, lane);
      most.x = fmaxf(most.x, dh * sqrtf(x));
    } else {
      const int j = (int)(r - p.m);
      const float g = row_magnitude<true>(p.w_gate, j, p.d, lane);
      const float u = row_magnitude<true>(p.w_up, j, p.d, lane);
      most.y = fmaxf(most.y, sqrtf(fmaxf(g, u)));
    }
  }
  if (lane == 0) tops[warp] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kBoundWarps; ++w)
      most.x = fmaxf(most.x, tops[w].x), most.y = fmaxf(most.y, tops[w].y);
    p.pairs[blockIdx.x] = most;
  }
}

// 2^k (INVERSE: 2^-k) in every lane of a warp; 1 where the bound is zero.  Bounds of float16
// operands lie between 2^-73 and 2^80, so both are normal numbers.
template <bool INVERSE>
__device__ __forceinline__ float range_scale(const Bounds& b, int lane) {
  float2 most = make_float2(0.f, 0.f);
  for (int i = lane; i < b.parts; i += 32) {
    const float2 v = ((const float2*)b.pairs)[i];
    most.x = fmaxf(most.x, v.x), most.y = fmaxf(most.y, v.y);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    most.x = fmaxf(most.x, __shfl_xor_sync(~0u, most.x, o));
    most.y = fmaxf(most.y, __shfl_xor_sync(~0u, most.y, o));
  }
  const float bound = 1.13f * most.x * most.y;
  if (!(bound > 0.f)) return 1.f;
  const int e = (int)(__float_as_uint(bound) >> 23) - 127;  // 2^e <= bound < 2^(e + 1)
  return __uint_as_float((uint32_t)(127 + (INVERSE ? e - 14 : 14 - e)) << 23);
}

// SPLIT: CTAs of a cluster that share out the contraction of a tile.
template <typename T, int MODE, int CG, int BN, int SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ GemmMaps maps, const GemmParams p) {
  using C = Config<CG, BN>;
  constexpr bool kPairedWeights = MODE == kForward || MODE == kGradients;
  constexpr bool kAcrossA = MODE == kDw, kAcrossB = MODE == kDx || MODE == kDw;
  constexpr int kCols = kPairedWeights ? BN / 2 : BN;  // output columns of a tile
  constexpr uint32_t kIdesc =
      instruction(std::is_same<T, __half>::value ? 0 : 1, kAcrossA, kAcrossB, 128 * CG, BN);

  extern __shared__ uint8_t dynamic[];
  __shared__ uint64_t full[C::kStages], empty[C::kStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_base;
  __shared__ volatile int gave_up;
  __shared__ volatile uint32_t copied;  // stages so far: an epilogue waits for a tile's all

  const uint32_t ring = (smem_u32(dynamic) + 1023u) & ~1023u;
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0 : cluster_rank();
  static_assert(CG == 1 || SPLIT == 1, "a pair shares the tile, not its contraction");
  const int tiles = p.tiles_m * p.tiles_n * p.outputs;
  const int first = blockIdx.x / (CG * SPLIT), stride = gridDim.x / (CG * SPLIT);
  // the CTA's stages of the contraction: all, or its share of them
  const int all = p.k_blocks * p.phases, share = (all + SPLIT - 1) / SPLIT;
  const int begin = SPLIT == 1 ? 0 : min(all, (int)cluster_rank() * share);
  const int end = SPLIT == 1 ? all : min(all, begin + share);
  bool met = false;  // whether the warp is past the cluster's first barrier

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&acc_full[i], 1), mbar_init(&acc_empty[i], 8 * CG);
    gave_up = 0, copied = 0;
    for (int i = 0; i < 2; ++i) prefetch_map(&maps.a[i]), prefetch_map(&maps.b[i]);
  }
  if (warp == 1) tmem_alloc<CG>(&tmem_base, 2 * BN);
  tmem_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = tmem_base;
  pdl_begin();

  if (warp == 0) {
    // copies
    [&] {
      int stage = 0;
      uint32_t parity = 1, bars = smem_u32(&full[0]);
      if constexpr (CG == 2) bars = map_to_rank(bars, 0);
      for (int index = first; index < tiles; index += stride) {
        const Tile t = tile_at(p, index, 128 * CG, kCols);
        for (int s = begin; s < end; ++s) {
          if (!wait_or_leave(&empty[stage], parity, &gave_up)) return;
          const uint32_t bar = bars + 8 * stage;
          const int phase = MODE == kDx ? s / p.k_blocks : 0;
          const int k = (MODE == kDx ? s - phase * p.k_blocks : s) * kTileK;
          const uint32_t a = ring + stage * C::kStage, b = a + C::kABytes;
          const CUtensorMap* ma = &maps.a[MODE == kDw ? t.output : phase];
          const int row = t.m0 + (int)rank * 128;
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], C::kStage * CG);
            if constexpr (kAcrossA) {
              tma_load_tile<CG>(a, ma, row, k, bar);
              tma_load_tile<CG>(a + 8192, ma, row + 64, k, bar);
            } else {
              tma_load_tile<CG>(a, ma, k, row, bar);
            }
            if constexpr (kPairedWeights) {
              if constexpr (CG == 2) {
                tma_load_tile<CG>(b, &maps.b[rank], k, t.n0, bar);
              } else {
                tma_load_tile<CG>(b, &maps.b[0], k, t.n0, bar);
                tma_load_tile<CG>(b + C::kBBytes / 2, &maps.b[1], k, t.n0, bar);
              }
            } else {
              const CUtensorMap* mb = &maps.b[phase];
#pragma unroll
              for (int c = 0; c < BN / CG / 64; ++c)
                tma_load_tile<CG>(b + c * 8192, mb, t.n0 + (int)rank * (BN / CG) + 64 * c, k, bar);
            }
          }
          __syncwarp();
          if (lane == 0) copied = copied + 1;
          if (++stage == C::kStages) stage = 0, parity ^= 1;
        }
      }
    }();
  } else if (warp == 1 && rank == 0) {
    // products
    [&] {
      int stage = 0, acc = 0;
      uint32_t parity = 0, acc_parity = 1;
      for (int index = first; index < tiles; index += stride) {
        if (!wait_or_leave(&acc_empty[acc], acc_parity, &gave_up)) return;
        tmem_fence_after();
        for (int s = begin; s < end; ++s) {
          if (!wait_or_leave(&full[stage], parity, &gave_up)) return;
          tmem_fence_after();
          const uint32_t a = ring + stage * C::kStage, b = a + C::kABytes;
          const uint64_t da = operand(a, kAcrossA ? 8192 : 16), db = operand(b, kAcrossB ? 8192 : 16);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kTileK / 16; ++kk)  // 16 along the contraction: 32 bytes of a
              mma_tile<CG, 2>(tmem + acc * BN,        // swizzle row, or 16 rows (units of 16)
                              da + kk * (kAcrossA ? 128 : 2), db + kk * (kAcrossB ? 128 : 2),
                              kIdesc, s - begin + kk > 0);
            mma_commit<CG>(&empty[stage]);
          }
          __syncwarp();
          if (++stage == C::kStages) stage = 0, parity ^= 1;
        }
        if (elect_one()) mma_commit<CG>(&acc_full[acc]);
        __syncwarp();
        if (++acc == 2) acc = 0, acc_parity ^= 1;
      }
    }();
  } else if (warp >= 2) {
    // epilogue: warp w reads lanes 32 (w mod 4) on, a row of the tile each, and half the columns
    [&] {
      int acc = 0;
      uint32_t acc_parity = 0;
      constexpr int kHalf = kCols / 2, kChunk = 32;
      const int quarter = warp & 3, half = (warp - 2) >> 2;
      uint32_t release = smem_u32(&acc_empty[0]);
      if constexpr (CG == 2) release = map_to_rank(release, 0);
      uint8_t* ring_memory = dynamic + (ring - smem_u32(dynamic));
      uint8_t* piece = ring_memory + C::kStages * C::kStage + (warp - 2) * kPieceBytes;
      constexpr bool kScaled = std::is_same<T, __half>::value && MODE != kForward;
      float scale = 1.f;
      if constexpr (kScaled) scale = range_scale<MODE != kGradients>(p.bounds, lane);
      for (int index = first; index < tiles; index += stride) {
        const Tile t = tile_at(p, index, 128 * CG, kCols);
        const int row0 = t.m0 + (int)rank * 128 + quarter * 32;
        const uint32_t at = tmem + acc * BN + ((uint32_t)quarter << 21);
        // W columns of the output from the tile's column c: v, and u beside it for two weights;
        // dh: the gradients' share of `grad`, overwritten
        auto emit = [&](int c, auto& v, auto& u, auto& dh) {
          constexpr int W = sizeof(v) / 4;
          uint32_t packed[W / 2];
          const int col = t.n0 + c;
#pragma unroll
          for (int i = 0; i < W / 2; ++i) {
            const float a0 = __uint_as_float(v[2 * i]), a1 = __uint_as_float(v[2 * i + 1]);
            if constexpr (kPairedWeights) {
              float v0, v1, s0, s1;
              activate(p.act, a0, v0, s0);
              activate(p.act, a1, v1, s1);
              const float u0 = __uint_as_float(u[2 * i]), u1 = __uint_as_float(u[2 * i + 1]);
              if constexpr (MODE == kForward) {
                packed[i] = pack2<T>(v0 * u0, v1 * u1);
              } else {
                float2 g = unpack2<T>(dh[i]);
                if constexpr (kScaled) g.x *= scale, g.y *= scale;
                packed[i] = pack2<T>(g.x * u0 * s0, g.y * u1 * s1);
                dh[i] = pack2<T>(g.x * v0, g.y * v1);
              }
            } else {
              packed[i] = kScaled ? pack2<T>(a0 * scale, a1 * scale) : pack2<T>(a0, a1);
            }
          }
          const int o = MODE == kDw ? t.output : 0;
          store_rows<T, W>((T*)p.out[o], p.ld_out[o], piece, row0, lane, p.m, col, p.n, p.vec, packed);
          if constexpr (MODE == kGradients)
            store_rows<T, W>((T*)p.out[1], p.ld_out[1], piece, row0, lane, p.m, col, p.n, p.vec, dh);
        };
        auto load_grad = [&](int c, auto& dh) {
          if constexpr (MODE == kGradients)
            load_rows<T, sizeof(dh) / 2>((const T*)p.grad, p.ld_grad, piece, row0, lane, p.m, t.n0 + c,
                                         p.n, dh);
        };
        uint32_t dh[2][kChunk / 2];  // on their way while the products run
        if constexpr (SPLIT == 1 && MODE == kGradients) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (i * kChunk < kHalf) load_grad(half * kHalf + i * kChunk, dh[i]);
        }
        if (!wait_or_leave(&acc_full[acc], acc_parity, &gave_up, false, &copied)) return;
        tmem_fence_after();
        if constexpr (SPLIT == 1) {
#pragma unroll
          for (int i = 0; i < kHalf / kChunk; ++i) {
            const int c = half * kHalf + i * kChunk;
            if (t.n0 + c >= p.n) break;
            uint32_t v[32], u[32];
            tmem_load32(at + c, v);
            if constexpr (kPairedWeights) tmem_load32(at + BN / 2 + c, u);
            tmem_wait_loads();
            emit(c, v, u, dh[i & 1]);
          }
          __syncwarp();
        } else {
          // Every CTA of the cluster leaves its sums in its own ring, which its products are
          // done with, and adds up and emits a share of the columns, in the order of ranks.
          float* mine = (float*)ring_memory + quarter * BN * 32 + lane;
          const bool some = begin < end;
#pragma unroll 1
          for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32) {
            uint32_t v[32];
            tmem_load32(at + c, v);
            tmem_wait_loads();
#pragma unroll
            for (int i = 0; i < 32; ++i) mine[(c + i) * 32] = some ? __uint_as_float(v[i]) : 0.f;
          }
          __syncwarp();
          cluster_sync();
          met = true;
          // whole 16-byte chunks of the warp's columns, the last CTAs' shares smaller or empty
          constexpr int kShare = (kHalf / 8 + SPLIT - 1) / SPLIT * 8;
          constexpr int W = kShare % 32 == 0 ? 32 : kShare % 16 == 0 ? 16 : 8;
          const int from = (int)cluster_rank() * kShare;
          const uint32_t there = smem_u32(mine);
#pragma unroll 1
          for (int at = from; at < min(from + kShare, kHalf); at += W) {
            const int c = half * kHalf + at;
            uint32_t v[W], u[W];
            auto gather = [&](int c0, uint32_t(&x)[W]) {
              float sum[W];
#pragma unroll
              for (int i = 0; i < W; ++i) sum[i] = 0.f;
#pragma unroll
              for (int r = 0; r < SPLIT; ++r) {
                const uint32_t peer = map_to_rank(there, r) + c0 * 128;
#pragma unroll
                for (int i = 0; i < W; ++i) sum[i] += load_cluster(peer + i * 128);
              }
#pragma unroll
              for (int i = 0; i < W; ++i) x[i] = __float_as_uint(sum[i]);
            };
            gather(c, v);
            if constexpr (kPairedWeights) gather(BN / 2 + c, u);
            uint32_t dh[W / 2];
            load_grad(c, dh);
            emit(c, v, u, dh);
          }
        }
        tmem_fence_before();
        __syncwarp();
        if constexpr (CG == 2) mbar_arrive_cluster(release + 8 * acc, lane == 0);
        else mbar_arrive(&acc_empty[acc], lane == 0);
        if (++acc == 2) acc = 0, acc_parity ^= 1;
      }
    }();
  }

  __syncwarp();
  if constexpr (SPLIT > 1) {
    if (!met) cluster_sync();
    cluster_sync();  // no CTA leaves while another reads its sums
  }
  tmem_fence_before();
  __syncthreads();
  if (gave_up) drain();
  if constexpr (CG == 2) cluster_sync();
  tmem_fence_after();
  if (warp == 1) tmem_free<CG>(tmem, 2 * BN);
}

template <typename T, int MODE, int CG, int BN, int SPLIT>
cudaError_t launch_config(const GemmMaps& maps, const GemmParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n * p.outputs;
  if (tiles > 0x7fffff00 / SPLIT) return cudaErrorInvalidConfiguration;
  const int64_t grid =
      SPLIT > 1 ? tiles * SPLIT : std::min<int64_t>(tiles, multiprocessors() / CG) * CG;
  constexpr const char* kMode[] = {"gated", "gated gradients", "gated dx", "gated dw"};
  log_kernel("%s %s rows=%d cols=%d stages=%lld | tiles %dx%d split=%d", kMode[MODE],
             std::is_same<T, __half>::value ? "f16" : "bf16", p.m, p.n, (long long)p.k_blocks * p.phases,
             128 * CG, BN, SPLIT);
  return launch_cluster(gemm_kernel<T, MODE, CG, BN, SPLIT>, ready, (unsigned)grid, kThreads,
                        Config<CG, BN>::kSmem, CG * SPLIT, st, maps, p);
}

// How a product is cut: pairs of CTAs on 256 x 256 tiles, or single ones on 128 x 128 whose
// contraction a cluster of `split` shares out where the tiles leave multiprocessors idle.
struct Cut {
  bool wide;
  int split;
};

// A stage costs a CTA about the same either way (it moves 32 KB), so what counts is the stages
// that one CTA after the other goes through, waves of tiles times stages a tile; sharing out
// costs about as much as eight of them (measured: 1.7 to 2.5 us, at 0.2 to 0.3 us a stage).
Cut choose_cut(int64_t m, int64_t n, int outputs, int64_t stages, int most_split) {
  const int64_t sms = multiprocessors();
  const auto tiles = [&](int64_t size) { return ((m + size - 1) / size) * ((n + size - 1) / size) * outputs; };
  const int64_t wide = (tiles(256) + sms / 2 - 1) / (sms / 2) * stages, small = tiles(128);
  int64_t least = (small + sms - 1) / sms * stages;
  int split = 1;
  // (clusters of three and more do not fill every multiprocessor of a graphics cluster)
  for (int s : {2, 3, 4, 6, 8})
    if (s <= most_split && s * small <= (s > 2 ? sms * 7 / 8 : sms) && (stages + s - 1) / s + 8 < least)
      split = s, least = (stages + s - 1) / s + 8;
  return wide < least ? Cut{true, 1} : Cut{false, split};
}

template <typename T, int MODE>
cudaError_t launch_mode(Cut cut, const GemmMaps& maps, GemmParams p, cudaStream_t st) {
  constexpr int halves = MODE == kForward || MODE == kGradients ? 2 : 1;
  const int rows = cut.wide ? 256 : 128, cols = (cut.wide ? 256 : 128) / halves;
  p.tiles_m = (p.m + rows - 1) / rows;
  p.tiles_n = (p.n + cols - 1) / cols;
  if (cut.wide) return launch_config<T, MODE, 2, 256, 1>(maps, p, st);
  if constexpr (halves == 1) {
    if (cut.split == 8) return launch_config<T, MODE, 1, 128, 8>(maps, p, st);
    if (cut.split == 6) return launch_config<T, MODE, 1, 128, 6>(maps, p, st);
  }
  if (cut.split == 4) return launch_config<T, MODE, 1, 128, 4>(maps, p, st);
  if (cut.split == 3) return launch_config<T, MODE, 1, 128, 3>(maps, p, st);
  if (cut.split == 2) return launch_config<T, MODE, 1, 128, 2>(maps, p, st);
  return launch_config<T, MODE, 1, 128, 1>(maps, p, st);
}

struct Operand {
  CMat mat;
  int64_t rows, cols;
  int box_rows;
};

template <typename T>
bool make_map(CUtensorMap* map, const Operand& o) {
  return swizzled_map(map, o.mat.p, 2,
                      std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      o.rows, o.cols, o.mat.ld, o.box_rows);
}

bool vector_rows(Mat m) { return ((uintptr_t)m.p & 15u) == 0 && m.ld % 8 == 0; }

template <typename T, int MODE>
cudaError_t run_paired(CMat x, CMat w_gate, CMat w_up, GemmParams p, int d, cudaStream_t st) {
  p.k_blocks = (d + kTileK - 1) / kTileK;
  p.phases = p.outputs = 1;
  // (both weights' columns count; an eighth of them would be narrower than a store)
  const Cut cut = choose_cut(p.m, 2 * (int64_t)p.n, 1, p.k_blocks, 4);
  const int box = cut.wide ? 128 : 64;  // lines of each weight in a stage
  GemmMaps maps;
  if (!make_map<T>(&maps.a[0], {x, p.m, d, 128}) ||
      !make_map<T>(&maps.b[0], {w_gate, p.n, d, box}) ||
      !make_map<T>(&maps.b[1], {w_up, p.n, d, box}))
    return cudaErrorInvalidValue;
  maps.a[1] = maps.a[0];
  return launch_mode<T, MODE>(cut, maps, p, st);
}

template <typename T>
cudaError_t run_dx(CMat dg, CMat du, CMat w_gate, CMat w_up, Mat dx, Bounds bounds, int m, int f,
                   int d, cudaStream_t st) {
  GemmMaps maps;
  if (!make_map<T>(&maps.a[0], {dg, m, f, 128}) || !make_map<T>(&maps.a[1], {du, m, f, 128}) ||
      !make_map<T>(&maps.b[0], {w_gate, f, d, kTileK}) ||
      !make_map<T>(&maps.b[1], {w_up, f, d, kTileK}))
    return cudaErrorInvalidValue;
  GemmParams p{};
  p.m = m, p.n = d, p.k_blocks = (f + kTileK - 1) / kTileK, p.phases = 2, p.outputs = 1;
  p.out[0] = dx.p, p.ld_out[0] = dx.ld, p.vec = vector_rows(dx), p.bounds = bounds;
  return launch_mode<T, kDx>(choose_cut(m, d, 1, 2 * (int64_t)p.k_blocks, 8), maps, p, st);
}

template <typename T>
cudaError_t run_dw(CMat dg, CMat du, CMat x, Mat dw_gate, Mat dw_up, Bounds bounds, int m, int f,
                   int d, cudaStream_t st) {
  GemmMaps maps;
  if (!make_map<T>(&maps.a[0], {dg, m, f, kTileK}) || !make_map<T>(&maps.a[1], {du, m, f, kTileK}) ||
      !make_map<T>(&maps.b[0], {x, m, d, kTileK}))
    return cudaErrorInvalidValue;
  maps.b[1] = maps.b[0];
  GemmParams p{};
  p.m = f, p.n = d, p.k_blocks = (m + kTileK - 1) / kTileK, p.phases = 1, p.outputs = 2;
  p.out[0] = dw_gate.p, p.ld_out[0] = dw_gate.ld;
  p.out[1] = dw_up.p, p.ld_out[1] = dw_up.ld;
  p.vec = vector_rows(dw_gate) && vector_rows(dw_up), p.bounds = bounds;
  return launch_mode<T, kDw>(choose_cut(f, d, 2, p.k_blocks, 8), maps, p, st);
}

}  // namespace

cudaError_t launch_gated(CMat x, CMat w_gate, CMat w_up, Mat h, int type, int act, int m, int f,
                         int d, cudaStream_t st) {
  // Straight from global memory up to 8 tokens, and further where the weights are few (both
  // ways measured, us: 16 tokens by 2 x 4096 x 4096 14.8 against 15.9 here, by 2 x 4096 x 8192
  // 27.1 against 24.0; 32 tokens by 2 x 2048 x 2048 8.7 against 8.8, by 2 x 2816 x 2816 15.0
  // against 11.0).
  const int64_t weights = 2 * (int64_t)f * d;
  if (m <= 8 || (m <= 16 && weights <= 48 << 20) || (m <= kMostTokens && weights <= 8 << 20))
    return launch_gated_tokens(x, w_gate, w_up, h, type, act, m, f, d, st);
  GemmParams p{};
  p.m = m, p.n = f, p.act = act;
  p.out[0] = h.p, p.ld_out[0] = h.ld, p.vec = vector_rows(h);
  return type == FWT_BF16 ? run_paired<__nv_bfloat16, kForward>(x, w_gate, w_up, p, d, st)
                          : run_paired<__half, kForward>(x, w_gate, w_up, p, d, st);
}

cudaError_t launch_gated_bounds(CMat grad, CMat x, CMat w_gate, CMat w_up, Bounds& bounds, int m,
                                int f, int d, cudaStream_t st) {
  const int64_t rows = (int64_t)m + f, most = std::min(kMostBounds, 3 * multiprocessors());
  bounds.parts = (int)std::min<int64_t>(most, (rows + kBoundWarps - 1) / kBoundWarps);
  const BoundParams p{grad, x, w_gate, w_up, (float2*)bounds.pairs, m, f, d};
  log_kernel("gated bounds f16 m=%d f=%d d=%d", m, f, d);
  return launch_overlapped(bounds_kernel, (unsigned)bounds.parts, kBoundWarps * 32, 0, 1, st, p);
}

cudaError_t launch_gated_gradients(CMat grad, CMat x, CMat w_gate, CMat w_up, Mat dg, Mat du,
                                   Bounds bounds, int type, int act, int m, int f, int d,
                                   cudaStream_t st) {
  GemmParams p{};
  p.bounds = bounds;
  p.m = m, p.n = f, p.act = act;
  p.grad = grad.p, p.ld_grad = grad.ld;
  p.out[0] = dg.p, p.ld_out[0] = dg.ld, p.out[1] = du.p, p.ld_out[1] = du.ld;
  p.vec = 1;  // the workspace's rows are
  return type == FWT_BF16 ? run_paired<__nv_bfloat16, kGradients>(x, w_gate, w_up, p, d, st)
                          : run_paired<__half, kGradients>(x, w_gate, w_up, p, d, st);
}

cudaError_t launch_gated_dx(CMat dg, CMat du, CMat w_gate, CMat w_up, Mat dx, Bounds bounds,
                            int type, int m, int f, int d, cudaStream_t st) {
  return type == FWT_BF16 ? run_dx<__nv_bfloat16>(dg, du, w_gate, w_up, dx, bounds, m, f, d, st)
                          : run_dx<__half>(dg, du, w_gate, w_up, dx, bounds, m, f, d, st);
}

cudaError_t launch_gated_dw(CMat dg, CMat du, CMat x, Mat dw_gate, Mat dw_up, Bounds bounds,
                            int type, int m, int f, int d, cudaStream_t st) {
  return type == FWT_BF16 ? run_dw<__nv_bfloat16>(dg, du, x, dw_gate, dw_up, bounds, m, f, d, st)
                          : run_dw<__half>(dg, du, x, dw_gate, dw_up, bounds, m, f, d, st);
}

// Reads and clears this translation unit's device error word (synchronising).
cudaError_t read_device_error_gated(unsigned int* out) {
  const unsigned int zero = 0;
  cudaError_t err = cudaMemcpyFromSymbol(out, g_device_error, sizeof(unsigned int));
  if (err == cudaSuccess && *out)
    err = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(unsigned int));
  return err;
}

}  // namespace ff
}  // namespace fwt
