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
// MN-major, so nothing is transposed in memory), one thread issues the products, and four
// warps turn finished accumulators into output while the next tile's products run in the
// other half of tensor memory.  Large products pair two CTAs on a tile of 256 x 256: each
// loads half of both operands, which halves the shared-memory traffic of the second.
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
};

struct GemmMaps {
  CUtensorMap a[2], b[2];
};

constexpr int kTileK = 64;  // elements of the contraction in a stage: one swizzle row
constexpr int kRingBytes = 196608;
constexpr int kThreads = 192;

// CG: CTAs that share a tile.  BN: columns of its accumulator.  Each CTA holds 128 rows of
// the first operand and BN / CG lines of the second.
template <int CG, int BN>
struct Config {
  static constexpr int kABytes = 128 * 128, kBBytes = BN / CG * 128;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = kRingBytes / kStage;
  static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
};

struct Tile {
  int m0, n0, output;
};

// Tiles in groups of 8 rows of tiles, so that those in flight together share operands in L2.
__device__ __forceinline__ Tile tile_at(const GemmParams& p, int index, int rows, int cols) {
  const int area = p.tiles_m * p.tiles_n;
  Tile t;
  t.output = index / area;
  index -= t.output * area;
  const int group = index / (8 * p.tiles_n);
  const int height = min(8, p.tiles_m - group * 8);
  index -= group * 8 * p.tiles_n;
  t.m0 = (group * 8 + index % height) * rows;
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

// 32 values of a row to columns [col, col + 32) of `out`, those below n.
template <typename T>
__device__ __forceinline__ void store32(T* row, int col, int n, bool vec, const uint32_t (&v)[16]) {
  if (vec && col + 32 <= n) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *(uint4*)(row + col + 8 * i) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (col + i < n)
      *(unsigned short*)(row + col + i) = (unsigned short)(v[i / 2] >> (16 * (i & 1)));
}
template <typename T>
__device__ __forceinline__ void load32(const T* row, int col, int n, uint32_t (&v)[16]) {
  if (col + 32 <= n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 q = __ldg((const uint4*)(row + col + 8 * i));
      v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t lo = col + 2 * i < n ? __ldg((const unsigned short*)row + col + 2 * i) : 0;
    const uint32_t hi = col + 2 * i + 1 < n ? __ldg((const unsigned short*)row + col + 2 * i + 1) : 0;
    v[i] = lo | (hi << 16);
  }
}

template <typename T, int MODE, int CG, int BN>
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

  const uint32_t ring = (smem_u32(dynamic) + 1023u) & ~1023u;
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0 : cluster_rank();
  const int steps = p.k_blocks * p.phases;
  const int tiles = p.tiles_m * p.tiles_n * p.outputs;
  const int first = blockIdx.x / CG, stride = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&acc_full[i], 1), mbar_init(&acc_empty[i], 4 * CG);
    gave_up = 0;
    for (int i = 0; i < 2; ++i) prefetch_map(&maps.a[i]), prefetch_map(&maps.b[i]);
  }
  if (warp == 1) tmem_alloc<CG>(&tmem_base, 2 * BN);
  tmem_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = tmem_base;

  if (warp == 0) {
    // copies
    [&] {
      int stage = 0;
      uint32_t parity = 1, bars = smem_u32(&full[0]);
      if constexpr (CG == 2) bars = map_to_rank(bars, 0);
      for (int index = first; index < tiles; index += stride) {
        const Tile t = tile_at(p, index, 128 * CG, kCols);
        for (int s = 0; s < steps; ++s) {
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
        for (int s = 0; s < steps; ++s) {
          if (!wait_or_leave(&full[stage], parity, &gave_up)) return;
          tmem_fence_after();
          const uint32_t a = ring + stage * C::kStage, b = a + C::kABytes;
          const uint64_t da = operand(a, kAcrossA ? 8192 : 16), db = operand(b, kAcrossB ? 8192 : 16);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kTileK / 16; ++kk)  // 16 along the contraction: 32 bytes of a
              mma_tile<CG, 2>(tmem + acc * BN,        // swizzle row, or 16 rows (units of 16)
                              da + kk * (kAcrossA ? 128 : 2), db + kk * (kAcrossB ? 128 : 2),
                              kIdesc, s + kk > 0);
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
    // epilogue: warp w reads lanes 32 (w mod 4) on, a row of the tile each
    [&] {
      int acc = 0;
      uint32_t acc_parity = 0;
      const int quarter = warp & 3;
      uint32_t release[2];
      for (int i = 0; i < 2; ++i)
        release[i] = CG == 2 ? map_to_rank(smem_u32(&acc_empty[i]), 0) : smem_u32(&acc_empty[i]);
      for (int index = first; index < tiles; index += stride) {
        const Tile t = tile_at(p, index, 128 * CG, kCols);
        const int row = t.m0 + (int)rank * 128 + quarter * 32 + lane;
        const bool live = row < p.m;
        const uint32_t at = tmem + acc * BN + ((uint32_t)quarter << 21);
        if (!wait_or_leave(&acc_full[acc], acc_parity, &gave_up)) return;
        tmem_fence_after();
        T* out0 = (T*)p.out[MODE == kDw ? t.output : 0] +
                  (int64_t)row * p.ld_out[MODE == kDw ? t.output : 0];
#pragma unroll 1
        for (int c = 0; c < kCols; c += 32) {
          const int col = t.n0 + c;
          if (col >= p.n) break;
          uint32_t v[32], packed[16];
          tmem_load32(at + c, v);
          if constexpr (kPairedWeights) {
            uint32_t u[32], second[16];
            tmem_load32(at + BN / 2 + c, u);
            if constexpr (MODE == kGradients) {
              if (live) load32((const T*)p.grad + (int64_t)row * p.ld_grad, col, p.n, second);
              __syncwarp();
            }
            tmem_wait_loads();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float v0, v1, s0, s1;
              activate(p.act, __uint_as_float(v[2 * i]), v0, s0);
              activate(p.act, __uint_as_float(v[2 * i + 1]), v1, s1);
              const float u0 = __uint_as_float(u[2 * i]), u1 = __uint_as_float(u[2 * i + 1]);
              if constexpr (MODE == kForward) {
                packed[i] = pack2<T>(v0 * u0, v1 * u1);
              } else {
                const float2 dh = unpack2<T>(second[i]);
                packed[i] = pack2<T>(dh.x * u0 * s0, dh.y * u1 * s1);
                second[i] = pack2<T>(dh.x * v0, dh.y * v1);
              }
            }
            if constexpr (MODE == kGradients) {
              if (live) store32((T*)p.out[1] + (int64_t)row * p.ld_out[1], col, p.n, p.vec, second);
            }
          } else {
            tmem_wait_loads();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              packed[i] = pack2<T>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
          }
          if (live) store32(out0, col, p.n, p.vec, packed);
          __syncwarp();
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2) mbar_arrive_cluster(release[acc]);
          else mbar_arrive(&acc_empty[acc]);
        }
        if (++acc == 2) acc = 0, acc_parity ^= 1;
      }
    }();
  }

  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (gave_up) drain();
  if constexpr (CG == 2) cluster_sync();
  tmem_fence_after();
  if (warp == 1) tmem_free<CG>(tmem, 2 * BN);
}

template <typename T, int MODE, int CG, int BN>
cudaError_t launch_config(const GemmMaps& maps, GemmParams p, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  constexpr int cols = MODE == kForward || MODE == kGradients ? BN / 2 : BN;
  p.tiles_m = (p.m + 128 * CG - 1) / (128 * CG);
  p.tiles_n = (p.n + cols - 1) / cols;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n * p.outputs;
  if (tiles > 0x7fffff00) return cudaErrorInvalidConfiguration;
  const int64_t grid = std::min<int64_t>(tiles, multiprocessors() / CG) * CG;
  return launch_cluster(gemm_kernel<T, MODE, CG, BN>, ready, (unsigned)grid, kThreads,
                        Config<CG, BN>::kSmem, CG, st, maps, p);
}

// Whether pairs of CTAs on 256 x 256 tiles fill the device: else smaller tiles.
bool wide_tiles(int m, int n, int outputs) {
  return (int64_t)((m + 255) / 256) * ((n + 255) / 256) * outputs * 2 >= multiprocessors();
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
  const bool wide = wide_tiles(p.m, 2 * p.n, 1);
  const int box = wide ? 128 : 64;  // lines of each weight in a stage
  GemmMaps maps;
  if (!make_map<T>(&maps.a[0], {x, p.m, d, 128}) ||
      !make_map<T>(&maps.b[0], {w_gate, p.n, d, box}) ||
      !make_map<T>(&maps.b[1], {w_up, p.n, d, box}))
    return cudaErrorInvalidValue;
  maps.a[1] = maps.a[0];
  p.k_blocks = (d + kTileK - 1) / kTileK;
  p.phases = p.outputs = 1;
  return wide ? launch_config<T, MODE, 2, 256>(maps, p, st)
              : launch_config<T, MODE, 1, 128>(maps, p, st);
}

template <typename T>
cudaError_t run_dx(CMat dg, CMat du, CMat w_gate, CMat w_up, Mat dx, int m, int f, int d,
                   cudaStream_t st) {
  GemmMaps maps;
  if (!make_map<T>(&maps.a[0], {dg, m, f, 128}) || !make_map<T>(&maps.a[1], {du, m, f, 128}) ||
      !make_map<T>(&maps.b[0], {w_gate, f, d, kTileK}) ||
      !make_map<T>(&maps.b[1], {w_up, f, d, kTileK}))
    return cudaErrorInvalidValue;
  GemmParams p{};
  p.m = m, p.n = d, p.k_blocks = (f + kTileK - 1) / kTileK, p.phases = 2, p.outputs = 1;
  p.out[0] = dx.p, p.ld_out[0] = dx.ld, p.vec = vector_rows(dx);
  return wide_tiles(m, d, 1) ? launch_config<T, kDx, 2, 256>(maps, p, st)
                             : launch_config<T, kDx, 1, 128>(maps, p, st);
}

template <typename T>
cudaError_t run_dw(CMat dg, CMat du, CMat x, Mat dw_gate, Mat dw_up, int m, int f, int d,
                   cudaStream_t st) {
  GemmMaps maps;
  if (!make_map<T>(&maps.a[0], {dg, m, f, kTileK}) || !make_map<T>(&maps.a[1], {du, m, f, kTileK}) ||
      !make_map<T>(&maps.b[0], {x, m, d, kTileK}))
    return cudaErrorInvalidValue;
  maps.b[1] = maps.b[0];
  GemmParams p{};
  p.m = f, p.n = d, p.k_blocks = (m + kTileK - 1) / kTileK, p.phases = 1, p.outputs = 2;
  p.out[0] = dw_gate.p, p.ld_out[0] = dw_gate.ld;
  p.out[1] = dw_up.p, p.ld_out[1] = dw_up.ld;
  p.vec = vector_rows(dw_gate) && vector_rows(dw_up);
  return wide_tiles(f, d, 2) ? launch_config<T, kDw, 2, 256>(maps, p, st)
                             : launch_config<T, kDw, 1, 128>(maps, p, st);
}

}  // namespace

cudaError_t launch_gated(CMat x, CMat w_gate, CMat w_up, Mat h, int type, int act, int m, int f,
                         int d, cudaStream_t st) {
  if (m <= kMostTokens) return launch_gated_tokens(x, w_gate, w_up, h, type, act, m, f, d, st);
  GemmParams p{};
  p.m = m, p.n = f, p.act = act;
  p.out[0] = h.p, p.ld_out[0] = h.ld, p.vec = vector_rows(h);
  return type == FWT_BF16 ? run_paired<__nv_bfloat16, kForward>(x, w_gate, w_up, p, d, st)
                          : run_paired<__half, kForward>(x, w_gate, w_up, p, d, st);
}

cudaError_t launch_gated_gradients(CMat grad, CMat x, CMat w_gate, CMat w_up, Mat dg, Mat du,
                                   int type, int act, int m, int f, int d, cudaStream_t st) {
  GemmParams p{};
  p.m = m, p.n = f, p.act = act;
  p.grad = grad.p, p.ld_grad = grad.ld;
  p.out[0] = dg.p, p.ld_out[0] = dg.ld, p.out[1] = du.p, p.ld_out[1] = du.ld;
  p.vec = 1;  // the workspace's rows are
  return type == FWT_BF16 ? run_paired<__nv_bfloat16, kGradients>(x, w_gate, w_up, p, d, st)
                          : run_paired<__half, kGradients>(x, w_gate, w_up, p, d, st);
}

cudaError_t launch_gated_dx(CMat dg, CMat du, CMat w_gate, CMat w_up, Mat dx, int type, int m,
                            int f, int d, cudaStream_t st) {
  return type == FWT_BF16 ? run_dx<__nv_bfloat16>(dg, du, w_gate, w_up, dx, m, f, d, st)
                          : run_dx<__half>(dg, du, w_gate, w_up, dx, m, f, d, st);
}

cudaError_t launch_gated_dw(CMat dg, CMat du, CMat x, Mat dw_gate, Mat dw_up, int type, int m,
                            int f, int d, cudaStream_t st) {
  return type == FWT_BF16 ? run_dw<__nv_bfloat16>(dg, du, x, dw_gate, dw_up, m, f, d, st)
                          : run_dw<__half>(dg, du, x, dw_gate, dw_up, m, f, d, st);
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
