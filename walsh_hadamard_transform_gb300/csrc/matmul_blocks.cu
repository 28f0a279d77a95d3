// Product of two 8-bit operands with a scale for each block of 128 along the contraction.
//
// The tensor cores sum one block's products (128 along the contraction, four instructions)
// into tensor memory; the scales are fp32 and differ from row to row, so each block's sums
// are then taken into registers and added there, times both scales, in fp32:
//
//     acc[i, j] += part_t[i, j] * (a_scale[i, t] * b_scale[j, t])
//
// CTAs are persistent, one an SM.  One warp fills a ring of operand stages by TMA, one thread
// issues the products of block after block into a ring of accumulator slots, and eight warps
// read slot after slot, half of the tile's columns each of two to a quarter of its rows: a
// tile of 256 columns costs them 128 values a thread and block, packed two to a multiply-add.
// Large products pair two CTAs on a tile of 256 x 256.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "feed_forward.cuh"
#include "ff_host.cuh"
#include "fwt.h"
#include "tcgen05.cuh"

namespace fwt {
namespace ff {
namespace {

constexpr int kBlock = 128;  // elements of the contraction that share a scale: one stage
constexpr int kRingBytes = 196608;
constexpr int kThreads = 384;  // a warp each for copies and products (of four), eight for the sums
// Registers of a thread: 168 at launch (384 threads), moved from the first warpgroup to the
// two that hold 128 sums a thread: 128 * 72 + 256 * 216 = 384 * 168.
constexpr int kLeanRegisters = 72, kSumRegisters = 216;
static_assert(128 * kLeanRegisters + 256 * kSumRegisters == 384 * 168, "the launch's registers");

struct BlocksParams {
  const float *a_scale, *b_scale;
  int64_t ld_as, ld_bs;
  void* c;
  int64_t ld_c;
  int c_type;
  int m, n, blocks;
  int tiles_m, tiles_n;
  int vec_c, vec_as, vec_bs;  // rows start on 16-byte boundaries
};

struct BlocksMaps {
  CUtensorMap a, b;
};

template <int CG, int BN>
struct Config {
  static constexpr int kABytes = 128 * 128, kBBytes = BN / CG * 128;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = kRingBytes / kStage;
  static constexpr int kSlots = 512 / BN > 4 ? 4 : 512 / BN;
  static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
};

// The scales of one line, read four blocks at a time, one group ahead.
struct Scales {
  const float* row;  // null: a line outside the matrix
  int blocks;
  bool vec;
  float4 now, next;

  __device__ __forceinline__ float4 group(int t) const {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!row || t >= blocks) return v;
    if (vec && t + 4 <= blocks) return __ldg((const float4*)(row + t));
    v.x = __ldg(row + t);
    if (t + 1 < blocks) v.y = __ldg(row + t + 1);
    if (t + 2 < blocks) v.z = __ldg(row + t + 2);
    if (t + 3 < blocks) v.w = __ldg(row + t + 3);
    return v;
  }
  __device__ __forceinline__ void start(const float* r, int n, bool v) {
    row = r, blocks = n, vec = v;
    next = group(0);
  }
  // The scale of block t; called for t = 0, 1, 2, ...
  __device__ __forceinline__ float at(int t) {
    if ((t & 3) == 0) now = next, next = group(t + 4);
    return (t & 2) ? ((t & 1) ? now.w : now.z) : ((t & 1) ? now.y : now.x);
  }
};

template <typename C>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same<C, __half>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    return *(const uint32_t*)&h;
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *(const uint32_t*)&h;
  }
}

// N values of a row of C to columns [col, col + N), those below n.
template <int N>
__device__ __forceinline__ void store_row(const BlocksParams& p, int row, int col,
                                          const float (&acc)[N]) {
  const bool vec = p.vec_c && col + N <= p.n;
  if (p.c_type == FWT_F32) {
    float* c = (float*)p.c + (int64_t)row * p.ld_c + col;
    if (vec) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *(float4*)(c + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (col + i < p.n) c[i] = acc[i];
    }
    return;
  }
  unsigned short* c = (unsigned short*)p.c + (int64_t)row * p.ld_c + col;
  const bool half = p.c_type == FWT_F16;
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    uint32_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = half ? pack2<__half>(acc[i + 2 * j], acc[i + 2 * j + 1])
                  : pack2<__nv_bfloat16>(acc[i + 2 * j], acc[i + 2 * j + 1]);
    if (vec) {
      *(uint4*)(c + i) = make_uint4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + i + j < p.n) c[i + j] = (unsigned short)(v[j / 2] >> (16 * (j & 1)));
    }
  }
}

template <int CG, int BN, int LINES>
__global__ void __launch_bounds__(kThreads, 1)
    blocks_kernel(const __grid_constant__ BlocksMaps maps, const BlocksParams p) {
  using C = Config<CG, BN>;
  constexpr uint32_t kIdesc = instruction(0, false, false, 128 * CG, BN);
  constexpr int kHalf = BN / 2;  // columns of a warp

  extern __shared__ uint8_t dynamic[];
  __shared__ uint64_t full[C::kStages], empty[C::kStages], slot_full[C::kSlots],
      slot_empty[C::kSlots], scales_ready[2];
  __shared__ uint32_t tmem_base;
  __shared__ volatile int gave_up;
  __shared__ __align__(16) float b_scales[2][LINES == 1 ? BN : 4];

  const uint32_t ring = (smem_u32(dynamic) + 1023u) & ~1023u;
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0 : cluster_rank();
  const int tiles = p.tiles_m * p.tiles_n;
  const int first = blockIdx.x / CG, stride = gridDim.x / CG;

  // Tiles in groups of 8 rows of tiles, so that those in flight together share operands in L2.
  auto place = [&](int index, int& m0, int& n0) {
    const int group = index / (8 * p.tiles_n);
    const int height = min(8, p.tiles_m - group * 8);
    index -= group * 8 * p.tiles_n;
    m0 = (group * 8 + index % height) * (128 * CG);
    n0 = index / height * BN;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < C::kSlots; ++i) mbar_init(&slot_full[i], 1), mbar_init(&slot_empty[i], 8 * CG);
    for (int i = 0; i < 2; ++i) mbar_init(&scales_ready[i], 8);
    gave_up = 0;
    prefetch_map(&maps.a), prefetch_map(&maps.b);
  }
  if (warp == 1) tmem_alloc<CG>(&tmem_base, C::kSlots * BN);
  tmem_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = tmem_base;

  if (warp < 4) {
    if constexpr (BN == 256)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLeanRegisters));
    if (warp == 0) {
      // copies
      [&] {
        int stage = 0;
        uint32_t parity = 1, bars = smem_u32(&full[0]);
        if constexpr (CG == 2) bars = map_to_rank(bars, 0);
        for (int index = first; index < tiles; index += stride) {
          int m0, n0;
          place(index, m0, n0);
          for (int t = 0; t < p.blocks; ++t) {
            if (!wait_or_leave(&empty[stage], parity, &gave_up)) return;
            const uint32_t a = ring + stage * C::kStage;
            const uint32_t bar = bars + 8 * stage;
            if (elect_one()) {
              if (rank == 0) mbar_arrive_expect_tx(&full[stage], C::kStage * CG);
              tma_load_tile<CG>(a, &maps.a, t * kBlock, m0 + (int)rank * 128, bar);
              tma_load_tile<CG>(a + C::kABytes, &maps.b, t * kBlock, n0 + (int)rank * (BN / CG), bar);
            }
            __syncwarp();
            if (++stage == C::kStages) stage = 0, parity ^= 1;
          }
        }
      }();
    } else if (warp == 1 && rank == 0) {
      // products
      [&] {
        int stage = 0, slot = 0;
        uint32_t parity = 0, slot_parity = 1;
        for (int index = first; index < tiles; index += stride) {
          for (int t = 0; t < p.blocks; ++t) {
            if (!wait_or_leave(&slot_empty[slot], slot_parity, &gave_up)) return;
            if (!wait_or_leave(&full[stage], parity, &gave_up)) return;
            tmem_fence_after();
            const uint32_t a = ring + stage * C::kStage, b = a + C::kABytes;
            const uint64_t da = operand(a, 16), db = operand(b, 16);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kBlock / 32; ++kk)  // 32 bytes of a swizzle row each
                mma_tile<CG, 1>(tmem + slot * BN, da + 2 * kk, db + 2 * kk, kIdesc, kk > 0);
              mma_commit<CG>(&empty[stage]);
              mma_commit<CG>(&slot_full[slot]);
            }
            __syncwarp();
            if (++stage == C::kStages) stage = 0, parity ^= 1;
            if (++slot == C::kSlots) slot = 0, slot_parity ^= 1;
          }
        }
      }();
    }
  } else {
    if constexpr (BN == 256)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegisters));
    // sums: warp w reads lanes 32 (w mod 4) on, a row of the tile each, and half its columns
    [&] {
      int slot = 0, buffer = 1;
      uint32_t slot_parity = 0, ready_parity = 0;
      const int quarter = warp & 3, half = (warp - 4) >> 2;
      const int thread = threadIdx.x - 128;
      uint32_t release = smem_u32(&slot_empty[0]);
      if constexpr (CG == 2) release = map_to_rank(release, 0);
      for (int index = first; index < tiles; index += stride) {
        int m0, n0;
        place(index, m0, n0);
        const int row = m0 + (int)rank * 128 + quarter * 32 + lane;
        const int col = n0 + half * kHalf;
        Scales sa, sb;
        sa.start(row < p.m ? p.a_scale + (int64_t)row * p.ld_as : nullptr, p.blocks, p.vec_as);
        if constexpr (LINES == 128)
          sb.start(col < p.n ? p.b_scale + (int64_t)(col / 128) * p.ld_bs : nullptr, p.blocks, p.vec_bs);
        else
          sb.start(thread < BN && n0 + thread < p.n ? p.b_scale + (int64_t)(n0 + thread) * p.ld_bs
                                                    : nullptr, p.blocks, p.vec_bs);
        float acc[kHalf];
#pragma unroll
        for (int i = 0; i < kHalf; ++i) acc[i] = 0.f;
        for (int t = 0; t < p.blocks; ++t) {
          float s = sa.at(t);
          buffer ^= 1;
          const float sbt = sb.at(t);
          if constexpr (LINES == 128) {
            s *= sbt;
          } else {
            if (thread < BN) b_scales[buffer][thread] = sbt;
            // a warp that is here for t + 2 has seen every warp arrive for t + 1, done with t
            __syncwarp();
            if (lane == 0) mbar_arrive(&scales_ready[buffer]);
            if (!wait_or_leave(&scales_ready[buffer], ready_parity, &gave_up)) return;
            if (buffer) ready_parity ^= 1;
          }
          if (!wait_or_leave(&slot_full[slot], slot_parity, &gave_up)) return;
          tmem_fence_after();
          const uint32_t at = tmem + slot * BN + half * kHalf + ((uint32_t)quarter << 21);
          uint32_t v[2][16];
          tmem_load16(at, v[0]);
#pragma unroll
          for (int c = 0; c < kHalf; c += 16) {
            tmem_wait_loads();
            if (c + 16 < kHalf) tmem_load16(at + c + 16, v[(c / 16 + 1) & 1]);
            const uint32_t(&x)[16] = v[(c / 16) & 1];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              float4 f = make_float4(s, s, s, s);
              if constexpr (LINES == 1) {
                f = *(const float4*)&b_scales[buffer][half * kHalf + c + i];
                f.x *= s, f.y *= s, f.z *= s, f.w *= s;
              }
              float* sum = &acc[c + i];
              sum[0] = fmaf(__uint_as_float(x[i]), f.x, sum[0]);
              sum[1] = fmaf(__uint_as_float(x[i + 1]), f.y, sum[1]);
              sum[2] = fmaf(__uint_as_float(x[i + 2]), f.z, sum[2]);
              sum[3] = fmaf(__uint_as_float(x[i + 3]), f.w, sum[3]);
            }
          }
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (CG == 2) mbar_arrive_cluster(release + 8 * slot);
            else mbar_arrive(&slot_empty[slot]);
          }
          if (++slot == C::kSlots) slot = 0, slot_parity ^= 1;
        }
        if (row < p.m && col < p.n) store_row<kHalf>(p, row, col, acc);
        __syncwarp();
      }
    }();
  }

  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (gave_up) drain();
  if constexpr (CG == 2) cluster_sync();
  tmem_fence_after();
  if (warp == 1) tmem_free<CG>(tmem, C::kSlots * BN);
}

template <int CG, int BN, int LINES>
cudaError_t launch_config(const BlocksMaps& maps, BlocksParams p, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  p.tiles_m = (p.m + 128 * CG - 1) / (128 * CG);
  p.tiles_n = (p.n + BN - 1) / BN;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles > 0x7fffff00) return cudaErrorInvalidConfiguration;
  const int64_t grid = std::min<int64_t>(tiles, multiprocessors() / CG) * CG;
  return launch_cluster(blocks_kernel<CG, BN, LINES>, ready, (unsigned)grid, kThreads,
                        Config<CG, BN>::kSmem, CG, st, maps, p);
}

template <int CG, int BN>
cudaError_t run(CMat a, CMat b, int b_lines, const BlocksParams& p, int k, cudaStream_t st) {
  BlocksMaps maps;
  if (!swizzled_map(&maps.a, a.p, 1, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.m, k, a.ld, 128) ||
      !swizzled_map(&maps.b, b.p, 1, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.n, k, b.ld, BN / CG))
    return cudaErrorInvalidValue;
  return b_lines == 1 ? launch_config<CG, BN, 1>(maps, p, st)
                      : launch_config<CG, BN, 128>(maps, p, st);
}

bool vector_rows(const void* p, int64_t ld_bytes) {
  return ((uintptr_t)p & 15u) == 0 && ld_bytes % 16 == 0;
}

}  // namespace

cudaError_t launch_matmul_blocks(CMat a, CMat a_scale, CMat b, CMat b_scale, int b_lines, Mat c,
                                 int c_type, int m, int n, int k, cudaStream_t st) {
  if (m <= kMostTokens)
    return launch_matmul_tokens(a, a_scale, b, b_scale, b_lines, c, c_type, m, n, k, st);
  BlocksParams p{};
  p.a_scale = (const float*)a_scale.p, p.ld_as = a_scale.ld;
  p.b_scale = (const float*)b_scale.p, p.ld_bs = b_scale.ld;
  p.c = c.p, p.ld_c = c.ld, p.c_type = c_type;
  p.m = m, p.n = n, p.blocks = (int)(((int64_t)k + kBlock - 1) / kBlock);
  p.vec_c = vector_rows(c.p, c.ld * (c_type == FWT_F32 ? 4 : 2));
  p.vec_as = vector_rows(a_scale.p, a_scale.ld * 4);
  p.vec_bs = vector_rows(b_scale.p, b_scale.ld * 4);
  // Pairs of CTAs on 256 x 256 tiles where these fill the device, else smaller tiles.
  const int sms = multiprocessors();
  if ((int64_t)((m + 255) / 256) * ((n + 255) / 256) * 2 >= sms)
    return run<2, 256>(a, b, b_lines, p, k, st);
  if ((int64_t)((m + 127) / 128) * ((n + 127) / 128) * 2 > sms)
    return run<1, 128>(a, b, b_lines, p, k, st);
  return run<1, 64>(a, b, b_lines, p, k, st);
}

// Reads and clears this translation unit's device error word (synchronising).
cudaError_t read_device_error_matmul(unsigned int* out) {
  const unsigned int zero = 0;
  cudaError_t err = cudaMemcpyFromSymbol(out, g_device_error, sizeof(unsigned int));
  if (err == cudaSuccess && *out)
    err = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(unsigned int));
  return err;
}

}  // namespace ff
}  // namespace fwt
