// Product of two 8-bit operands with a scale for each block of 128 along the contraction.
//
// The tensor cores sum one block's products (128 along the contraction, four instructions)
// into tensor memory; the scales are fp32 and differ from row to row, so each block's sums
// are then taken into registers and added there, times both scales, in fp32:
//
//     acc[i, j] += part_t[i, j] * (a_scale[i, t] * b_scale[j, t])
//
// CTAs are persistent, one an SM.  One warp fills a ring of operand stages by TMA, one or two
// threads issue the products of block after block into rings of accumulator slots, one warp
// brings the scales, and eight warps read slot after slot, half of the tile's columns each of
// two to a quarter of its rows: a tile of 256 columns costs them 128 values a thread and block.
// Large products pair two CTAs on a tile of 256 x 256.
//
// Bound, large: the latency of those sums.  8192 x 8192 x 4096: 194 us in bursts, 2830 TFLOP/s, and
// 218 us for seconds on end (1755 MHz under the power limit); the tensor pipe is active 50 to 53%
// of the cycles, the issue slots 42%.  A block's products take 512 clocks and its sums some 800, in
// which a warp mostly waits: without the additions, or without the reads of tensor memory, the
// same kernel takes 167 us, without both and the stores 143.  Tried and slower: packed pairs of
// multiply-adds (628 clocks a block against 327 for the sums alone: half the rate, and tensor
// memory's registers had to be moved into pairs), 64 columns a warp and sixteen warps (216 us:
// the steps around the sums then fill the issue slots), the next block's reads begun before the
// last sums (225 us), the next wait asked ahead (219 us).  With a scale for every line of b
// each sum takes two operations: 4096 x 8192 x 4096 in 155 us.
// Small: latency, some 3 us and 0.25 us a block; 48 x 8192 x 4096 11.6 us (3.0 TB/s).
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "feed_forward.cuh"
#include "ff_host.cuh"
#include "fwt.h"
#include "scales.cuh"
#include "tcgen05.cuh"

namespace fwt {
namespace ff {
namespace {

constexpr int kBlock = 128;  // elements of the contraction that share a scale: one stage
constexpr int kSharedBytes = 230400;  // of 232448: the rest is for alignment and barriers
constexpr int kStoreBytes = 8 * 4096;  // a piece of C of each of eight warps, see store_rows
constexpr int kThreads = 384;  // a warp each for copies and products (of four), eight for the sums
// Registers of a thread: 168 at launch (384 threads), moved from the first warpgroup to the
// two that hold 128 sums a thread: 128 * 72 + 256 * 216 = 384 * 168.
constexpr int kLeanRegisters = 72, kSumRegisters = 216;
static_assert(128 * kLeanRegisters + 256 * kSumRegisters == 384 * 168, "the launch's registers");

struct BlocksParams {
  const uint8_t *a, *b;
  int64_t ld_a, ld_b;
  int k;
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

// CG: CTAs that share a tile.  BN: its columns.  LINES: lines of b that share a scale.  ROWS:
// lines of a in a stage; with 64 the products read on into the next bytes for the other rows
// of their 128, which are not stored.  SPLIT: CTAs of a cluster that share out a tile's blocks.
template <int CG, int BN, int LINES, int ROWS, int SPLIT>
struct Config {
  static constexpr int kABytes = ROWS * 128, kBBytes = BN / CG * 128;
  static constexpr int kStage = kABytes + kBBytes;
  // A tile of 256 columns is multiplied in two halves, each by a warp of its own into slots of
  // its own, which four of the eight summing warps read: from the issue of a block's products
  // to its slot's return is some 1500 clocks (of which the products take 512), too long for
  // the two slots that whole blocks leave room for.
  static constexpr int kParts = BN == 256 ? 2 : 1;
  static constexpr int kCols = BN / kParts;         // columns of a slot
  static constexpr int kSlots = BN == 256 ? 2 : 4;  // of each part
  // scales of four blocks: one of a for each row; of b for each column, or each 128
  static constexpr int kBScales = LINES == 1 ? BN : BN == 256 ? 2 : 1;
  static constexpr int kScales = 4 * (128 + kBScales);  // floats
  static constexpr int kFixed = 2 * kScales * 4 + kStoreBytes;
  static constexpr int kStages = (kSharedBytes - kFixed) / kStage < 12 ? (kSharedBytes - kFixed) / kStage : 12;
  static constexpr size_t kSmem = (size_t)kStages * kStage + kFixed + 1024;
};

// The scales of four blocks of one line from block `t` on; zero past the line's end and for
// lines outside the matrix.
__device__ __forceinline__ float4 scales4(const float* base, int64_t ld, int line, int lines, int t,
                                          int blocks, bool vec) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (line >= lines) return v;
  const float* row = base + line * ld + t;
  if (vec && t + 4 <= blocks) return *(const float4*)row;
  v.x = *row;
  if (t + 1 < blocks) v.y = row[1];
  if (t + 2 < blocks) v.z = row[2];
  if (t + 3 < blocks) v.w = row[3];
  return v;
}

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

// A warp's rows of C, N columns from `col`, one row a thread: in pieces of 128 bytes a row
// through the warp's 4 KB of shared memory (16-byte chunks swizzled by row), so that global
// stores are whole 128-byte lines.  Stored from the registers as they lie, 16 bytes a row and
// instruction, they took a quarter of a tile's time.
template <typename C, int N>
__device__ __forceinline__ void store_rows(const BlocksParams& p, uint8_t* piece, int row0, int lane,
                                           int col, const float (&acc)[N]) {
  constexpr int kPiece = 128 / sizeof(C) < N ? 128 / sizeof(C) : N;  // columns
  constexpr int kChunks = kPiece * sizeof(C) / 16, kPer = 16 / sizeof(C);
  const bool vec = p.vec_c != 0;
#pragma unroll
  for (int c = 0; c < N; c += kPiece) {
    if (col + c >= p.n) return;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      uint32_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(C) == 4)
          v[j] = __float_as_uint(acc[c + i * kPer + j]);
        else
          v[j] = pack2<C>(acc[c + i * kPer + 2 * j], acc[c + i * kPer + 2 * j + 1]);
      }
      *(uint4*)(piece + lane * 128 + ((i ^ (lane & 7)) & (kChunks - 1)) * 16) =
          make_uint4(v[0], v[1], v[2], v[3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int r = i * (32 / kChunks) + lane / kChunks, chunk = lane & (kChunks - 1);
      const uint4 v = *(const uint4*)(piece + r * 128 + ((chunk ^ (r & 7)) & (kChunks - 1)) * 16);
      const int at = col + c + chunk * kPer;
      if (row0 + r < p.m && at < p.n) {
        C* out = (C*)p.c + (int64_t)(row0 + r) * p.ld_c + at;
        if (vec && at + kPer <= p.n) {
          *(uint4*)out = v;
        } else {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            if (at + j < p.n) {
              if constexpr (sizeof(C) == 4) *(uint32_t*)(out + j) = w[j];
              else *(unsigned short*)(out + j) = (unsigned short)(w[j / 2] >> (16 * (j & 1)));
            }
        }
      }
    }
    __syncwarp();
  }
}

// 16 bytes of a line of k from `at` on: zero past its end and for line = null.
__device__ __forceinline__ uint4 codes16(const uint8_t* line, int at, int k) {
  uint32_t w[4] = {0, 0, 0, 0};
  if (line && at + 16 <= k) return *(const uint4*)(line + at);
  if (line)
    for (int i = 0; at + i < k; ++i) w[i / 4] |= (uint32_t)line[at + i] << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp's 32 rows and `cols` columns of C again, straight from global memory into 16 x 8 products:
// for tiles with scales whose product overflows.  (In the loop of sums itself, a way for these
// costs the others 5%, though no call takes it: the loop then holds its 128 sums differently.)
template <int LINES>
__device__ __noinline__ void sum_apart(const BlocksParams& p, int row0, int col0, int cols) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll 1
  for (int sub = 0; sub < 2 * (cols / 8); ++sub) {
    const int row = row0 + 16 * (sub & 1) + g, col = col0 + 8 * (sub >> 1);
    if (col >= p.n) break;
    const int rows[2] = {row, row + 8}, line = col + g;
    const uint8_t* a[2] = {rows[0] < p.m ? p.a + (int64_t)rows[0] * p.ld_a : nullptr,
                           rows[1] < p.m ? p.a + (int64_t)rows[1] * p.ld_a : nullptr};
    const uint8_t* b = line < p.n ? p.b + (int64_t)line * p.ld_b : nullptr;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int block = 0; block < p.blocks; ++block) {
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (which bytes meet in which slot of a product is free as long as both operands agree)
        const int at = block * kBlock + 64 * h + 16 * t;
        const uint4 lo = codes16(a[0], at, p.k), hi = codes16(a[1], at, p.k), x = codes16(b, at, p.k);
        mma_e4m3(part, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
        mma_e4m3(part, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = rows[e >> 1], j = col + 2 * t + (e & 1);
        if (i < p.m && j < p.n)
          sum[e] = add_apart(sum[e], part[e], p.a_scale[i * p.ld_as + block],
                             p.b_scale[j / LINES * p.ld_bs + block]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = rows[e >> 1], j = col + 2 * t + (e & 1);
      if (i >= p.m || j >= p.n) continue;
      const int64_t at = i * p.ld_c + j;
      if (p.c_type == FWT_F32) ((float*)p.c)[at] = sum[e];
      else if (p.c_type == FWT_BF16) ((__nv_bfloat16*)p.c)[at] = __float2bfloat16_rn(sum[e]);
      else ((__half*)p.c)[at] = __float2half_rn(sum[e]);
    }
  }
}

template <int CG, int BN, int LINES, int ROWS, int SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    blocks_kernel(const __grid_constant__ BlocksMaps maps, const BlocksParams p) {
  using C = Config<CG, BN, LINES, ROWS, SPLIT>;
  static_assert(CG == 1 || SPLIT == 1, "a pair shares the tile, not its blocks");
  constexpr uint32_t kIdesc = instruction(0, false, false, 128 * CG, C::kCols);
  constexpr int kHalf = BN / 2;  // columns of a warp

  extern __shared__ uint8_t dynamic[];
  // done: a stage's products (of a part) are, so the slot is there to read, and with both
  // parts the stage's memory free again
  __shared__ uint64_t full[C::kStages], done[C::kParts][C::kStages], slot_empty[C::kParts][C::kSlots],
      scales_full[2], scales_empty[2];
  __shared__ uint32_t tmem_base;
  __shared__ volatile int gave_up;
  __shared__ float overflow;  // not 0: some product of scales may

  const uint32_t ring = (smem_u32(dynamic) + 1023u) & ~1023u;
  uint8_t* after_ring = dynamic + (ring - smem_u32(dynamic)) + C::kStages * C::kStage;
  float* scales = (float*)(after_ring + kStoreBytes);  // [2][4][rows, then of b]
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0 : cluster_rank();
  const int tiles = p.tiles_m * p.tiles_n;
  const int first = blockIdx.x / (CG * SPLIT), stride = gridDim.x / (CG * SPLIT);
  // the CTA's blocks: all, or its share of them
  const int share = (p.blocks + SPLIT - 1) / SPLIT;
  const int begin = SPLIT == 1 ? 0 : min(p.blocks, (int)cluster_rank() * share);
  const int end = SPLIT == 1 ? p.blocks : min(p.blocks, begin + share);

  // Tiles in groups of 16 rows of tiles, so that those in flight together share operands in L2
  // (4096 x 8192 x 8192: 195 us, with 8 rows 200).
  constexpr int kGroup = 16;
  auto place = [&](int index, int& m0, int& n0) {
    const int group = index / (kGroup * p.tiles_n);
    const int height = min(kGroup, p.tiles_m - group * kGroup);
    index -= group * kGroup * p.tiles_n;
    m0 = (group * kGroup + index % height) * (128 * CG);
    n0 = index / height * BN;
  };

  bool met = false;  // whether the warp is past the cluster's first barrier

  auto store = [&](uint8_t* piece, int row0, int col, const auto& sums) {
    if (p.c_type == FWT_F32) store_rows<float>(p, piece, row0, lane, col, sums);
    else if (p.c_type == FWT_BF16) store_rows<__nv_bfloat16>(p, piece, row0, lane, col, sums);
    else store_rows<__half>(p, piece, row0, lane, col, sums);
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(&full[i], 1);
    for (int part = 0; part < C::kParts; ++part) {
      for (int i = 0; i < C::kStages; ++i) mbar_init(&done[part][i], 1);
      for (int i = 0; i < C::kSlots; ++i) mbar_init(&slot_empty[part][i], 8 / C::kParts * CG);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&scales_full[i], 1), mbar_init(&scales_empty[i], 8);
    gave_up = 0, overflow = 0.f;
    prefetch_map(&maps.a), prefetch_map(&maps.b);
  }
  if (warp == 1) tmem_alloc<CG>(&tmem_base, C::kParts * C::kSlots * C::kCols);
  tmem_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = tmem_base;
  pdl_begin();

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
          for (int t = begin; t < end; ++t) {
#pragma unroll
            for (int part = 0; part < C::kParts; ++part)
              if (!wait_or_leave(&done[part][stage], parity, &gave_up)) return;
            const uint32_t a = ring + stage * C::kStage;
            const uint32_t bar = bars + 8 * stage;
            if (elect_one()) {
              if (rank == 0) mbar_arrive_expect_tx(&full[stage], C::kStage * CG);
              tma_load_tile<CG>(a, &maps.a, t * kBlock, m0 + (int)rank * 128, bar);
              // each part's lines together, half of them in each CTA of a pair
#pragma unroll
              for (int part = 0; part < C::kParts; ++part)
                tma_load_tile<CG>(a + C::kABytes + part * (C::kBBytes / C::kParts), &maps.b,
                                  t * kBlock, n0 + part * C::kCols + (int)rank * (C::kCols / CG), bar);
            }
            __syncwarp();
            if (++stage == C::kStages) stage = 0, parity ^= 1;
          }
        }
      }();
    } else if (warp <= C::kParts) {
      // products (of the pair's first CTA for both): warp 1, and 2 for the second part
      if (rank == 0)
      [&] {
        const int part = warp - 1;
        int stage = 0, slot = 0;
        uint32_t parity = 0, slot_parity = 1;
        bool filled = false, returned = false;  // asked one block ahead
        for (int index = first; index < tiles; index += stride) {
          for (int t = begin; t < end; ++t) {
            if (!wait_or_leave(&full[stage], parity, &gave_up, filled)) return;
            if (!wait_or_leave(&slot_empty[part][slot], slot_parity, &gave_up, returned)) return;
            tmem_fence_after();
            const uint32_t a = ring + stage * C::kStage;
            const uint64_t da = operand(a, 16);
            const uint64_t db = operand(a + C::kABytes + part * (C::kBBytes / C::kParts), 16);
            const uint32_t d = tmem + (part * C::kSlots + slot) * C::kCols;
            uint64_t* summed = &done[part][stage];
            if (++stage == C::kStages) stage = 0, parity ^= 1;
            if (++slot == C::kSlots) slot = 0, slot_parity ^= 1;
            filled = mbar_test(&full[stage], parity);
            returned = mbar_test(&slot_empty[part][slot], slot_parity);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kBlock / 32; ++kk)  // 32 bytes of a swizzle row each
                mma_tile<CG, 1>(d, da + 2 * kk, db + 2 * kk, kIdesc, kk > 0);
              mma_commit<CG>(summed);
            }
            __syncwarp();
          }
        }
      }();
    } else if (warp == 3) {
      // scales: those of four blocks at a time to shared memory, a row of kScales / 4 floats
      // for each block
      [&] {
        int buffer = 0;
        uint32_t parity = 1;
        constexpr int kRow = C::kScales / 4;
        const bool vec_as = p.vec_as && begin % 4 == 0, vec_bs = p.vec_bs && begin % 4 == 0;
        for (int index = first; index < tiles; index += stride) {
          int m0, n0;
          place(index, m0, n0);
          for (int t = begin; t < end; t += 4) {
            float4 a[4], b[LINES == 1 ? BN / 32 : 1];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              a[i] = scales4(p.a_scale, p.ld_as, m0 + (int)rank * 128 + lane + 32 * i, p.m, t,
                             p.blocks, vec_as);
            if constexpr (LINES == 1) {
#pragma unroll
              for (int i = 0; i < BN / 32; ++i)
                b[i] = scales4(p.b_scale, p.ld_bs, n0 + lane + 32 * i, p.n, t, p.blocks, vec_bs);
            } else if (lane < C::kBScales) {
              b[0] = scales4(p.b_scale, p.ld_bs, n0 / 128 + lane, (p.n + 127) / 128, t, p.blocks,
                             vec_bs);
            }
            // the largest magnitudes, as whole numbers, of scales that are finite (of others the
            // products are not, however they are taken)
            uint32_t most[2] = {0, 0};
            auto look = [&](uint32_t& top, float4 v) {
              for (const float s : {v.x, v.y, v.z, v.w})
                if (fabsf(s) < INFINITY) top = max(top, __float_as_uint(s) & 0x7fffffffu);
            };
#pragma unroll
            for (int i = 0; i < 4; ++i) look(most[0], a[i]);
#pragma unroll
            for (int i = 0; i < (LINES == 1 ? BN / 32 : 1); ++i)
              if (LINES == 1 || lane < C::kBScales) look(most[1], b[i]);
            const float top = __uint_as_float(__reduce_max_sync(~0u, most[0])) *
                              __uint_as_float(__reduce_max_sync(~0u, most[1]));
            if (!wait_or_leave(&scales_empty[buffer], parity, &gave_up)) return;
            if (!(top < INFINITY) && lane == 0) overflow = 1.f;
            float* to = scales + buffer * C::kScales;
            auto put = [&](int at, float4 v) {
              to[at] = v.x, to[at + kRow] = v.y, to[at + 2 * kRow] = v.z, to[at + 3 * kRow] = v.w;
            };
#pragma unroll
            for (int i = 0; i < 4; ++i) put(lane + 32 * i, a[i]);
            if constexpr (LINES == 1) {
#pragma unroll
              for (int i = 0; i < BN / 32; ++i) put(128 + lane + 32 * i, b[i]);
            } else if (lane < C::kBScales) {
              put(128 + lane, b[0]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&scales_full[buffer]);
            buffer ^= 1;
            if (buffer == 0) parity ^= 1;
          }
        }
      }();
    }
  } else {
    if constexpr (BN == 256)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegisters));
    // sums: warp w reads lanes 32 (w mod 4) on, a row of the tile each, and half its columns
    [&] {
      int stage = 0, slot = 0, buffer = 0;
      uint32_t done_parity = 0, parity = 0;
      const int quarter = warp & 3, half = (warp - 4) >> 2;
      const int part = C::kParts == 2 ? half : 0;
      uint32_t release = smem_u32(&slot_empty[part][0]);
      if constexpr (CG == 2) release = map_to_rank(release, 0);
      uint8_t* piece = after_ring + (warp - 4) * 4096;
      const uint32_t lanes = tmem + part * (C::kSlots * C::kCols) +
                             (C::kParts == 2 ? 0 : half * kHalf) + ((uint32_t)quarter << 21);
      for (int index = first; index < tiles; index += stride) {
        int m0, n0;
        place(index, m0, n0);
        float acc[kHalf];
#pragma unroll
        for (int i = 0; i < kHalf; ++i) acc[i] = 0.f;
        for (int t0 = begin; t0 < end; t0 += 4) {
          // the scales of four blocks: the row's (times b's one, or b's row beside it)
          if (!wait_or_leave(&scales_full[buffer], parity, &gave_up)) return;
          const float* row = scales + buffer * C::kScales;
          float s[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            s[u] = row[u * (C::kScales / 4) + quarter * 32 + lane];
            if constexpr (LINES == 128) s[u] *= row[u * (C::kScales / 4) + 128 + (BN == 256 ? half : 0)];
          }
          if constexpr (LINES == 128) {
            __syncwarp();
            mbar_arrive(&scales_empty[buffer], lane == 0);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (t0 + u >= end) break;
            uint32_t v[2][32];
            auto add = [&](int c, const uint32_t(&x)[32]) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                float4 f = make_float4(s[u], s[u], s[u], s[u]);
                if constexpr (LINES == 1) {
                  // two scales of columns at a time by the row's
                  const ulonglong2 pair = *(const ulonglong2*)&row[u * (C::kScales / 4) + 128 + half * kHalf + c + i];
                  unsigned long long ss, lo, hi;
                  asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s[u]));
                  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(lo) : "l"(pair.x), "l"(ss));
                  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(hi) : "l"(pair.y), "l"(ss));
                  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(lo));
                  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.z), "=f"(f.w) : "l"(hi));
                }
                float* sum = &acc[c + i];
                sum[0] = fmaf(__uint_as_float(x[i]), f.x, sum[0]);
                sum[1] = fmaf(__uint_as_float(x[i + 1]), f.y, sum[1]);
                sum[2] = fmaf(__uint_as_float(x[i + 2]), f.z, sum[2]);
                sum[3] = fmaf(__uint_as_float(x[i + 3]), f.w, sum[3]);
              }
            };
            if (!wait_or_leave(&done[part][stage], done_parity, &gave_up)) return;
            if (++stage == C::kStages) stage = 0, done_parity ^= 1;
            tmem_fence_after();
            const uint32_t at = lanes + slot * C::kCols;
            tmem_load32(at, v[0]);
            if constexpr (kHalf >= 64) tmem_load32(at + 32, v[1]);
            tmem_wait_loads();
            if constexpr (kHalf == 128) {
              add(0, v[0]);
              tmem_load32(at + 64, v[0]);
              add(32, v[1]);
              tmem_load32(at + 96, v[1]);
              tmem_wait_loads();
            }
            // the slot is read: it goes back before the last sums, as products may wait for it
            tmem_fence_before();
            if constexpr (CG == 2) mbar_arrive_cluster(release + 8 * slot, lane == 0);
            else mbar_arrive(&slot_empty[part][slot], lane == 0);
            if (++slot == C::kSlots) slot = 0;
            add(kHalf == 128 ? 64 : 0, v[0]);
            if constexpr (kHalf >= 64) add(kHalf == 128 ? 96 : 32, v[1]);
          }
          if constexpr (LINES == 1) {
            __syncwarp();
            mbar_arrive(&scales_empty[buffer], lane == 0);
          }
          if (++buffer == 2) buffer = 0, parity ^= 1;
        }
        const int row0 = m0 + (int)rank * 128 + quarter * 32, col = n0 + half * kHalf;
        if constexpr (SPLIT == 1) {
          store(piece, row0, col, acc);
        } else {
          // Every CTA of the cluster leaves its sums in its own ring, which its products are
          // done with, and adds up and stores a share of the columns, in the order of ranks.
          // whole eights of the warp's columns, the last CTAs' shares smaller or empty
          constexpr int kShare = (kHalf / 8 + SPLIT - 1) / SPLIT * 8;
          constexpr int W = kShare % 32 == 0 ? 32 : kShare % 16 == 0 ? 16 : 8;
          float* mine = (float*)(dynamic + (ring - smem_u32(dynamic))) + (warp - 4) * kHalf * 32 + lane;
#pragma unroll
          for (int i = 0; i < kHalf; ++i) mine[i * 32] = acc[i];
          cluster_sync();
          met = true;
          const int from = (int)cluster_rank() * kShare;
#pragma unroll 1
          for (int c = from; c < min(from + kShare, kHalf); c += W) {
            float sum[W];
#pragma unroll
            for (int i = 0; i < W; ++i) sum[i] = 0.f;
            const uint32_t there = smem_u32(mine) + c * 128;
#pragma unroll
            for (int r = 0; r < SPLIT; ++r) {
              const uint32_t peer = map_to_rank(there, r);
#pragma unroll
              for (int i = 0; i < W; ++i) sum[i] += load_cluster(peer + i * 128);
            }
            store(piece, row0, col + c, sum);
          }
          bool again = false;
          for (int r = 0; r < SPLIT; ++r)
            again |= load_cluster(map_to_rank(smem_u32(&overflow), r)) != 0.f;
          __syncwarp();
          if (again && from < kHalf) sum_apart<LINES>(p, row0, col + from, min(kShare, kHalf - from));
        }
      }
      if (SPLIT == 1 && overflow != 0.f) {
        for (int index = first; index < tiles; index += stride) {
          int m0, n0;
          place(index, m0, n0);
          __syncwarp();
          sum_apart<LINES>(p, m0 + (int)rank * 128 + quarter * 32, n0 + half * kHalf, kHalf);
        }
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
  if (warp == 1) tmem_free<CG>(tmem, C::kParts * C::kSlots * C::kCols);
}

template <int CG, int BN, int LINES, int ROWS, int SPLIT>
cudaError_t launch_config(const BlocksMaps& maps, BlocksParams p, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  p.tiles_m = (p.m + 128 * CG - 1) / (128 * CG);
  p.tiles_n = (p.n + BN - 1) / BN;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles > 0x7fffff00 / SPLIT) return cudaErrorInvalidConfiguration;
  const int64_t grid = SPLIT > 1 ? tiles * SPLIT : std::min<int64_t>(tiles, multiprocessors() / CG) * CG;
  log_kernel("matmul_blocks m=%d n=%d k=%d scale_lines=%d | tiles %dx%d rows=%d split=%d", p.m, p.n, p.k,
             LINES, 128 * CG, BN, ROWS, SPLIT);
  return launch_cluster(blocks_kernel<CG, BN, LINES, ROWS, SPLIT>, ready, (unsigned)grid, kThreads,
                        Config<CG, BN, LINES, ROWS, SPLIT>::kSmem, CG * SPLIT, st, maps, p);
}

template <int CG, int BN, int ROWS = 128, int SPLIT = 1>
cudaError_t run(CMat a, CMat b, int b_lines, const BlocksParams& p, int k, cudaStream_t st) {
  BlocksMaps maps;
  if (!swizzled_map(&maps.a, a.p, 1, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.m, k, a.ld, ROWS) ||
      !swizzled_map(&maps.b, b.p, 1, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.n, k, b.ld,
                    Config<CG, BN, 128, ROWS, SPLIT>::kCols / CG))
    return cudaErrorInvalidValue;
  return b_lines == 1 ? launch_config<CG, BN, 1, ROWS, SPLIT>(maps, p, st)
                      : launch_config<CG, BN, 128, ROWS, SPLIT>(maps, p, st);
}

// Tiles of 128 columns, each shared out over `split` CTAs.
template <int ROWS>
cudaError_t run_split(int split, CMat a, CMat b, int b_lines, const BlocksParams& p, int k,
                      cudaStream_t st) {
  if (split == 8) return run<1, 128, ROWS, 8>(a, b, b_lines, p, k, st);
  if (split == 6) return run<1, 128, ROWS, 6>(a, b, b_lines, p, k, st);
  if (split == 4) return run<1, 128, ROWS, 4>(a, b, b_lines, p, k, st);
  if (split == 3) return run<1, 128, ROWS, 3>(a, b, b_lines, p, k, st);
  if (split == 2) return run<1, 128, ROWS, 2>(a, b, b_lines, p, k, st);
  return run<1, 128, ROWS, 1>(a, b, b_lines, p, k, st);
}

bool vector_rows(const void* p, int64_t ld_bytes) {
  return ((uintptr_t)p & 15u) == 0 && ld_bytes % 16 == 0;
}

}  // namespace

cudaError_t launch_matmul_blocks(CMat a, CMat a_scale, CMat b, CMat b_scale, int b_lines, Mat c,
                                 int c_type, int m, int n, int k, cudaStream_t st) {
  // Straight from global memory up to 16 tokens, and to 32 where b is small (both ways
  // measured, us: 16 tokens by 4096 x 4096 6.3 against 9.1 here; 32 tokens by 2048 x 2048 3.9
  // against 6.1, by 2816 x 2816 8.2 against 7.5).
  if (m <= 16 || (m <= kMostTokens && (int64_t)n * k <= 6 << 20))
    return launch_matmul_tokens(a, a_scale, b, b_scale, b_lines, c, c_type, m, n, k, st);
  BlocksParams p{};
  p.a = (const uint8_t*)a.p, p.ld_a = a.ld, p.b = (const uint8_t*)b.p, p.ld_b = b.ld, p.k = k;
  p.a_scale = (const float*)a_scale.p, p.ld_as = a_scale.ld;
  p.b_scale = (const float*)b_scale.p, p.ld_bs = b_scale.ld;
  p.c = c.p, p.ld_c = c.ld, p.c_type = c_type;
  p.m = m, p.n = n, p.blocks = (int)(((int64_t)k + kBlock - 1) / kBlock);
  p.vec_c = vector_rows(c.p, c.ld * (c_type == FWT_F32 ? 4 : 2));
  p.vec_as = vector_rows(a_scale.p, a_scale.ld * 4);
  p.vec_bs = vector_rows(b_scale.p, b_scale.ld * 4);
  // Pairs of CTAs on 256 x 256 tiles, or single ones on 128 x 128 whose blocks a cluster shares
  // out where the tiles leave multiprocessors idle.  A block costs a CTA about the same either
  // way (it moves 32 KB), so what counts is the blocks that one CTA after the other goes
  // through, waves of tiles times blocks a tile; sharing out costs about as much as eight of
  // them (measured: 1.7 us and more, at 0.25 us a block).
  const int64_t sms = multiprocessors();
  const auto tiles = [&](int64_t size) { return ((m + size - 1) / size) * ((n + size - 1) / size); };
  const int64_t wide = (tiles(256) + sms / 2 - 1) / (sms / 2) * p.blocks, small = tiles(128);
  int64_t least = (small + sms - 1) / sms * p.blocks;
  int split = 1;
  // (clusters of three and more do not fill every multiprocessor of a graphics cluster)
  for (int s : {2, 3, 4, 6, 8})
    if (s * small <= (s > 2 ? sms * 7 / 8 : sms) && (p.blocks + s - 1) / s + 8 < least)
      split = s, least = (p.blocks + s - 1) / s + 8;
  if (wide < least) return run<2, 256>(a, b, b_lines, p, k, st);
  return m <= 64 ? run_split<64>(split, a, b, b_lines, p, k, st)
                 : run_split<128>(split, a, b, b_lines, p, k, st);
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
