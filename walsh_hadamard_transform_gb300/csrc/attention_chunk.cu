// Attention of many rows (new tokens x query heads of a key head) over the 8-bit cache, on tensor cores:
// prompts and chunks of them.
//
// An item is 256 rows with one key head, two tiles of 128; its keys come by 128.  For each tile and
// step
//
//   S = Q K^T            128 x 128 in tensor memory
//   P = 2^(c S - m + 11) a row a thread; float16, over S in tensor memory; l += P in fp32
//   O += P V             in tensor memory, fp32; every 8192 keys added to those before
//
// and the two tiles take turns: while the tensor cores work on one, the other's softmax runs.  m is a
// maximum of the row that may lag behind by a factor of 2^4 in P: only a larger step multiplies O
// again, which is rare after the first keys.  So P is at most 2^15, and of a probability p, the row's largest 1,
// float16 keeps all its bits down to 2^-25 and steps of 2^-35 below: many small ones next to a large one are
// a part of the output, whether the large one's value is or not.  (Both times 2^11, so O / l is the output.)
//
// Four warps turn codes into float16 operands in the layout the products read (128-byte swizzle; keys
// along the contraction, values across it).  The scales go in with them, exactly: a key's
// factor is 2^(4 + e - e_ref), e_ref the largest scale's exponent of the item's first keys, moved only
// when one is more than 2^3 above it; what lies more than 2^19 below it keeps fewer bits
// (float16's smallest step).  So c is one number a row and the softmax has no scales to look up.
// Values the same, with O in units of 2^e_ref.  Queries are rounded to float16 once after their rotation,
// each row at a power of two (for outputs of float16 and heads of 64, where there is room, as two float16:
// their rounding would add as much again as the output's own).
//
// Bound, large: the chain of a tile, softmax (some 2000 clocks) and its two products (1000), of which
// two are under way at a time; the issue slots and the exponentials (32 a clock an SM, 1024 clocks a step
// of both tiles) are not full (over 8192: tensor cores 37% active, exponentials 19%, issue 39%).  4096 tokens by 32 query
// and 8 key heads of 128 over 32768: 1.88 ms, 1.09 PFLOP/s, 57% of what cuBLAS reaches.  Short items: their queries
// and output, some eight steps an item; 8192 tokens by 16 heads 0.42 ms, 0.65 PFLOP/s, with a window of 1024 0.20 ms,
// not causal 0.63 ms.  With scores read twice instead of held in 128 registers
// (so no split of registers among the warps) the first took 4.9 ms; with the softmax at 176 and the operands
// at 104 registers 1.88, at 192 and 80, which spills, 2.24.
//
// Warps: 0 to 3 and 4 to 7 softmax and output of tile 0 and 1, 8 to 11 operands, 12 products, 13 the
// pages and scales of the steps ahead, 14 what there is to join.
#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attention_plan.cuh"
#include "cache.cuh"
#include "feed_forward.cuh"
#include "ff_host.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace fwt {
namespace ff {
namespace {

constexpr int kThreads = 512;
constexpr int kKeys = 128;    // of a step; a unit of the plan
constexpr int kStages = 2;    // of keys, and of values
constexpr int kAhead = 4;     // steps known at a time (4096 tokens over 32768: 3 2.09 ms, 4 1.88, 6 1.99)
// Steps that an item costs besides, its queries and its output (measured, us, at 6, 8 and 10: 8192 tokens by 16
// heads 438, 421, 419; five ragged chunks of up to 701 tokens 58.0, 59.3, 59.9; a chunk of 512 and 32 single tokens
// 199, 194, 194; the first two at 0 481 and 74, at 16 423 and 65).
constexpr int kExtra = 8;
// How far P may pass a row's maximum, in powers of two, and what lifts P: together 15, what float16 has.  (8 and 7
// lose small P sooner and measured 0.5% faster: 8192 tokens by 16 heads 421 and 423 us.)
constexpr float kLag = 4.f, kLift = 11.f;
// With c above 2^-15 a score may pass 2^23 (S is at most 2^38).  What the row's maximum lost to its rounding, and
// fma() keeps of a score, is then whole powers of two, so such scores are rounded first.
constexpr float kLargeFactor = 0x1p-15f;

// What a step's keys are, found by one warp some steps ahead and kept until its last product.
struct alignas(16) Step {  // (its factors are written 16 bytes at a time)
  uint32_t factors[2][kKeys];  // of keys and of values: a power of two, float16 twice
  const uint8_t* codes[2][8];  // of each 16 tokens of the key head; null: no page
  int there;                   // tokens of the step that the item has
  int more;                    // whether a step follows
  int key_ref, value_ref;      // scale bytes that stand for 2^kRaise in the operands
  int special;                 // whether any bit below is set
  uint32_t hidden[4];          // bit i of word j: token 32 j + i is no token
  uint32_t poison[4];          //                   its key or value is not a number
};
constexpr int kSumSteps = kSumKeys / kKeys;
constexpr int kRaise = 4;  // the largest scale at first; it may rise to 2^7 before the unit moves

template <int DIM>
struct Layout {
  static constexpr int kChunks = DIM / 64;                 // of 64 elements, 128 bytes a row
  static constexpr uint32_t kChunk = 128 * 128;            // bytes
  static constexpr uint32_t kTile = kChunks * kChunk;      // 128 rows
  static constexpr uint32_t kKeysAt = 2 * kTile, kValuesAt = kKeysAt + kStages * kTile;
  static constexpr bool kFine = DIM == 64;  // room for what the queries' rounding leaves
  static constexpr uint32_t kRestAt = kValuesAt + kStages * kTile;
  static constexpr uint32_t kStepsAt = kRestAt + (kFine ? 2 * kTile : 0);
  static constexpr size_t kBytes = kStepsAt + kAhead * sizeof(Step) + 1024;
};

constexpr uint32_t kScoresAt = 0, kOutAt = 256;  // tensor memory columns; 128 and DIM a tile
constexpr uint32_t kColumns = 512;

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Registers a thread from here on, for whole warpgroups: their sum stays what the CTA started with
// (4 x 128 x 128).
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
constexpr int kSoftmaxRegisters = 184, kOperandRegisters = 96, kProductRegisters = 48;
static_assert(2 * kSoftmaxRegisters + kOperandRegisters + kProductRegisters <= 4 * 128, "what the CTA has");

// 2^e in two factors, for -252 <= e <= 254.
__device__ __forceinline__ float times_power(float v, int e) {
  const int half = e >> 1;
  return v * __uint_as_float((uint32_t)(127 + half) << 23) * __uint_as_float((uint32_t)(127 + e - half) << 23);
}

// 2^f in both halves of a pair of float16, f <= 7; zero below 2^-24.
__device__ __forceinline__ uint32_t power_f16x2(int f) {
  const uint32_t h = f >= -14 ? (uint32_t)(f + 15) << 10 : f >= -24 ? 1u << (f + 24) : 0u;
  return h | h << 16;
}
__device__ __forceinline__ uint32_t multiply_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Bits 0 to R - 1 of the rotation among a thread's own N values, without the norm.
template <int N>
__device__ __forceinline__ void turn_all(float (&v)[N], int r) {
  if (r > 0) turn_own<N, 1>(v);
  if (r > 1) turn_own<N, 2>(v);
  if (r > 2) turn_own<N, 4>(v);
  if (r > 3) turn_own<N, 8>(v);
  if (r > 4) turn_own<N, 16>(v);
  if (r > 5) turn_own<N, 32>(v);
}

__device__ __forceinline__ int rows_of(const AttentionParams& p, const Walk& w) {  // of the item
  return min(kChunkRows, w.s.count * p.group - w.block * kChunkRows);
}

// The queries of tile `t` of the item where `w` stands: rotated, each row at a power of two, as
// float16 into the layout that the products read.  By the four warps of the tile, 32 rows each;
// a row is spread over DIM / 16 lanes.
template <int DIM>
__device__ __forceinline__ void stage_queries(const AttentionParams& p, const Walk& w, int t, uint8_t* memory,
                                           float* row_scale, uint64_t* full) {
  using L = Layout<DIM>;
  constexpr int kLanes = DIM / 16, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, part = lane & (kLanes - 1);
  const int row0 = 32 * (threadIdx.x >> 5 & 3) + sub, rows = rows_of(p, w) - 128 * t;
  if (rows <= 0) return;
  const float before = rotation_before(p.rot_bits), norm = rotation_after(p.rot_bits) * (p.scale < 0.f ? -1.f : 1.f);
  constexpr int kBatch = 2;  // rows on their way at a time
#pragma unroll 1
  for (int r0 = row0; r0 < row0 + 32; r0 += kBatch * kRows) {
    uint4 raw[kBatch][2];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * kRows;
      raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int row = w.block * kChunkRows + 128 * t + r;  // (rows times heads fit 31 bits)
        const int token = w.s.row + quotient(row, p.by_group), head = w.head * p.group + remainder(row, p.by_group);
        const uint16_t* q = (const uint16_t*)p.q.p + token * p.q.token + head * p.q.head + 8 * part;
        raw[i][0] = *(const uint4*)q, raw[i][1] = *(const uint4*)(q + DIM / 2);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * kRows;
      float v[16];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t x[4] = {raw[i][k].x, raw[i][k].y, raw[i][k].z, raw[i][k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = pair_to_float(x[j], p.type);
          v[8 * k + 2 * j] = f.x * before, v[8 * k + 2 * j + 1] = f.y * before;
        }
      }
      turn_spread<DIM>(v, p.rot_bits, part);
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        v[j] *= norm;
        top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
      }
#pragma unroll
      for (int step = 1; step < kLanes; step *= 2) top = max(top, __shfl_xor_sync(~0u, top, step));
      const int e = max((int)(top >> 23), 27);  // (zero, and what is nearly so)
      const float up = __uint_as_float((uint32_t)(254 + 14 - e) << 23);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int piece = part + (DIM == 128 ? 0 : 4 * k);
        uint32_t x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = pair_from_float<__half>(v[8 * k + 2 * j] * up, v[8 * k + 2 * j + 1] * up);
        uint8_t* to = memory + t * L::kTile + (DIM == 128 ? k * L::kChunk : 0) + r * 128 + ((piece ^ (r & 7)) << 4);
        *(uint4*)to = make_uint4(x[0], x[1], x[2], x[3]);
        if (L::kFine && p.type == FWT_F16) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 high = pair_to_float<__half>(x[j]);
            x[j] = pair_from_float<__half>(v[8 * k + 2 * j] * up - high.x, v[8 * k + 2 * j + 1] * up - high.y);
          }
          *(uint4*)(to + L::kRestAt) = make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
      if (part == 0) row_scale[128 * t + r] = fabsf(p.scale) * __uint_as_float((uint32_t)(e - 14) << 23);
    }
  }
  fence_to_products();
  __syncwarp();
  mbar_arrive(full, lane == 0);
}

template <int DIM>
__global__ void __launch_bounds__(kThreads, 1) attention_chunk_kernel(const AttentionParams p) {
  using L = Layout<DIM>;
  extern __shared__ uint8_t dynamic[];
  __shared__ uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
  __shared__ uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  __shared__ uint64_t known[kAhead], done[kAhead];  // steps that are found, and over
  __shared__ float row_scale[kChunkRows], sums_top[kChunkRows], sums_total[kChunkRows];
  __shared__ int sums_ref[8];
  __shared__ PlanScratch scratch;
  __shared__ uint32_t tmem_base;
  __shared__ volatile int gave_up;
  __shared__ volatile uint32_t issued;  // steps so far: a tile may sit out many
  __shared__ Walk walks[kThreads / 32][2];  // of each warp: where it stands, and one item ahead

  const uint32_t base = (smem_u32(dynamic) + 1023u) & ~1023u;
  uint8_t* memory = dynamic + (base - smem_u32(dynamic));
  Step* const ring = (Step*)(memory + L::kStepsAt);
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t)
      mbar_init(&q_full[t], 4), mbar_init(&s_full[t], 1), mbar_init(&p_full[t], 4), mbar_init(&o_full[t], 1);
    for (int s = 0; s < kStages; ++s)
      mbar_init(&k_full[s], 4), mbar_init(&k_empty[s], 1), mbar_init(&v_full[s], 4), mbar_init(&v_empty[s], 1);
    for (int i = 0; i < kAhead; ++i) mbar_init(&known[i], 1), mbar_init(&done[i], 1);
    gave_up = 0, issued = 0;
  }
  if (warp == 12) tmem_alloc<1>(&tmem_base, kColumns);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = tmem_base;
  pdl_begin();

  // (in shared memory: registers are dear, and a step needs little of it)
  Walk &walk = walks[warp][0], &next = walks[warp][1];
  {
    const Walk share = find_share<kChunkRows, kKeys, kExtra, 1, kThreads>(p, blockIdx.x, gridDim.x, scratch);
    if (lane == 0) walk = next = share;
    __syncwarp();
  }
  const auto advance = [&](Walk& w) {
    __syncwarp();
    if (lane == 0) next_piece<kChunkRows, kKeys, kExtra>(p, w);
    __syncwarp();
  };
  if (warp < 8) {
    registers_up<kSoftmaxRegisters>();
    // softmax and output of tile `t`; this thread's row of it is 32 (warp & 3) + lane
    [&] {
      const int t = warp >> 2, quarter = warp & 3, mine = 32 * quarter + lane;
      const uint32_t lanes = (uint32_t)quarter << 21;
      const uint32_t scores = tmem + kScoresAt + 128 * t + lanes, out = tmem + kOutAt + DIM * t + lanes;
      uint32_t steps = 0;              // of the share so far
      uint32_t turns = 0, pieces = 0;  // steps and items of this tile

      bool pending = false;  // an item whose output is to come: `walk` stands there, `next` after it
      bool starts = false, ends = false;
      int rows = 0, value_ref = 0;
      float top = -INFINITY;
      float2 total = make_float2(0.f, 0.f);
      // Where sums of the piece's earlier keys wait (kSumKeys), 32 i + 4 j on of this thread's row: within what the
      // warp's rows have in the part, the lanes' side by side.
      const auto sums_at = [&](int i, int j) {
        return (float4*)(p.parts + (2 * (int64_t)blockIdx.x + (starts ? 1 : 0)) * part_floats(kChunkRows, DIM) +
                         (128 * t + 32 * quarter) * DIM + (8 * i + j) * 128 + 4 * lane);
      };
      const auto output = [&] {
        const bool valid = 128 * t + mine < rows;
        if (!wait_or_leave(&o_full[t], pieces & 1, &gave_up)) return false;
        ++pieces;
        tmem_fence_after();
        const float l = total.x + total.y;
        // 2^e, e from -131 to 123, in two factors
        const int e = value_ref - (127 + kRaise), half_e = e >> 1;
        const float units[2] = {__uint_as_float((uint32_t)(127 + half_e) << 23), __uint_as_float((uint32_t)(127 + e - half_e) << 23)};
        // (in units of the scales up to the end: sums of values and of rows may pass fp32 where the output does not)
        const float norm = l == 0.f ? 0.f : (starts && ends ? rotation_norm(p.rot_bits) : 1.f) / l;
        const float unit[2] = {norm * units[0], units[1]};
        if (starts && ends) {
          const int row = walk.block * kChunkRows + 128 * t + mine;  // of the sequence's with this head
          const int token = walk.s.row + quotient(row, p.by_group), head = walk.head * p.group + remainder(row, p.by_group);
          uint16_t* to = (uint16_t*)p.out.p + token * p.out.token + head * p.out.head;
          // (64 of a row's elements at a time: the top bit of 128 first)
#pragma unroll 1
          for (int half = 0; half < DIM / 64; ++half) {
            float o[64];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t v[32];
              const bool both = DIM == 128 && p.rot_bits == 7;
              tmem_load32(out + 32 * i + (both ? 0 : 64 * half), v);
              tmem_wait_loads();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[32 * i + j] = __uint_as_float(v[j]);
              if (both) {
                tmem_load32(out + 32 * i + 64, v);
                tmem_wait_loads();
                const float sign = half ? -1.f : 1.f;
#pragma unroll
                for (int j = 0; j < 32; ++j) o[32 * i + j] = fmaf(sign, __uint_as_float(v[j]), o[32 * i + j]);
              }
            }
            turn_all(o, p.rot_bits);
#pragma unroll
            for (int j = 0; j < 64; ++j) o[j] = o[j] * unit[0] * unit[1];
            if (valid) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                *(uint4*)(to + 64 * half + 8 * j) =
                    make_uint4(pair_from_float(o[8 * j], o[8 * j + 1], p.type), pair_from_float(o[8 * j + 2], o[8 * j + 3], p.type),
                               pair_from_float(o[8 * j + 4], o[8 * j + 5], p.type), pair_from_float(o[8 * j + 6], o[8 * j + 7], p.type));
            }
          }
        } else {
          float* part = p.parts + (2 * (int64_t)blockIdx.x + (starts ? 1 : 0)) * part_floats(kChunkRows, DIM);
          const int r = 128 * t + mine;
#pragma unroll 1
          for (int i = 0; i < DIM / 32; ++i) {
            uint32_t v[32];
            tmem_load32(out + 32 * i, v);
            tmem_wait_loads();
            if (valid) {
              float4* to = (float4*)(part + (int64_t)r * DIM + 32 * i);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                float o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = __uint_as_float(v[4 * j + k]) * unit[0] * unit[1];
                to[j] = make_float4(o[0], o[1], o[2], o[3]);
              }
            }
          }
          if (valid) part[kChunkRows * DIM + r] = top, part[kChunkRows * DIM + kChunkRows + r] = l;
        }
        tmem_fence_before();  // (before the next item's products write there, which wait for p_full)
        return true;
      };
      while (true) {
        // the next item's queries while the last products of the one before run
        if (next.left > 0) stage_queries<DIM>(p, next, t, memory, row_scale, &q_full[t]);
        if (pending) {
          pending = false;
          if (!output()) return;
          advance(walk);
        }
        if (walk.left == 0) break;
        const int count = piece_units(walk);
        rows = rows_of(p, walk), starts = walk.unit == 0, ends = walk.unit + count == walk.units;
        advance(next);
        if (rows <= 128 * t) {
          steps += count;
          advance(walk);
          continue;
        }
        pending = true;
        const bool valid = 128 * t + mine < rows;
        const Keys seen = valid ? seen_by(p, walk.s, walk.block * kChunkRows + 128 * t + mine) : Keys{0, 0x7fffffff};
        const int first_key = walk.keys.low + walk.unit * kKeys;
        const float scale = row_scale[128 * t + mine];
        // (scale bytes of keys up to which no row of the warp has such a c)
        const int key_limit = -16 + (127 + kRaise) + 127 - (int)__reduce_max_sync(~0u, __float_as_uint(scale) >> 23);
        top = -INFINITY, total = make_float2(0.f, 0.f), value_ref = 0;
        int step = 0;
#pragma unroll 1
        while (true) {
          const int until = count > 2 * kSumSteps ? min(step + kSumSteps, count) : count;
#pragma unroll 1
          for (; step < until; ++step, ++steps, ++turns) {
            const int pos = first_key + step * kKeys;
            // (the scores before the first look at the ring: a tile that sits items out would see it long
            // before its step)
            if (step == 0 && !wait_or_leave(&s_full[t], turns & 1, &gave_up, false, &issued)) return;
            if (!wait_or_leave(&known[steps % kAhead], steps / kAhead & 1, &gave_up)) return;
            const Step& info = ring[steps % kAhead];
            float c = fmaxf(times_power(scale, info.key_ref - (127 + kRaise)), 0x1p-120f);
            const int new_ref = info.value_ref;
            const int from = seen.low - pos, to = seen.high - pos;  // of the step's keys
            const bool special = info.special != 0;
            const bool large = info.key_ref > key_limit;
            const bool masked = special || large || __any_sync(~0u, from > 0 || to < kKeys);
            if (step > 0 && !wait_or_leave(&s_full[t], turns & 1, &gave_up, false, &issued)) return;
            tmem_fence_after();

            uint32_t v[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_load32(scores + 32 * i, v[i]);
            tmem_wait_loads();
            if (masked) {
              const bool first = c > kLargeFactor;  // (each row for itself: what others hold does not matter)
              const float factor = first ? c : 1.f;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                // bits of keys 32 i on: those below `to`, less those below `from`
                const int low = min(max(from - 32 * i, 0), 32), high = min(max(to - 32 * i, 0), 32);
                uint32_t see = (uint32_t)((1ull << high) - 1) & ~(uint32_t)((1ull << low) - 1);
                uint32_t poison = 0;
                if (special) see &= ~info.hidden[i], poison = info.poison[i] & see;
#pragma unroll
                for (int j = 0; j < 32; ++j) v[i][j] = see & 1u << j ? __float_as_uint(__uint_as_float(v[i][j]) * factor) : 0xff800000u;
                if (__any_sync(~0u, poison != 0)) {
#pragma unroll
                  for (int j = 0; j < 32; ++j) v[i][j] = poison & 1u << j ? 0x7fc00000u : v[i][j];
                }
              }
              if (first) c = 1.f;
            }
            float m[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < 32; j += 2)
                m[j / 2 & 7] = max3(m[j / 2 & 7], __uint_as_float(v[i][j]), __uint_as_float(v[i][j + 1]));
            const float most = max3(max3(m[0], m[1], m[2]), max3(m[3], m[4], m[5]), fmaxf(m[6], m[7])) * c;  // (c > 0)
            float less = 1.f;
            bool again = false;
            if (most > __fadd_rd(top, kLag) || top == -INFINITY) {
              again = most > top && top != -INFINITY;
              if (again) less = exp2_fast(top - most);
              if (most > top) top = most;
            }
            const bool moved = step > 0 && __any_sync(~0u, again || new_ref != value_ref);
            // (down, as above: no P passes 2^15, whatever the size of the scores)
            const float shift = top == -INFINITY ? 0.f : __fadd_rd(kLift, -top);
            const float2 c2 = make_float2(c, c), shift2 = make_float2(shift, shift);
            float2 sums[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[i] = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t packed[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float2 x = fma_pair(make_float2(__uint_as_float(v[i][2 * j]), __uint_as_float(v[i][2 * j + 1])), c2, shift2);
                x.x = exp2_fast(x.x), x.y = exp2_fast(x.y);
                sums[j & 3] = add_pair(sums[j & 3], x);
                packed[j] = pair_from_float<__half>(x.x, x.y);
              }
              tmem_store16(scores + 16 * i, packed);
            }
            if (moved) {  // what is there so far, in the new units
              total.x *= less, total.y *= less;
              less *= __uint_as_float((uint32_t)max(127 + value_ref - new_ref, 0) << 23);
#pragma unroll 1
              for (int i = 0; i < DIM / 32; ++i) {
                uint32_t o[32];
                tmem_load32(out + 32 * i, o);
                tmem_wait_loads();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * less);
                tmem_store16(out + 32 * i, o);
                tmem_store16(out + 32 * i + 16, o + 16);
              }
            }
            value_ref = new_ref;
            total = add_pair(total, add_pair(add_pair(sums[0], sums[1]), add_pair(sums[2], sums[3])));
            tmem_wait_stores();
            tmem_fence_before();
            __syncwarp();
            mbar_arrive(&p_full[t], lane == 0);
          }
          if (step == count) break;
          // The sums so far, done when the next step's scores are there, and those before them: to wait, and that
          // step's products begin again, or back for the last keys to be added to.
          const bool last = step + kSumSteps >= count;
          if (!wait_or_leave(&s_full[t], turns & 1, &gave_up, false, &issued)) return;
          tmem_fence_after();
          float f = 0.f;  // to the units of now
          if (step > kSumSteps) {
            const float before = sums_top[128 * t + mine];
            f = before == -INFINITY ? 1.f : exp2_fast(before - top);
            total.x = fmaf(sums_total[128 * t + mine], f, total.x);
            f *= __uint_as_float((uint32_t)max(127 + sums_ref[warp] - value_ref, 0) << 23);
          }
          if (!last) sums_total[128 * t + mine] = total.x + total.y, total = make_float2(0.f, 0.f);
#pragma unroll 2
          for (int i = 0; i < DIM / 32; ++i) {
            uint32_t o[32];
            tmem_load32(out + 32 * i, o);
            float4 sums[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) sums[j] = step > kSumSteps ? *sums_at(i, j) : make_float4(0.f, 0.f, 0.f, 0.f);
            tmem_wait_loads();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 x = sums[j];
              const float4 sum = make_float4(fmaf(x.x, f, __uint_as_float(o[4 * j])), fmaf(x.y, f, __uint_as_float(o[4 * j + 1])),
                                             fmaf(x.z, f, __uint_as_float(o[4 * j + 2])), fmaf(x.w, f, __uint_as_float(o[4 * j + 3])));
              if (!last) *sums_at(i, j) = sum;
              o[4 * j] = __float_as_uint(sum.x), o[4 * j + 1] = __float_as_uint(sum.y);
              o[4 * j + 2] = __float_as_uint(sum.z), o[4 * j + 3] = __float_as_uint(sum.w);
            }
            if (last) tmem_store16(out + 32 * i, o), tmem_store16(out + 32 * i + 16, o + 16);
          }
          tmem_wait_stores();
          sums_top[128 * t + mine] = top;
          if (lane == 0) sums_ref[warp] = value_ref;
          __syncwarp();
        }
      }
    }();
  } else if (warp < 12) {
    // operands: a row of codes is spread over DIM / 16 lanes, 16 bytes each: two runs of 8, half a
    // row apart (64: one of 16), so that eight lanes' stores meet all banks
    registers_down<kOperandRegisters>();
    [&] {
      constexpr int kLanes = DIM / 16, kRows = 32 / kLanes, kTimes = 128 / (4 * kRows);
      constexpr int kApart = DIM == 128 ? 64 : 8;  // bytes between a lane's two runs
      const int w = warp - 8, sub = lane / kLanes, part = lane & (kLanes - 1);
      const int row0 = w * kRows + sub;  // and every 4 kRows on, a multiple of 16
      const int code_at = (row0 & 15) * DIM + part * (DIM == 128 ? 8 : 16);
      // where the two runs go: pieces of 16 bytes, swizzled by row
      uint32_t to[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int piece = DIM == 128 ? part : 2 * part + k;
        to[k] = (DIM == 128 ? k * L::kChunk : 0) + row0 * 128 + ((piece ^ (row0 & 7)) << 4);
      }
      uint2 codes[2][kTimes][2];
      const auto fetch = [&](const Step& at, int o) {
        const int there = at.there;
#pragma unroll
        for (int i = 0; i < kTimes; ++i) {
          const uint8_t* from = at.codes[o][(4 * i + w) * kRows / 16];
          codes[o][i][0] = codes[o][i][1] = make_uint2(0, 0);
          if (from && row0 + 4 * kRows * i < there) {
            from += code_at;
            codes[o][i][0] = *(const uint2*)from, codes[o][i][1] = *(const uint2*)(from + kApart);
          }
        }
      };
      // the fetched operand into shared memory
      const auto convert = [&](const Step& at, int o, uint32_t tile) {
#pragma unroll
        for (int i = 0; i < kTimes; ++i) {
          const uint32_t factor = at.factors[o][row0 + 4 * kRows * i];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint2 c = codes[o][i][k];
            *(uint4*)(memory + tile + to[k] + 4 * kRows * 128 * i) =
                make_uint4(multiply_f16x2(e4m3_to_f16x2(c.x), factor), multiply_f16x2(e4m3_to_f16x2(c.x >> 16), factor),
                           multiply_f16x2(e4m3_to_f16x2(c.y), factor), multiply_f16x2(e4m3_to_f16x2(c.y >> 16), factor));
          }
        }
        fence_to_products();
        __syncwarp();
      };

      if (walk.left == 0 || !wait_or_leave(&known[0], 0, &gave_up)) return;
      fetch(ring[0], 0), fetch(ring[0], 1);
      // (keys a step ahead of values, or values signalled in halves, measured 2 to 8% slower)
#pragma unroll 1
      for (uint32_t steps = 0;; ++steps) {
        const int stage = steps % kStages;
        const uint32_t parity = (steps / kStages & 1) ^ 1;
        const Step &now = ring[steps % kAhead], &after = ring[(steps + 1) % kAhead];
        const bool more = now.more != 0;
        if (!wait_or_leave(&k_empty[stage], parity, &gave_up)) return;
        convert(now, 0, L::kKeysAt + stage * L::kTile);
        mbar_arrive(&k_full[stage], lane == 0);
        if (more) {
          if (!wait_or_leave(&known[(steps + 1) % kAhead], (steps + 1) / kAhead & 1, &gave_up)) return;
          fetch(after, 0);
        }
        if (!wait_or_leave(&v_empty[stage], parity, &gave_up)) return;
        convert(now, 1, L::kValuesAt + stage * L::kTile);
        mbar_arrive(&v_full[stage], lane == 0);
        if (!more) break;
        fetch(after, 1);
      }
    }();
  } else {
    registers_down<kProductRegisters>();
    // products, by the first of these warps
    if (warp == 12) [&] {
      constexpr uint32_t kOfScores = instruction(0, false, false, 128, 128);
      constexpr uint32_t kOfOut = instruction(0, false, true, 128, DIM);
      uint32_t steps = 0, turns[2] = {0, 0}, pieces[2] = {0, 0};
      const auto scores = [&](int t, int stage) {
        const uint64_t a = operand(base + t * L::kTile, 16), b = operand(base + L::kKeysAt + stage * L::kTile, 16);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < DIM / 16; ++kk) {
            const uint32_t at = (kk >> 2) * (L::kChunk >> 4) + (kk & 3) * 2;
            mma_tile<1, 2>(tmem + kScoresAt + 128 * t, a + at, b + at, kOfScores, kk > 0);
            if (L::kFine && p.type == FWT_F16)
              mma_tile<1, 2>(tmem + kScoresAt + 128 * t, a + (L::kRestAt >> 4) + at, b + at, kOfScores, 1);
          }
          mma_commit<1>(&s_full[t]);
        }
        __syncwarp();
      };
      while (walk.left > 0) {
        const int count = piece_units(walk), tiles = rows_of(p, walk) > 128 ? 2 : 1;
        if (!wait_or_leave(&k_full[steps % kStages], steps / kStages & 1, &gave_up)) return;
        for (int t = 0; t < tiles; ++t) {
          if (!wait_or_leave(&q_full[t], pieces[t] & 1, &gave_up)) return;
          ++pieces[t];
          tmem_fence_after();
          scores(t, steps % kStages);
        }
        if (elect_one()) mma_commit<1>(&k_empty[steps % kStages]);
        __syncwarp();
        for (int step = 0; step < count; ++step, ++steps) {
          if (lane == 0) issued = steps;
          const int stage = steps % kStages, next_stage = (steps + 1) % kStages;
          const bool more = step + 1 < count;
          for (int t = 0; t < tiles; ++t) {
            if (t == 0 && !wait_or_leave(&v_full[stage], steps / kStages & 1, &gave_up)) return;
            const uint64_t b = operand(base + L::kValuesAt + stage * L::kTile, L::kChunk);
            if (!wait_or_leave(&p_full[t], turns[t] & 1, &gave_up)) return;
            ++turns[t];
            tmem_fence_after();
            const bool begins = count > 2 * kSumSteps && step % kSumSteps == 0 && step + kSumSteps < count;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)  // 16 rows of values, 8 columns of pairs of P
                mma_tile_from_tmem(tmem + kOutAt + DIM * t, tmem + kScoresAt + 128 * t + 8 * kk, b + kk * 128,
                                   kOfOut, (begins ? 0 : step) + kk > 0);
              if (t + 1 == tiles) mma_commit<1>(&v_empty[stage]), mma_commit<1>(&done[steps % kAhead]);
              if (!more) mma_commit<1>(&o_full[t]);
            }
            __syncwarp();
            if (more) {
              if (t == 0 && !wait_or_leave(&k_full[next_stage], (steps + 1) / kStages & 1, &gave_up)) return;
              scores(t, next_stage);
              if (t + 1 == tiles) {
                if (elect_one()) mma_commit<1>(&k_empty[next_stage]);
                __syncwarp();
              }
            }
          }
        }
        advance(walk);
      }
    }();
    // what the steps are, by the second
    if (warp == 13) [&] {
      const CacheView& cache = p.cache;
      // A step's place: lane i has the page of tokens 16 (i & 7) on, and where they start in it.  Found
      // two steps ahead, and its scales read one ahead.
      struct Spot {
        int there, page, token;
        bool first;  // of an item
        bool some;   // whether there is such a step
      };
      int far_step = 0;
      const auto look = [&]() -> Spot {
        Spot at{0, -1, 0, false, walk.left > 0};
        if (!at.some) return at;
        const int from = walk.keys.low + (walk.unit + far_step) * kKeys;
        at.there = min(walk.keys.high - from, kKeys), at.first = far_step == 0;
        const int pos = from + 16 * (lane & 7);
        if (pos < walk.keys.high) at.page = page_of(cache, p.at, walk.b, pos);
        at.token = remainder(pos, cache.by_page) + walk.head * cache.page_tokens;
        if (++far_step == piece_units(walk)) advance(walk), far_step = 0;
        return at;
      };
      uint32_t bytes[2];  // scales of tokens 4 lane .. 4 lane + 3
      const auto read_scales = [&](const Spot& at) {
        const int page = __shfl_sync(~0u, at.page, lane >> 2), token = __shfl_sync(~0u, at.token, lane >> 2);
#pragma unroll
        for (int o = 0; o < 2; ++o)
          bytes[o] = page < 0 ? 0
                              : *(const uint32_t*)(cache.scales[o] + page * cache.scale_stride[o] + token + 4 * (lane & 3));
      };
      Spot now = look(), next = look();
      read_scales(now);
      int ref[2] = {0, 0};
#pragma unroll 1
      for (uint32_t steps = 0; now.some; ++steps) {
        Step& to = ring[steps % kAhead];
        const Spot then = look();
        const uint32_t read[2] = {bytes[0], bytes[1]};
        read_scales(next);
        if (!wait_or_leave(&done[steps % kAhead], (steps / kAhead & 1) ^ 1, &gave_up)) return;
        const int there = min(max(now.there - 4 * lane, 0), 4);
        const uint32_t valid = there == 4 ? ~0u : (1u << (8 * there)) - 1u;
        uint32_t bad = 0;  // bytes of tokens that are not numbers
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const uint32_t nan = __vcmpeq4(read[o], ~0u) & valid, clean = read[o] & valid & ~nan;
          bad |= nan;
          uint32_t most = __vmaxu4(clean, clean >> 16);
          most = __reduce_max_sync(~0u, max(most & 255u, most >> 8 & 255u));
          if (now.first || (int)most > ref[o] + 7 - kRaise) ref[o] = (int)most;
          uint32_t f[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = power_f16x2((int)(clean >> (8 * j) & 255u) - ref[o] + kRaise);
          *(uint4*)(to.factors[o] + 4 * lane) = make_uint4(f[0], f[1], f[2], f[3]);
          if (lane < 8)
            to.codes[o][lane] = now.page < 0 ? nullptr : cache.codes[o] + now.page * cache.code_stride[o] + (int64_t)now.token * DIM;
        }
        const bool none = __shfl_sync(~0u, now.page, lane >> 2) < 0 && 16 * (lane >> 2) < now.there;
        const uint32_t special = __ballot_sync(~0u, none || bad);
        if (special) {
          // four bits of a lane's tokens each, eight lanes a word
          uint32_t h = none ? 0xfu : 0u, q = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) q |= (bad >> (8 * j) & 1u) << j;
          h <<= 4 * (lane & 7), q <<= 4 * (lane & 7);
#pragma unroll
          for (int o = 1; o < 8; o *= 2) h |= __shfl_xor_sync(~0u, h, o), q |= __shfl_xor_sync(~0u, q, o);
          if ((lane & 7) == 0) to.hidden[lane >> 3] = h, to.poison[lane >> 3] = q;
        }
        if (lane == 0) to.there = now.there, to.more = next.some, to.key_ref = ref[0], to.value_ref = ref[1], to.special = special != 0;
        __syncwarp();
        mbar_arrive(&known[steps % kAhead], lane == 0);
        now = next, next = then;
      }
    }();
  }

  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (gave_up) drain();
  tmem_fence_after();
  if (warp == 12) tmem_free<1>(tmem, kColumns);
  // what there is to join (warp 14 has kept the share's start and walks it once more)
  if (warp == 14) {
    bool tail = false;
    while (walk.left > 0) {
      if (walk.unit == 0 && piece_units(walk) < walk.units && !gave_up) {
        if (lane == 0) note_tail(walk, blockIdx.x, p.notes);
        tail = true;
      }
      advance(walk);
    }
    if (lane == 0 && !tail) p.notes[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
  }
}

template <int DIM>
cudaError_t launch(const AttentionParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  // The warpgroups' registers come out of what the CTA starts with; with less they would wait for ever.
  static std::atomic<int> registers{0};
  int each = registers.load(std::memory_order_relaxed);
  if (!each) {
    cudaFuncAttributes attributes;
    const cudaError_t err = cudaFuncGetAttributes(&attributes, (const void*)attention_chunk_kernel<DIM>);
    if (err != cudaSuccess) return err;
    registers.store(each = attributes.numRegs, std::memory_order_relaxed);
  }
  if (4 * each < 2 * kSoftmaxRegisters + kOperandRegisters + kProductRegisters) return cudaErrorInvalidConfiguration;
  const int ctas = std::min(multiprocessors(), kMostCtas);
  log_kernel("cache_attention tokens=%d heads=%dx%d dim=%d sequences=%d | rows=%d ctas=%d", p.at.tokens,
             p.cache.heads, p.group, DIM, p.at.sequences, kChunkRows, ctas);
  const cudaError_t err = launch_cluster(attention_chunk_kernel<DIM>, ready, (unsigned)ctas, kThreads,
                                         Layout<DIM>::kBytes, 1, st, p);
  return err == cudaSuccess ? launch_attention_join(p, kChunkRows, ctas, st) : err;
}

}  // namespace

cudaError_t launch_attention_chunk(const AttentionParams& p, cudaStream_t st) {
  return p.dim == 64 ? launch<64>(p, st) : launch<128>(p, st);
}

// Reads and clears this translation unit's device error word (synchronising).
cudaError_t read_device_error_attention(unsigned int* out) {
  const unsigned int zero = 0;
  cudaError_t err = cudaMemcpyFromSymbol(out, g_device_error, sizeof(unsigned int));
  if (err == cudaSuccess && *out)
    err = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(unsigned int));
  return err;
}

}  // namespace ff
}  // namespace fwt
