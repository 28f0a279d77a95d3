// Attention of few rows (new tokens x query heads of a key head) over the 8-bit cache: decoding,
// drafts, any call whose rows do not fill a tensor-memory tile.
//
//   S^T = K Q^T   keys are the 16 lines of a 16 x 8 product, rows its 8 columns
//   p = 2^(s - m), m a running maximum; l = sum of p
//   O^T += V^T P^T   the head dimension is the lines, the contraction runs over keys
//
// Bound: HBM, every byte of the cache seen once.  A warp is on its own: it takes 32 tokens at a time
// through a ring of its own in shared memory that asynchronous copies fill, over items as well, and
// reads the codes straight into the fragments of both products: which elements of a contraction
// meet in which slot is free as long as both operands agree, so a thread takes 16 consecutive bytes
// of a key, and of two values that are neighbours in P one byte each side by side.  Queries and
// outputs are turned in those fragments' layouts too.  (With the warps of a CTA on one item, and their sums
// joined in shared memory, an item cost 15,000 clocks besides its keys: 64 sequences of 256 to 16384 tokens
// 237 us.)  These, 32 query and 8 key heads of 128, now take 100 us, 5.0 TB/s; what is left is the copies'
// own pace (they stall on a full queue, no wait for data) and items of few keys.  One sequence of 4099
// tokens: 19 us in both launches, mostly a chain of lookups (sequence, page, codes) and the join.
//
// Codes become float16 without a rounding; the scales of keys multiply scores, those of values
// multiply p.  P is rounded to float16 as p * 2^(15 + e - e_max), at most 2^15, e the scale's
// exponent and e_max the largest so far: half a unit in 2^-11, down to 2^-29 of the largest possible.
// Queries are rounded to float16 once after their rotation, each row at a power of two that takes
// its largest to 2^14.  (For outputs of float16 both keep what the rounding leaves as a second float16:
// errors against 64 bits are 2.0e-4 then, the output's own rounding, and 3.6e-4 without.)
#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attention_plan.cuh"
#include "cache.cuh"
#include "feed_forward.cuh"
#include "ff_host.cuh"
#include "tma.cuh"

namespace fwt {
namespace ff {
namespace {

constexpr int kWarps = kTokenWorkers, kThreads = kWarps * 32;
constexpr int kStep = 32;   // tokens that a warp takes at a time
// Steps that an item costs besides (64 decoding sequences: 109 us at 0, 102 at 1, 98 at 2).
constexpr int kExtra = 2;
constexpr int kLeast = 4;   // steps of a share: fewer cost more in joining than they save (one sequence of 4099: 20.3 us,
                            // with 2 22.4, 8 22.7, 16 31.0)

template <int DIM>
struct Layout {
  static constexpr int kValues = kStep * DIM, kKeyScales = 2 * kValues, kValueScales = kKeyScales + kStep;
  static constexpr int kStage = kValueScales + kStep;
  static constexpr int kStages = DIM == 128 ? 3 : 6;  // (what fits; 2 measured 2 us less for 64 decoding sequences)
  static constexpr int kRing = kStages * kStage;  // of a warp
  static constexpr int kBytes = kWarps * kRing;
};

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Rows of codes in a stage: 16-byte pieces in an order by row, so that the fragments' reads meet all
// banks (rows 2 c of values, half rows of keys).
template <int DIM>
__device__ __forceinline__ int piece_at(int row, int piece) {
  return row * DIM + ((piece ^ (DIM == 128 ? row & 6 : (row >> 1) & 3)) << 4);
}

// The part of a pair that its rounding to float16 `high` leaves, rounded to float16.
__device__ __forceinline__ uint32_t rest_f16x2(float a, float b, uint32_t high) {
  const float2 h = pair_to_float<__half>(high);
  return pair_from_float<__half>(a - h.x, b - h.y);
}

// NT: groups of 8 rows.  FINE: queries and p as two float16 each, for outputs of float16, whose own half
// unit one rounding of them would pass (64 sequences of 256 to 16384 with float16 queries, 663 MB: 143 us for 129 with
// bfloat16).
template <int DIM, int NT, bool FINE>
__global__ void __launch_bounds__(kThreads, 1) attention_tokens_kernel(const AttentionParams p) {
  using L = Layout<DIM>;
  constexpr int kRows = 8 * NT, kTiles = DIM / 16, kHalves = DIM / 64;
  extern __shared__ __align__(16) uint8_t memory[];
  __shared__ PlanScratch scratch;
  __shared__ Walk walks[kWarps][2];  // of each warp: where it stands, and where its copies do
  __shared__ float sums_top[kWarps][kRows];  // what the sums that wait (kSumKeys) are in units of
  __shared__ int sums_most[kWarps];
  __shared__ float sums_total[kWarps][2 * NT][32];  // each lane's sums of p that wait with them
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  // (the shares of few go to as many multiprocessors as there are)
  const int worker = warp * (int)gridDim.x + (int)blockIdx.x;
  const uint8_t* ring = memory + warp * L::kRing;
  const uint32_t ring_at = smem_u32(ring);
  const CacheView& cache = p.cache;
  pdl_begin();

  // (in shared memory: a step needs little of them)
  Walk &walk = walks[warp][0], &ahead = walks[warp][1];
  {
    const Walk share = find_share<kRows, kStep, kExtra, kLeast, kThreads>(p, worker, kWarps * (int)gridDim.x, scratch);
    if (lane == 0) walk = ahead = share;
    __syncwarp();
  }
  if (walk.left == 0) {
    if (lane == 0) p.notes[2 * worker] = make_int4(0, 0, 0, 0);
    return;
  }
  const auto advance = [&](Walk& w) {
    __syncwarp();
    if (lane == 0) next_piece<kRows, kStep, kExtra>(p, w);
    __syncwarp();
  };

  // The warp's copies run ahead of its work, over items as well: where the next one starts, and ends.
  int pos_ahead = 0, to_ahead = 0, head_ahead = 0;
  bool some = true;       // whether there is a next one
  bool fresh = true;      // whether `ahead` is at an item not looked at yet
  uint32_t present = 0;   // two bits a stage in flight: whether its halves have a page
  int pages = -1;         // lanes 0 and 1: the pages of the next step's halves
  const auto settle = [&] {
    while (true) {
      if (fresh) {
        pos_ahead = ahead.keys.low + ahead.unit * kStep;
        to_ahead = min(pos_ahead + piece_units(ahead) * kStep, ahead.keys.high);
        head_ahead = ahead.head, fresh = false;
      }
      if (pos_ahead < to_ahead) break;
      advance(ahead);
      fresh = true;
      if (ahead.left <= 0) {
        some = false;
        return;
      }
    }
    const int pos = pos_ahead + 16 * (lane & 1);
    pages = pos < to_ahead ? page_of(cache, p.at, ahead.b, pos) : -1;
  };
  const auto fill = [&](int stage) {
    uint32_t bits = 0;
    if (some) {
      const int pos = pos_ahead, to = to_ahead;
      const uint32_t at = ring_at + stage * L::kStage;
      constexpr int kPieces = DIM / 16, kRowsAtOnce = 32 / kPieces;
      const int piece = lane & (kPieces - 1), row0 = lane / kPieces;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int page = __shfl_sync(~0u, pages, half);
        if (page >= 0) bits |= 1u << half;
        const int64_t token = (int64_t)head_ahead * cache.page_tokens + remainder(pos + 16 * half, cache.by_page);
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const uint8_t* codes = cache.codes[o] + page * cache.code_stride[o] + (token + row0) * DIM + 16 * piece;
#pragma unroll
          for (int i = 0; i < 16 / kRowsAtOnce; ++i) {
            const int row = i * kRowsAtOnce + row0;
            const bool there = page >= 0 && pos + 16 * half + row < to;
            copy16(at + (o ? L::kValues : 0) + piece_at<DIM>(16 * half + row, piece),
                   there ? (const void*)(codes + i * kRowsAtOnce * DIM) : p.parts, there);
          }
          if (lane == o)
            copy16(at + (o ? L::kValueScales : L::kKeyScales) + 16 * half,
                   page >= 0 ? (const void*)(cache.scales[o] + page * cache.scale_stride[o] + token) : p.parts,
                   page >= 0);
        }
      }
      pos_ahead += kStep;
      settle();
    }
    present |= bits << (2 * (L::kStages - 1));
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  settle();
#pragma unroll 1
  for (int s = 0; s < L::kStages; ++s) {
    if (s) present >>= 2;
    fill(s);
  }

  int stage = 0;
  bool tail = false;
  while (walk.left > 0) {
    const int piece = piece_units(walk);
    const bool starts = walk.unit == 0, ends = walk.unit + piece == walk.units;
    const int from = walk.keys.low + walk.unit * kStep;
    const int to = min(from + piece * kStep, walk.keys.high);
    const int row0 = walk.block * kRows;  // of the sequence's rows with this head
    const int rows = min(kRows, walk.s.count * p.group - row0);

    // queries: rotated, a power of two for each row, float16; thread (g, c) has of row g the 16
    // elements from 64 j + 16 c on
    uint32_t q[NT][kHalves][8], q_rest[FINE ? NT : 1][kHalves][8];
    float scale[NT][2];
    Keys seen[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + g, bits = p.rot_bits;
      const float before = rotation_before(bits), norm = rotation_after(bits);
      float v[kHalves * 16];
#pragma unroll
      for (int i = 0; i < kHalves * 16; ++i) v[i] = 0.f;
      if (r < rows) {
        const int token = walk.s.row + quotient(row0 + r, p.by_group);
        const int head = walk.head * p.group + remainder(row0 + r, p.by_group);
        const uint16_t* from_q = (const uint16_t*)p.q.p + token * p.q.token + head * p.q.head + 16 * c;
#pragma unroll
        for (int i = 0; i < kHalves * 2; ++i) {
          const uint4 w = *(const uint4*)(from_q + (i >> 1) * 64 + (i & 1) * 8);
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = pair_to_float(x[k], p.type);
            v[8 * i + 2 * k] = f.x * before, v[8 * i + 2 * k + 1] = f.y * before;
          }
        }
      }
      if (bits > 0) turn_own<kHalves * 16, 1>(v);
      if (bits > 1) turn_own<kHalves * 16, 2>(v);
      if (bits > 2) turn_own<kHalves * 16, 4>(v);
      if (bits > 3) turn_own<kHalves * 16, 8>(v);
      if (bits > 4) turn_lanes(v, 1, lane);
      if (bits > 5) turn_lanes(v, 2, lane);
      if constexpr (DIM == 128)
        if (bits > 6) turn_own<kHalves * 16, 16>(v);
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < kHalves * 16; ++i) {
        v[i] *= norm;
        most = max(most, __float_as_uint(v[i]) & 0x7fffffffu);
      }
      most = max(most, __shfl_xor_sync(~0u, most, 1));
      most = max(most, __shfl_xor_sync(~0u, most, 2));
      const int e = max((int)(most >> 23), 27);  // (zero, and what is nearly so)
      const float up = __uint_as_float((uint32_t)(254 + 14 - e) << 23);
#pragma unroll
      for (int i = 0; i < kHalves * 8; ++i) {
        q[n][i / 8][i & 7] = pair_from_float<__half>(v[2 * i] * up, v[2 * i + 1] * up);
        if constexpr (FINE) q_rest[n][i / 8][i & 7] = rest_f16x2(v[2 * i] * up, v[2 * i + 1] * up, q[n][i / 8][i & 7]);
      }
      const float mine = p.scale * __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {  // of the rows that the scores' fragment has here
        scale[n][e2] = __shfl_sync(~0u, mine, 4 * (2 * c + e2));
        const int r2 = 8 * n + 2 * c + e2;
        seen[n][e2] = r2 < rows ? seen_by(p, walk.s, row0 + r2) : Keys{0, 0};
      }
    }
    float top[NT][2], total[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) top[n][e] = -INFINITY, total[n][e] = 0.f;
    float o[kTiles][NT][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    int most = 0;  // the largest scale byte of the values so far
    float* part = p.parts + (2 * (int64_t)worker + (starts ? 1 : 0)) * part_floats(kRows, DIM);
    // The sums together with those that wait, if any, in the present units: to wait in turn, or for good.
    const auto add_sums = [&](bool some, bool wait) {
      float f[NT][2];
      const float less = __uint_as_float((uint32_t)max(some ? 127 + sums_most[warp] - most : 0, 0) << 23);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float before = sums_top[warp][8 * n + 2 * c + e];
          const float f_e = before == -INFINITY ? 1.f : exp2_fast(before - top[n][e]);
          float& waits = sums_total[warp][2 * n + e][lane];
          if (some) total[n][e] = fmaf(waits, f_e, total[n][e]);
          if (wait) waits = total[n][e], total[n][e] = 0.f;
          f[n][e] = f_e * less;
        }
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float4* at = (float4*)part + (i * NT + n) * 32 + lane;
          if (some) {
            const float4 x = *at;
            o[i][n][0] = fmaf(x.x, f[n][0], o[i][n][0]), o[i][n][1] = fmaf(x.y, f[n][1], o[i][n][1]);
            o[i][n][2] = fmaf(x.z, f[n][0], o[i][n][2]), o[i][n][3] = fmaf(x.w, f[n][1], o[i][n][3]);
          }
          if (wait) {
            *at = make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
            o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
          }
        }
      __syncwarp();  // (and the part's rows are written over other lanes' sums)
      if (wait) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (g == 0) sums_top[warp][8 * n + 2 * c + e] = top[n][e];
        if (lane == 0) sums_most[warp] = most;
        __syncwarp();
      }
    };

    for (int pos = from; pos < to; pos += kStep) {
      asm volatile("cp.async.wait_group %0;" ::"n"(L::kStages - 1) : "memory");
      __syncwarp();
      const uint8_t* at = ring + stage * L::kStage;
      const uint32_t here = present & 3u;
      float s[2][NT][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.f;
        // (halves in the other order for odd rows: their pieces then lie in other banks)
        uint4 k[2][DIM / 64];
#pragma unroll
        for (int j = 0; j < DIM / 64; ++j) {
          const int half = DIM == 128 ? j ^ (g & 1) : j;
          k[0][j] = *(const uint4*)(at + piece_at<DIM>(16 * t + g, 4 * half + c));
          k[1][j] = *(const uint4*)(at + piece_at<DIM>(16 * t + g + 8, 4 * half + c));
        }
        if (DIM == 128 && (g & 1)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint4 w = k[r][0];
            k[r][0] = k[r][DIM / 64 - 1], k[r][DIM / 64 - 1] = w;
          }
        }
#pragma unroll
        for (int j = 0; j < DIM / 64; ++j) {
          const uint32_t lo[4] = {k[0][j].x, k[0][j].y, k[0][j].z, k[0][j].w};
          const uint32_t hi[4] = {k[1][j].x, k[1][j].y, k[1][j].z, k[1][j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = e4m3_to_f16x2(lo[i]), a2 = e4m3_to_f16x2(lo[i] >> 16);
            const uint32_t a1 = e4m3_to_f16x2(hi[i]), a3 = e4m3_to_f16x2(hi[i] >> 16);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_f16(s[t][n], a0, a1, a2, a3, q[n][j][2 * i], q[n][j][2 * i + 1]);
              if constexpr (FINE) mma_f16(s[t][n], a0, a1, a2, a3, q_rest[n][j][2 * i], q_rest[n][j][2 * i + 1]);
            }
          }
        }
      }
      // this thread's tokens: pos + 16 t + 8 h + g
      float key_scale[2][2];
      int value_byte[2][2], largest = 0;
      bool there[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int token = 16 * t + 8 * h + g;
          there[t][h] = (here >> t & 1u) && pos + token < to;
          key_scale[t][h] = scale_value(at[L::kKeyScales + token]);
          value_byte[t][h] = there[t][h] ? at[L::kValueScales + token] : 0;
          // (a value that is not a number: so is the score, for whoever sees it)
          if (value_byte[t][h] == 255) key_scale[t][h] = scale_value(255), value_byte[t][h] = 0;
          largest = max(largest, value_byte[t][h]);
        }
      largest = (int)__reduce_max_sync(~0u, (unsigned)largest);
      bool moved = largest > most;
      const float less = moved ? __uint_as_float((uint32_t)max(127 + most - largest, 0) << 23) : 1.f;
      most = max(most, largest);
      float keep[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = -INFINITY;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int token = pos + 16 * t + 8 * h + g;
              float& v = s[t][n][2 * h + e];
              v = there[t][h] && token >= seen[n][e].low && token < seen[n][e].high
                      ? v * (scale[n][e] * key_scale[t][h])  // (v is up to 2^30, and v times one of them may pass fp32)
                      : -INFINITY;
              x = fmaxf(x, v);
            }
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
          x = fmaxf(x, top[n][e]);
          const float base = x == -INFINITY ? 0.f : x;
          keep[n][e] = exp2_fast(top[n][e] - base);
          moved |= x > top[n][e];
          top[n][e] = x;
          total[n][e] *= keep[n][e];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& v = s[t][n][2 * h + e];
              v = exp2_fast(v - base);
              total[n][e] += v;
            }
        }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][n][e] *= keep[n][e & 1] * less;
      }
      // p with the values' scales, as the second product's columns
      uint32_t b[2][NT][2], b_rest[2][FINE ? NT : 1][2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float f = __uint_as_float((uint32_t)max(127 + 15 + value_byte[t][h] - most, 0) << 23);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint32_t high = pair_from_float<__half>(s[t][n][2 * h] * f, s[t][n][2 * h + 1] * f);
            b[t][n][h] = transpose8x8(high);
            if constexpr (FINE) b_rest[t][n][h] = transpose8x8(rest_f16x2(s[t][n][2 * h] * f, s[t][n][2 * h + 1] * f, high));
          }
        }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint32_t v[4][DIM / 32];  // tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9: DIM / 8 bytes from DIM / 8 g on
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * t + 2 * c + (i & 1) + 8 * (i >> 1);
          const uint8_t* values = at + L::kValues;
          if constexpr (DIM == 128) {
            const uint4 w = *(const uint4*)(values + piece_at<DIM>(row, g));
            v[i][0] = w.x, v[i][1] = w.y, v[i][2] = w.z, v[i][3] = w.w;
          } else {
            const uint2 w = *(const uint2*)(values + piece_at<DIM>(row, g >> 1) + 8 * (g & 1));
            v[i][0] = w.x, v[i][1] = w.y;
          }
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          const uint32_t pick = i & 1 ? 0x7362u : 0x5140u;
          const uint32_t w0 = __byte_perm(v[0][i / 2], v[1][i / 2], pick);
          const uint32_t w1 = __byte_perm(v[2][i / 2], v[3][i / 2], pick);
          const uint32_t a0 = e4m3_to_f16x2(w0), a1 = e4m3_to_f16x2(w0 >> 16);
          const uint32_t a2 = e4m3_to_f16x2(w1), a3 = e4m3_to_f16x2(w1 >> 16);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(o[i][n], a0, a1, a2, a3, b[t][n][0], b[t][n][1]);
            if constexpr (FINE) mma_f16(o[i][n], a0, a1, a2, a3, b_rest[t][n][0], b_rest[t][n][1]);
          }
        }
      }
      if ((pos + kStep - from) % kSumKeys == 0 && pos + kStep < to) add_sums(pos + kStep - from > kSumKeys, true);
      __syncwarp();
      present >>= 2;
      fill(stage);
      if (++stage == L::kStages) stage = 0;
    }

    if (to - from > kSumKeys) add_sums(true, false);

    // out: the item's rows, or a part of them for launch_attention_join.  Thread (g, c) has of rows
    // 2 c and 2 c + 1 the DIM / 8 elements from DIM / 8 g on.
    const bool whole = starts && ends;
    // 2^e, e from -142 to 112, in two factors
    const int e = most - 142, half_e = e >> 1;
    const float unit[2] = {__uint_as_float((uint32_t)(127 + half_e) << 23), __uint_as_float((uint32_t)(127 + e - half_e) << 23)};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = 8 * n + 2 * c + k;
        float l = total[n][k];
        l += __shfl_xor_sync(~0u, l, 4);
        l += __shfl_xor_sync(~0u, l, 8);
        l += __shfl_xor_sync(~0u, l, 16);
        // (in units of the scales up to the end: sums of values and of rows may pass fp32 where the output does not)
        const int bits = p.rot_bits;
        const float norm = l == 0.f ? 0.f : (whole ? rotation_norm(bits) : 1.f) / l;
        float v[DIM / 8];
#pragma unroll
        for (int i = 0; i < DIM / 8; ++i) v[i] = o[i / 2][n][2 * (i & 1) + k] * norm;
        if (whole) {
          constexpr int kOwn = DIM == 128 ? 4 : 3;  // bits of a thread's own elements
          if (bits > 0) turn_own<DIM / 8, 1>(v);
          if (bits > 1) turn_own<DIM / 8, 2>(v);
          if (bits > 2) turn_own<DIM / 8, 4>(v);
          if constexpr (DIM == 128)
            if (bits > 3) turn_own<DIM / 8, 8>(v);
#pragma unroll
          for (int bit = 0; bit < 3; ++bit)
            if (bits > kOwn + bit) turn_lanes(v, 4 << bit, lane);
        }
#pragma unroll
        for (int i = 0; i < DIM / 8; ++i) v[i] = v[i] * unit[0] * unit[1];
        if (whole) {
          if (r < rows) {
            const int token = walk.s.row + quotient(row0 + r, p.by_group);
            const int head = walk.head * p.group + remainder(row0 + r, p.by_group);
            uint16_t* to_out = (uint16_t*)p.out.p + token * p.out.token + head * p.out.head + DIM / 8 * g;
#pragma unroll
            for (int i = 0; i < DIM / 64; ++i) {
              uint32_t x[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = pair_from_float(v[8 * i + 2 * j], v[8 * i + 2 * j + 1], p.type);
              *(uint4*)(to_out + 8 * i) = make_uint4(x[0], x[1], x[2], x[3]);
            }
          }
        } else if (r < rows) {
          float4* to_part = (float4*)(part + r * DIM + DIM / 8 * g);
#pragma unroll
          for (int i = 0; i < DIM / 32; ++i) to_part[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          if (g == 0) part[kRows * DIM + r] = top[n][k], part[kRows * DIM + kRows + r] = l;
        }
      }
    if (starts && !ends) {  // (the last)
      if (lane == 0) note_tail(walk, worker, p.notes);
      tail = true;
    }
    advance(walk);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (lane == 0 && !tail) p.notes[2 * worker] = make_int4(0, 0, 0, 0);
}

template <int DIM, int NT, bool FINE>
cudaError_t launch(const AttentionParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  const int ctas = std::min(multiprocessors(), kMostCtas);
  log_kernel("cache_attention tokens=%d heads=%dx%d dim=%d sequences=%d | rows=%d ctas=%d", p.at.tokens,
             p.cache.heads, p.group, DIM, p.at.sequences, 8 * NT, ctas);
  const cudaError_t err = launch_cluster(attention_tokens_kernel<DIM, NT, FINE>, ready, (unsigned)ctas, kThreads,
                                         Layout<DIM>::kBytes, 1, st, p);
  return err == cudaSuccess ? launch_attention_join(p, 8 * NT, kWarps * ctas, st) : err;
}
template <int DIM>
cudaError_t launch_rows(const AttentionParams& p, int rows, cudaStream_t st) {
  if (p.type == FWT_F16) return rows == 8 ? launch<DIM, 1, true>(p, st) : launch<DIM, 2, true>(p, st);
  return rows == 8 ? launch<DIM, 1, false>(p, st) : launch<DIM, 2, false>(p, st);
}

}  // namespace

cudaError_t launch_attention_tokens(const AttentionParams& p, int rows, cudaStream_t st) {
  return p.dim == 64 ? launch_rows<64>(p, rows, st) : launch_rows<128>(p, rows, st);
}

}  // namespace ff
}  // namespace fwt
