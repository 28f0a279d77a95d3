// Rotation and quantisation to 8-bit floating point with a scale for each block of 128.
//
// A warp owns 16 lines by one block of 128 elements along the axis.  The rotation of a
// group of 2^r <= 128 elements is a Kronecker product of 2 x 2 factors, one for each
// index bit below r, so its factors may be applied in any order and by different means:
//
//   bits 0, 1, 3, 4   one m16n8k16 matrix product of 16 lines by 16 elements with the
//                     16 x 16 matrix of signs (zeros where an index bit stays as it is).
//                     Signs and inputs are exact in 16 bits and the sums fp32; an fp32
//                     input goes in as three bf16 pieces that add up to it exactly (bf16
//                     ends at 2^-133: a line's block below 2^-64 goes in times 2^64).
//   bits 2, 5, 6      additions between the thread's own registers.
//
// Elements are assigned to the product's slots so that a thread holds the same elements
// before and after it: 8 consecutive ones (bits 0..2) in each of the four groups of 32
// (bits 5, 6), the lanes t = 0..3 of a quad being bits 3 and 4, for the lines g = lane / 4
// and g + 8.  So inputs are 16-byte loads, codes 8-byte stores, and only the maximum of a
// block crosses lanes (two shuffles a line, where butterflies across lanes would take four
// shuffles an element and be bound by them).
//
// Bound: HBM by its bytes, issue and the latency of dependent instructions as it stands (48% of
// the issue slots, 12 to 16 warps an SM): 8192 x 8192 bf16 in 39.5 us along the columns and 36.5
// down the rows, 5.1 and 5.5 TB/s, with 128 lines to a scale 39 and 40.4; one line of 8192 2.0 us,
// the launch.  fp32 (eight warps an SM, no block ahead): 90 and 125 us, with 128 lines 98 and 118,
// 2.7 to 3.7 TB/s.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "feed_forward.cuh"
#include "ff_host.cuh"
#include "fwt.h"
#include "tma.cuh"

namespace fwt {
namespace ff {
namespace {

struct QuantizeParams {
  const void* x;
  int64_t ld_x;
  uint8_t* q;
  int64_t ld_q;
  float* scale;
  int64_t ld_scale;
  int nl, length, full;  // lines, elements along the axis, and these with the zeros
  int blocks, strips;    // blocks of 128 along the axis, strips of 16 lines
  int r;
  float norm;  // 2^(-r/2)
  float norm_448;  // 2^(-r/2) / 448
  int rounds;  // blocks a warp goes through
  int vec;     // rows of x start on 16-byte boundaries (axis 0: on two elements')
  int vec16;   // on 16-byte boundaries, whichever axis
};

// d = a b (FIRST) or d + a b.
template <typename T, bool FIRST>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  const float c[4] = {FIRST ? 0.f : d[0], FIRST ? 0.f : d[1], FIRST ? 0.f : d[2], FIRST ? 0.f : d[3]};
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
        " {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
        " {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
}

// The type the product runs in and the pieces an input is split into.
template <typename T>
struct Input {
  using Mma = T;
  static constexpr int kPieces = 1;
};
template <>
struct Input<float> {
  using Mma = __nv_bfloat16;
  static constexpr int kPieces = 3;
};

// One sign of the 16 x 16 matrix as a 16-bit value: elements ek (in) and en (out).
template <typename M>
__device__ __forceinline__ uint32_t sign16(int ek, int en, int r) {
  const int low = (1 << r) - 1;
  if ((ek ^ en) & ~low) return 0;
  constexpr uint32_t one = sizeof(M) == 2 && std::is_same<M, __half>::value ? 0x3c00u : 0x3f80u;
  return one | ((__popc(ek & en & low) & 1) << 15);
}

// max(|a|, b), NaN if either is.
__device__ __forceinline__ float max_magnitude(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(fabsf(a)), "f"(b));
  return d;
}

// The largest of |a|, |b| and |c|, NaN if one of them is.
__device__ __forceinline__ float max_magnitude(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// What a thread loads of one block: 8 consecutive elements in each group of 32 of its two
// lines.  Axis 1: lines g and g + 8 of the strip, 16 bytes along a row at a time.  Axis 0:
// lines 2 g and 2 g + 1, which lie side by side in every row of x, both with one load.
template <typename T, int AXIS>
struct Block {
  uint32_t w[4][2 * sizeof(T)][2];  // group; axis 1: words of a line, line; axis 0: see below

  static __device__ __forceinline__ int line(int strip, int g, int s) {
    return strip * 16 + (AXIS == 1 ? g + 8 * s : 2 * g + s);
  }

  // Zero outside the matrix.
  __device__ __forceinline__ void load(const QuantizeParams& p, int strip, int block, int g, int t) {
    constexpr int kWords = 2 * (int)sizeof(T);  // 32-bit words of 8 elements
    const T* x = (const T*)p.x;
#pragma unroll
    for (int grp = 0; grp < 4; ++grp) {
      const int pos = block * 128 + 32 * grp + 8 * t;
      if constexpr (AXIS == 1) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int l = line(strip, g, s);
          const T* from = x + (int64_t)l * p.ld_x + pos;
          if (sizeof(T) == 4 && p.vec && l < p.nl && pos + 8 <= p.length) {  // (16 bits: staged)
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
              const uint4 v = ((const uint4*)from)[i / 4];
              w[grp][i][s] = v.x, w[grp][i + 1][s] = v.y, w[grp][i + 2][s] = v.z, w[grp][i + 3][s] = v.w;
            }
          } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[grp][i][s] = 0;
            if (l < p.nl) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (pos + j < p.length) {
                  if constexpr (sizeof(T) == 2)
                    w[grp][j / 2][s] |= (uint32_t)((const unsigned short*)from)[j] << (16 * (j & 1));
                  else
                    w[grp][j][s] = ((const uint32_t*)from)[j];
                }
            }
          }
        }
      } else {
        // element j of both lines: one word (16-bit types, w[..][j / 2][j & 1]) or two
        const int l = line(strip, g, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const T* from = x + (int64_t)(pos + j) * p.ld_x + l;
          const bool in = pos + j < p.length;
          if constexpr (sizeof(T) == 2) {
            uint32_t v = 0;
            if (p.vec && in && l + 1 < p.nl) {
              v = *(const uint32_t*)from;
            } else {
              if (in && l < p.nl) v = *(const unsigned short*)from;
              if (in && l + 1 < p.nl) v |= (uint32_t)((const unsigned short*)from)[1] << 16;
            }
            w[grp][j / 2][j & 1] = v;
          } else {
            uint2 v = make_uint2(0, 0);
            if (p.vec && in && l + 1 < p.nl) {
              v = *(const uint2*)from;
            } else {
              if (in && l < p.nl) v.x = *(const uint32_t*)from;
              if (in && l + 1 < p.nl) v.y = ((const uint32_t*)from)[1];
            }
            w[grp][j][0] = v.x, w[grp][j][1] = v.y;
          }
        }
      }
    }
  }

  // fp32 lines whose values in this block are all below 2^-64, times 2^64: an element's pieces end
  // 2^-24 below it, and bf16 at 2^-133.  (In other lines what is lost there is 2^-69 of the
  // largest.)  undo: 2^-64 for such lines, else 1.  (8192 x 8192 87 -> 90.5 us along the columns, 118
  // -> 125 down the rows; to look at the rotated values and go back where they are small cost as much.)
  __device__ __forceinline__ void lift(float (&undo)[2]) {
    static_assert(sizeof(T) == 4, "16-bit inputs are their own pieces");
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float top = 0.f;
#pragma unroll
      for (int grp = 0; grp < 4; ++grp)
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          top = max_magnitude(__uint_as_float(w[grp][j][s]), __uint_as_float(w[grp][j + 1][s]), top);
      top = max_magnitude(__shfl_xor_sync(~0u, top, 1), top);
      top = max_magnitude(__shfl_xor_sync(~0u, top, 2), top);
      const bool small = top < 0x1p-64f && top != 0.f;
      undo[s] = small ? 0x1p-64f : 1.f;
      if (__any_sync(~0u, small)) {
        const float up = small ? 0x1p64f : 1.f;
#pragma unroll
        for (int grp = 0; grp < 4; ++grp)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            w[grp][j][s] = __float_as_uint(__uint_as_float(w[grp][j][s]) * up);
      }
    }
  }

  // Elements 2 i and 2 i + 1 of a group of line s, as 16-bit pairs: the k-th piece.  An fp32
  // input is taken apart as it is read: call with k = 0, 1, 2 in turn.  Truncation leaves no
  // piece larger than its input, and 8 + 8 + 8 significant bits hold it exactly.
  __device__ __forceinline__ uint32_t pair(int grp, int i, int s) {
    if constexpr (sizeof(T) == 2) {
      if constexpr (AXIS == 1) return w[grp][i][s];
      else return __byte_perm(w[grp][i][0], w[grp][i][1], s ? 0x7632 : 0x5410);
    } else {
      uint32_t &lo = w[grp][2 * i][s], &hi = w[grp][2 * i + 1][s];
      const uint32_t top_lo = lo & 0xffff0000u, top_hi = hi & 0xffff0000u;
      lo = __float_as_uint(__uint_as_float(lo) - __uint_as_float(top_lo));
      hi = __float_as_uint(__uint_as_float(hi) - __uint_as_float(top_hi));
      return (top_lo >> 16) | top_hi;
    }
  }
};

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// 16-bit inputs whose rows are 16-byte aligned take another way in: asynchronous 16-byte copies
// bring blocks ahead to shared memory, where they cost no registers (loaded to registers, a
// block ahead, the warps an SM holds had too few bytes on their way: 8192 x 8192 took 42.9 us
// along the columns and 53 down the rows).
//
// Along the columns each warp has its own stages: 16 rows of 256 bytes, the halves of every 128
// swapped in odd rows so that the reads (64 bytes of two rows at a time) meet all banks.
__device__ __forceinline__ uint32_t row_at(int row, int chunk) {
  return (uint32_t)(row * 256 + ((chunk ^ ((row & 1) << 2)) << 4));
}
__device__ __forceinline__ void copy16(uint32_t to, const QuantizeParams& p, int64_t element, int valid) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(to),
               "l"((const uint8_t*)p.x + (valid ? element * 2 : 0)), "r"(valid)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t to, const uint8_t* from) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void stage_rows(const QuantizeParams& p, uint32_t to, int strip, int block) {
  const int lane = threadIdx.x & 31, chunk = lane & 15, col = block * 128 + 8 * chunk;
  if (block * 128 + 128 <= p.length && strip * 16 + 16 <= p.nl) {  // all of it is there
    const uint8_t* from = (const uint8_t*)p.x + ((strip * 16 + (lane >> 4)) * p.ld_x + col) * 2;
    const int64_t step = p.ld_x * 4;
    to += row_at(lane >> 4, chunk);
#pragma unroll
    for (int i = 0; i < 8; ++i, from += step) copy16(to + i * 512, from);
    return;
  }
  const int bytes = 2 * min(8, max(0, p.length - col));  // (of a length times two, 31 bits are too few)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = 2 * i + (lane >> 4), line = strip * 16 + row;
    copy16(to + row_at(row, chunk), p, (int64_t)line * p.ld_x + col, line < p.nl ? bytes : 0);
  }
}
// Down the rows the CTA has stages in common: 128 rows of its lines (16 a warp), 32 W bytes
// apart, which go into the product's slots transposed.  The chunks are swizzled so that the
// eight rows that one 8 x 8 matrix takes (0, 1, 8, 9, 16, ...) meet different banks.
template <int W>
__device__ __forceinline__ uint32_t column_at(int pos, int chunk) {
  return (uint32_t)(pos * 2 * W + (chunk ^ ((pos & 1) | ((pos >> 2) & 6)))) * 16;
}
template <int W>
__device__ __forceinline__ void stage_columns(const QuantizeParams& p, uint32_t to, int line0, int block) {
  constexpr int kChunks = 2 * W;
  const int chunk = threadIdx.x % kChunks, line = line0 + 8 * chunk;
  if (block * 128 + 128 <= p.length && line0 + 16 * W <= p.nl) {
    const int pos = threadIdx.x / kChunks;
    const uint8_t* from = (const uint8_t*)p.x + ((int64_t)(block * 128 + pos) * p.ld_x + line) * 2;
    const int64_t step = p.ld_x * 32;
#pragma unroll
    for (int i = 0; i < 8; ++i, from += step) copy16(to + column_at<W>(pos + 16 * i, chunk), from);
    return;
  }
  const int bytes = 2 * min(8, max(0, p.nl - line));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int pos = i * 16 + threadIdx.x / kChunks, row = block * 128 + pos;
    copy16(to + column_at<W>(pos, chunk), p, (int64_t)row * p.ld_x + line, row < p.length ? bytes : 0);
  }
}

// Warps of a CTA: consecutive blocks of one strip (axis 1) or consecutive strips (axis 0), so
// that a CTA reads long runs of rows; with 128 lines to a scale, the eight strips of one tile.
// Each then goes on along the axis, `rounds` blocks in all, the loads of the next block on
// their way while one is worked on.
template <int LINES>
constexpr int kWarps = LINES == 1 ? 4 : 8;

// CTAs that an SM is to hold: 16 warps of 128 registers (16-bit inputs; 0.2 to 1.2 us of 15 to
// 39 faster than as many registers as the compiler takes), but for the rows' own scales, where
// those 137 measured 41.4 us against 44.4 for 8192 x 8192.
template <typename T, int AXIS, int LINES>
constexpr int kLeast = sizeof(T) == 2 && !(AXIS == 1 && LINES == 1) ? 16 / kWarps<LINES> : 1;

template <int AXIS, int LINES>
struct Stages {
  static constexpr int kCount = AXIS == 1 && LINES == 1 ? 3 : 2;
  static constexpr size_t kBytes = (size_t)kCount * kWarps<LINES> * 4096;
};

template <typename T, int AXIS, int LINES, bool STAGED>
__global__ void __launch_bounds__(kWarps<LINES> * 32, kLeast<T, AXIS, LINES>)
    quantize_kernel(QuantizeParams p) {
  constexpr int W = kWarps<LINES>;
  constexpr bool kAhead = sizeof(T) == 2 && !STAGED;  // fp32 blocks take twice the registers
  constexpr int kStaged = AXIS == 1 ? 4096 : 128 * 32 * W;  // bytes of a stage (axis 1: a warp's)
  constexpr int kStages = Stages<AXIS, LINES>::kCount;
  extern __shared__ __align__(128) uint8_t staged[];
  constexpr int kStep = AXIS == 1 && LINES == 1 ? W : 1;
  using M = typename Input<T>::Mma;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int per = (p.blocks + kStep * p.rounds - 1) / (kStep * p.rounds);  // CTAs along the axis
  int block = blockIdx.x % per * (kStep * p.rounds);
  int strip = blockIdx.x / per;
  if constexpr (kStep == W) block += warp;
  else strip = strip * W + warp;
  if (!(STAGED && AXIS == 0) && LINES == 1 && (block >= p.blocks || strip >= p.strips)) {
    pdl_begin();
    return;
  }
  const int end = min(p.blocks, block + kStep * p.rounds);

  uint32_t b[2][2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int en = 8 * (g >> 1) + (g & 1) + 2 * n;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      b[n][h] = sign16<M>(8 * t + 2 * h, en, p.r) | (sign16<M>(8 * t + 2 * h + 1, en, p.r) << 16);
  }
  const int lines[2] = {STAGED ? strip * 16 + g : Block<T, AXIS>::line(strip, g, 0),
                        STAGED ? strip * 16 + g + 8 : Block<T, AXIS>::line(strip, g, 1)};

  Block<T, AXIS> x;
  pdl_begin();
  const uint32_t buffers = STAGED ? smem_u32(staged) + (AXIS == 1 ? warp * kStages * kStaged : 0) : 0;
  auto stage = [&](int round, int at) {
    if (at < end) {
      const uint32_t to = buffers + round % kStages * kStaged;
      if constexpr (AXIS == 1) stage_rows(p, to, strip, at);
      else stage_columns<W>(p, to, (strip - warp) * 16, at);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if constexpr (STAGED) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) stage(i, block + i * kStep);
  } else {
    x.load(p, strip, block, g, t);
  }
  for (int round = 0; block < end; block += kStep, ++round) {
    float y[4][2][2][4];  // group of 32, bit 2, bit 1, (line, bit 0)
    float undo[2] = {1.f, 1.f};  // what takes y back to its size
    if constexpr (sizeof(T) == 4) x.lift(undo);
    const int now = round % kStages * kStaged;
    if constexpr (STAGED) {
      stage(round + kStages - 1, block + (kStages - 1) * kStep);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      if constexpr (AXIS == 1) __syncwarp();
      else __syncthreads();
    }
#pragma unroll
    for (int grp = 0; grp < 4; ++grp) {
      uint4 lo, hi;
      if constexpr (STAGED && AXIS == 1) {
        const uint8_t* from = staged + (buffers - smem_u32(staged)) + now;
        lo = *(const uint4*)(from + row_at(g, 4 * grp + t));
        hi = *(const uint4*)(from + row_at(g + 8, 4 * grp + t));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int k = 0; k < Input<T>::kPieces; ++k) {
          uint32_t a[4];
          if constexpr (STAGED && AXIS == 1) {
            a[0] = h ? lo.z : lo.x, a[1] = h ? hi.z : hi.x, a[2] = h ? lo.w : lo.y, a[3] = h ? hi.w : hi.y;
          } else if constexpr (STAGED) {
            // lane -> a row of one of four 8 x 8 matrices: elements 0, 1 or 2, 3 (lanes 16 on)
            // of each thread's four, lines 0..7 or 8..15 (odd eights of lanes)
            const int pos = 32 * grp + 4 * h + 8 * ((lane & 7) >> 1) + 2 * (lane >> 4) + (lane & 1);
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                         : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                         : "r"(buffers + now + column_at<W>(pos, 2 * warp + ((lane >> 3) & 1)))
                         : "memory");
          } else {
            a[0] = x.pair(grp, 2 * h, 0), a[1] = x.pair(grp, 2 * h, 1);
            a[2] = x.pair(grp, 2 * h + 1, 0), a[3] = x.pair(grp, 2 * h + 1, 1);
          }
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (k == 0) mma16<M, true>(y[grp][h][n], a, b[n]);
            else mma16<M, false>(y[grp][h][n], a, b[n]);
          }
        }
      }
    }
    // the next round's copies overwrite the stage that was read the longest ago: this one
    if constexpr (STAGED && AXIS == 1) __syncwarp();
    else if constexpr (STAGED) __syncthreads();
    if (kAhead && block + kStep < end) x.load(p, strip, block + kStep, g, t);

    if (p.r > 2) {
#pragma unroll
      for (int grp = 0; grp < 4; ++grp)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float lo = y[grp][0][n][i], hi = y[grp][1][n][i];
            y[grp][0][n][i] = lo + hi, y[grp][1][n][i] = lo - hi;
          }
    }
#pragma unroll
    for (int bit = 1; bit < 4; bit <<= 1)
      if (p.r > (bit == 1 ? 5 : 6)) {
#pragma unroll
        for (int grp = 0; grp < 4; ++grp)
          if (!(grp & bit))
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float lo = y[grp][h][n][i], hi = y[grp | bit][h][n][i];
                  y[grp][h][n][i] = lo + hi, y[grp | bit][h][n][i] = lo - hi;
                }
      }

    // 2^(-r/2) is left to the scale: |y| is the largest where the normalised value is
    float top[2] = {0.f, 0.f};
#pragma unroll
    for (int grp = 0; grp < 4; ++grp)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int s = 0; s < 2; ++s)
            top[s] = max_magnitude(y[grp][h][n][2 * s], y[grp][h][n][2 * s + 1], top[s]);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      top[s] = max_magnitude(__shfl_xor_sync(~0u, top[s], 1), top[s]);
      top[s] = max_magnitude(__shfl_xor_sync(~0u, top[s], 2), top[s]);
      if constexpr (sizeof(T) == 4) top[s] *= undo[s];
    }
    if constexpr (LINES == 128) {
      __shared__ float tops[2][W];  // in turn: a warp may be a round ahead of another
      float m = max_magnitude(top[0], top[1]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) m = max_magnitude(__shfl_xor_sync(~0u, m, o), m);
      if (lane == 0) tops[round & 1][warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) m = max_magnitude(tops[round & 1][w], m);
      top[0] = top[1] = m;
    }

    float scales[2], factors[2];
#pragma unroll
    for (int s = 0; s < (LINES == 128 ? 1 : 2); ++s) {
      // s = top norm / 448, and norm / s: above the least scale the norm cancels
      scales[s] = fmaxf(top[s] * p.norm_448, 0x1p-126f);
      factors[s] = scales[s] <= 0x1p-126f ? p.norm * 0x1p126f : __fdiv_rn(448.f, top[s]);
      if (!(top[s] < INFINITY)) scales[s] = factors[s] = __uint_as_float(0x7fffffffu);
    }
    if constexpr (LINES == 128) scales[1] = scales[0], factors[1] = factors[0];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bool whole = block * 128 + 128 <= p.full;
      const float scale = scales[s], factor = sizeof(T) == 4 ? factors[s] * undo[s] : factors[s];
      const int l = lines[s];
      if (LINES == 1 ? t == 0 && l < p.nl : threadIdx.x == 0 && s == 0)
        p.scale[(int64_t)(LINES == 1 ? l : l / 128) * p.ld_scale + block] = scale;
      if (l < p.nl) {
        uint8_t* q = p.q + (int64_t)l * p.ld_q;
#pragma unroll
        for (int grp = 0; grp < 4; ++grp) {
          uint2 code;
          code.x = codes4(y[grp][0][0][2 * s] * factor, y[grp][0][0][2 * s + 1] * factor,
                          y[grp][0][1][2 * s] * factor, y[grp][0][1][2 * s + 1] * factor);
          code.y = codes4(y[grp][1][0][2 * s] * factor, y[grp][1][0][2 * s + 1] * factor,
                          y[grp][1][1][2 * s] * factor, y[grp][1][1][2 * s + 1] * factor);
          const int at = block * 128 + 32 * grp + 8 * t;
          if (whole || at + 8 <= p.full) {
            *(uint2*)(q + at) = code;
          } else {
            for (int j = 0; j < 8 && at + j < p.full; ++j)
              q[at + j] = (uint8_t)((j < 4 ? code.x : code.y) >> (8 * (j & 3)));
          }
        }
      }
      __syncwarp();
    }
    if (!kAhead && !STAGED && block + kStep < end) x.load(p, strip, block + kStep, g, t);
  }
}

template <typename T, int AXIS, int LINES, bool STAGED>
cudaError_t launch(QuantizeParams p, cudaStream_t st) {
  constexpr int W = kWarps<LINES>;
  constexpr int kStep = AXIS == 1 && LINES == 1 ? W : 1;
  const int64_t across = kStep == W ? p.strips : (p.strips + W - 1) / W;
  const int64_t steps = (p.blocks + kStep - 1) / kStep;
  // as many blocks a warp as leave eight CTAs an SM, at most 4
  p.rounds = (int)std::max<int64_t>(1, std::min<int64_t>(4, across * steps / (8 * multiprocessors())));
  const int64_t grid = (steps + p.rounds - 1) / p.rounds * across;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  log_kernel("quantize_blocks lines=%d length=%d rotate=%d axis=%d scale_lines=%d | %d bits%s rounds=%d",
             p.nl, p.length, p.r, AXIS, LINES, (int)sizeof(T) * 8, STAGED ? " staged" : "", p.rounds);
  if constexpr (STAGED) {
    static std::atomic<uint64_t> ready{0};
    return launch_cluster(quantize_kernel<T, AXIS, LINES, true>, ready, (unsigned)grid, W * 32,
                          Stages<AXIS, LINES>::kBytes, 1, st, p);
  } else {
    return launch_overlapped(quantize_kernel<T, AXIS, LINES, false>, (unsigned)grid, W * 32, 0, 1, st, p);
  }
}

template <typename T, bool STAGED>
cudaError_t launch(const QuantizeParams& p, int axis, int lines, cudaStream_t st) {
  if (axis == 1) return lines == 1 ? launch<T, 1, 1, STAGED>(p, st) : launch<T, 1, 128, STAGED>(p, st);
  return lines == 1 ? launch<T, 0, 1, STAGED>(p, st) : launch<T, 0, 128, STAGED>(p, st);
}

template <typename T>
cudaError_t launch(const QuantizeParams& p, int axis, int lines, cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (p.vec16) return launch<T, true>(p, axis, lines, st);
  return launch<T, false>(p, axis, lines, st);
}

}  // namespace

cudaError_t launch_quantize(CMat x, int x_type, int rows, int cols, int rot_bits, int axis,
                            int lines, Mat q, Mat scale, cudaStream_t st) {
  // 2^(-r/2), correctly rounded
  constexpr float kNorm[8] = {1.f, 0.707106781186547524f, 0.5f, 0.353553390593273762f,
                              0.25f, 0.176776695296636881f, 0.125f, 0.0883883476483184406f};
  QuantizeParams p{};
  p.x = x.p, p.ld_x = x.ld;
  p.q = (uint8_t*)q.p, p.ld_q = q.ld;
  p.scale = (float*)scale.p, p.ld_scale = scale.ld;
  p.nl = axis ? rows : cols;
  p.length = axis ? cols : rows;
  p.full = (int)((((int64_t)p.length + (1 << rot_bits) - 1) >> rot_bits) << rot_bits);
  p.blocks = (p.full + 127) / 128;
  p.strips = (p.nl + 15) / 16;
  p.r = rot_bits;
  p.norm = kNorm[rot_bits];
  p.norm_448 = (float)((double)kNorm[rot_bits] / 448.0);
  const int size = x_type == FWT_F32 ? 4 : 2;
  const int unit = axis ? 16 : 2 * size;
  p.vec = (uintptr_t)x.p % (unsigned)unit == 0 && (x.ld * size) % unit == 0;
  p.vec16 = (uintptr_t)x.p % 16 == 0 && (x.ld * size) % 16 == 0;
  if (x_type == FWT_F32) return launch<float>(p, axis, lines, st);
  if (x_type == FWT_BF16) return launch<__nv_bfloat16>(p, axis, lines, st);
  return launch<__half>(p, axis, lines, st);
}

}  // namespace ff
}  // namespace fwt
