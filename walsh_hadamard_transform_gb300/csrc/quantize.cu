// Rotation and quantisation to 8-bit floating point with a scale for each block of 128.
//
// A warp owns 16 lines by one block of 128 elements along the axis.  The rotation of a
// group of 2^r <= 128 elements is a Kronecker product of 2 x 2 factors, one for each
// index bit below r, so its factors may be applied in any order and by different means:
//
//   bits 0, 1, 3, 4   one m16n8k16 matrix product of 16 lines by 16 elements with the
//                     16 x 16 matrix of signs (zeros where an index bit stays as it is).
//                     Signs and inputs are exact in 16 bits and the sums fp32; an fp32
//                     input goes in as three bf16 pieces that add up to it exactly.
//   bits 2, 5, 6      additions between the thread's own registers.
//
// Elements are assigned to the product's slots so that a thread holds the same elements
// before and after it: 8 consecutive ones (bits 0..2) in each of the four groups of 32
// (bits 5, 6), the lanes t = 0..3 of a quad being bits 3 and 4, for the lines g = lane / 4
// and g + 8.  So inputs are 16-byte loads, codes 8-byte stores, and only the maximum of a
// block crosses lanes (two shuffles a line, where butterflies across lanes would take four
// shuffles an element and be bound by them).  Bound: HBM.
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "feed_forward.cuh"
#include "fwt.h"

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
  int vec;     // rows of x start on 16-byte boundaries
};

template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]);
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4],
                                                     const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
template <>
__device__ __forceinline__ void mma16<__half>(float (&d)[4], const uint32_t (&a)[4],
                                              const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
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

// Eight elements along the axis from position `pos` of line `line`, as packed 16-bit pairs
// (one set for each piece).  Zero outside the matrix.
template <typename T, int AXIS>
__device__ __forceinline__ void load8(const QuantizeParams& p, int line, int pos,
                                      uint32_t (&out)[Input<T>::kPieces][4]) {
  const T* x = (const T*)p.x;
  if constexpr (sizeof(T) == 2) {
    if (AXIS == 1 && p.vec && line < p.nl && pos + 8 <= p.length) {
      const uint4 v = __ldg((const uint4*)(x + (int64_t)line * p.ld_x + pos));
      out[0][0] = v.x, out[0][1] = v.y, out[0][2] = v.z, out[0][3] = v.w;
      return;
    }
    uint32_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t at = AXIS == 1 ? (int64_t)line * p.ld_x + pos + j
                                   : (int64_t)(pos + j) * p.ld_x + line;
      e[j] = line < p.nl && pos + j < p.length ? __ldg((const unsigned short*)x + at) : 0;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) out[0][j] = e[2 * j] | (e[2 * j + 1] << 16);
  } else {
    float e[8];
    if (AXIS == 1 && p.vec && line < p.nl && pos + 8 <= p.length) {
      const float4* v = (const float4*)(x + (int64_t)line * p.ld_x + pos);
      const float4 lo = __ldg(v), hi = __ldg(v + 1);
      e[0] = lo.x, e[1] = lo.y, e[2] = lo.z, e[3] = lo.w;
      e[4] = hi.x, e[5] = hi.y, e[6] = hi.z, e[7] = hi.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t at = AXIS == 1 ? (int64_t)line * p.ld_x + pos + j
                                     : (int64_t)(pos + j) * p.ld_x + line;
        e[j] = line < p.nl && pos + j < p.length ? __ldg((const float*)x + at) : 0.f;
      }
    }
    // Truncation leaves no piece larger than its input; 8 + 8 + 8 significant bits.
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = __float_as_uint(e[2 * j]) & 0xffff0000u;
        const uint32_t hi = __float_as_uint(e[2 * j + 1]) & 0xffff0000u;
        out[k][j] = (lo >> 16) | hi;
        e[2 * j] -= __uint_as_float(lo);
        e[2 * j + 1] -= __uint_as_float(hi);
      }
    }
  }
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Warps of a CTA: consecutive blocks of one strip (axis 1) or consecutive strips of one
// block (axis 0), so that a CTA reads long runs of rows; with 128 lines to a scale, the
// eight strips of one tile.
template <int LINES>
constexpr int kWarps = LINES == 1 ? 4 : 8;

template <typename T, int AXIS, int LINES>
__global__ void __launch_bounds__(kWarps<LINES> * 32) quantize_kernel(QuantizeParams p) {
  constexpr int W = kWarps<LINES>;
  using M = typename Input<T>::Mma;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  int strip, block;
  if constexpr (LINES == 128) {
    block = blockIdx.x % p.blocks;
    strip = blockIdx.x / p.blocks * W + warp;
  } else if constexpr (AXIS == 1) {
    const int per = (p.blocks + W - 1) / W;
    block = blockIdx.x % per * W + warp;
    strip = blockIdx.x / per;
  } else {
    const int per = (p.strips + W - 1) / W;
    strip = blockIdx.x % per * W + warp;
    block = blockIdx.x / per;
  }
  if (LINES == 1 && (block >= p.blocks || strip >= p.strips)) return;

  uint32_t b[2][2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int en = 8 * (g >> 1) + (g & 1) + 2 * n;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      b[n][h] = sign16<M>(8 * t + 2 * h, en, p.r) | (sign16<M>(8 * t + 2 * h + 1, en, p.r) << 16);
  }

  const int line = strip * 16 + g, pos = block * 128 + 8 * t;
  float y[4][2][2][4];  // group of 32, bit 2, bit 1, (line, bit 0)
#pragma unroll
  for (int grp = 0; grp < 4; ++grp) {
    uint32_t u[Input<T>::kPieces][4], v[Input<T>::kPieces][4];
    load8<T, AXIS>(p, line, pos + 32 * grp, u);
    load8<T, AXIS>(p, line + 8, pos + 32 * grp, v);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[grp][h][n][i] = 0.f;
#pragma unroll
        for (int k = Input<T>::kPieces - 1; k >= 0; --k) {
          const uint32_t a[4] = {u[k][2 * h], v[k][2 * h], u[k][2 * h + 1], v[k][2 * h + 1]};
          mma16<M>(y[grp][h][n], a, b[n]);
        }
      }
  }
#pragma unroll
  for (int grp = 0; grp < 4; ++grp)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = y[grp][0][n][i], hi = y[grp][1][n][i];
        if (p.r > 2) y[grp][0][n][i] = lo + hi, y[grp][1][n][i] = lo - hi;
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

  // The maximum by the bits of |y|: a NaN's are above every number's.
  uint32_t top[2] = {0, 0};
#pragma unroll
  for (int grp = 0; grp < 4; ++grp)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[grp][h][n][i] *= p.norm;
          top[i >> 1] = max(top[i >> 1], __float_as_uint(y[grp][h][n][i]) & 0x7fffffffu);
        }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    top[s] = max(top[s], __shfl_xor_sync(~0u, top[s], 1));
    top[s] = max(top[s], __shfl_xor_sync(~0u, top[s], 2));
  }
  if constexpr (LINES == 128) {
    __shared__ uint32_t tops[W];
    uint32_t m = max(top[0], top[1]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
    if (lane == 0) tops[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) m = max(m, tops[w]);
    top[0] = top[1] = m;
  }

#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int l = line + 8 * s;
    float scale = fmaxf(__fdiv_rn(__uint_as_float(top[s]), 448.f), 0x1p-126f);
    if (top[s] >= 0x7f800000u) scale = __uint_as_float(0x7fffffffu);
    const float inv = __fdiv_rn(1.f, scale);
    if (LINES == 1 ? t == 0 && l < p.nl : threadIdx.x == 0 && s == 0)
      p.scale[(int64_t)(LINES == 1 ? l : l / 128) * p.ld_scale + block] = scale;
    if (l >= p.nl) continue;
    uint8_t* q = p.q + (int64_t)l * p.ld_q;
#pragma unroll
    for (int grp = 0; grp < 4; ++grp) {
      uint2 code;
      code.x = codes4(y[grp][0][0][2 * s] * inv, y[grp][0][0][2 * s + 1] * inv,
                      y[grp][0][1][2 * s] * inv, y[grp][0][1][2 * s + 1] * inv);
      code.y = codes4(y[grp][1][0][2 * s] * inv, y[grp][1][0][2 * s + 1] * inv,
                      y[grp][1][1][2 * s] * inv, y[grp][1][1][2 * s + 1] * inv);
      const int at = pos + 32 * grp;
      if (at + 8 <= p.full) {
        *(uint2*)(q + at) = code;
      } else {
        for (int j = 0; j < 8 && at + j < p.full; ++j)
          q[at + j] = (uint8_t)((j < 4 ? code.x : code.y) >> (8 * (j & 3)));
      }
    }
  }
}

template <typename T, int AXIS, int LINES>
cudaError_t launch(const QuantizeParams& p, cudaStream_t st) {
  constexpr int W = kWarps<LINES>;
  const int64_t grid = LINES == 128 ? (int64_t)((p.strips + W - 1) / W) * p.blocks
                       : AXIS == 1  ? (int64_t)((p.blocks + W - 1) / W) * p.strips
                                    : (int64_t)((p.strips + W - 1) / W) * p.blocks;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  quantize_kernel<T, AXIS, LINES><<<(unsigned)grid, W * 32, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const QuantizeParams& p, int axis, int lines, cudaStream_t st) {
  if (axis == 1) return lines == 1 ? launch<T, 1, 1>(p, st) : launch<T, 1, 128>(p, st);
  return lines == 1 ? launch<T, 0, 1>(p, st) : launch<T, 0, 128>(p, st);
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
  const int size = x_type == FWT_F32 ? 4 : 2;
  p.vec = ((uintptr_t)x.p & 15u) == 0 && (x.ld * size) % 16 == 0;
  if (x_type == FWT_F32) return launch<float>(p, axis, lines, st);
  if (x_type == FWT_BF16) return launch<__nv_bfloat16>(p, axis, lines, st);
  return launch<__half>(p, axis, lines, st);
}

}  // namespace ff
}  // namespace fwt
