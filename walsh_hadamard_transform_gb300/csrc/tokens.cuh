// Products of a few tokens (lines of the first operand) with all lines of a weight: the scheme of
// the kernels for single tokens and small batches, and their reads of 16-bit operands.
//
// With few tokens a product is bound by reading the weights once.  A warp reads 16 weight
// lines into the fragments of 16 x 8 matrix products, 16 bytes a thread, without a tile that
// the CTA would share: which elements of the contraction meet in which slot of a product is
// free as long as both operands agree, so thread t of a quad takes 16 consecutive bytes of a
// line at 64 c + 16 t, and the tokens' fragment the same bytes of its line.  The warps of a
// CTA split the contraction and add their sums up in shared memory, in a fixed order.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace fwt {
namespace ff {

constexpr int kTokenWarps = 8;

// 16 bytes of a line of `bytes` bytes of 16-bit elements from `at` on: zero past its end and for
// line = null (the line's start and `at` are multiples of 16 bytes).
__device__ __forceinline__ uint4 load16(const uint8_t* line, int64_t at, int64_t bytes) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (!line || at >= bytes) return v;
  if (at + 16 <= bytes) return *(const uint4*)(line + at);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; i += 2)
    if (at + i < bytes) w[i / 4] |= (uint32_t)*(const unsigned short*)(line + at + i) << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The same for weights: read once, so kept out of the way of what is used again.
__device__ __forceinline__ uint4 load16_once(const uint8_t* line, int64_t at, int64_t bytes) {
  if (line && at + 16 <= bytes) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(line + at));
    return v;
  }
  return load16(line, at, bytes);
}

}  // namespace ff
}  // namespace fwt
