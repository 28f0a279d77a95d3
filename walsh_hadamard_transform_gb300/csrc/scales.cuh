// What the kernels of the block-scaled 8-bit product share: the 16 x 8 products of the legacy tensor
// path, and scales whose own product overflows.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace fwt {
namespace ff {

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// sum + x a b.  Scales whose product overflows are both above 1, so x times one and then the other
// overflows where the result does, and a sum of 0 stays 0.
__device__ __forceinline__ float add_apart(float sum, float x, float a, float b) {
  const float both = a * b;
  return fabsf(both) < INFINITY ? fmaf(x, both, sum) : fmaf(x * a, b, sum);
}

}  // namespace ff
}  // namespace fwt
