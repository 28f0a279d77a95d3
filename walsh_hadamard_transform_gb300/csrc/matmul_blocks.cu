// Product of two 8-bit operands with a scale for each block of 128 along the contraction.
//
// Each thread owns one element of C: the fp32 sum of a block's products, times both
// scales, added up over the blocks.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "feed_forward.cuh"
#include "fwt.h"

namespace fwt {
namespace ff {
namespace {

__device__ __forceinline__ float from_code(uint8_t v) {
  __nv_fp8_e4m3 q;
  q.__x = v;
  return (float)q;
}

struct MatmulParams {
  const uint8_t *a, *b;
  const float *a_scale, *b_scale;
  void* c;
  int64_t ld_a, ld_b, ld_as, ld_bs, ld_c;
  int b_lines, m, n, k;
};

template <typename C>
__global__ void __launch_bounds__(256) matmul_blocks_kernel(MatmulParams p) {
  __shared__ float as[16][17], bs[16][17];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int tiles_n = (p.n + 15) / 16;
  const int i0 = blockIdx.x / tiles_n * 16, j0 = blockIdx.x % tiles_n * 16;
  const int i = i0 + ty, j = j0 + tx;
  float sum = 0.f;
  for (int k0 = 0; k0 < p.k; k0 += 128) {
    float part = 0.f;
    for (int s = k0; s < k0 + 128 && s < p.k; s += 16) {
      const int k = s + tx;
      as[ty][tx] = i0 + ty < p.m && k < p.k ? from_code(p.a[(int64_t)(i0 + ty) * p.ld_a + k]) : 0.f;
      bs[ty][tx] = j0 + ty < p.n && k < p.k ? from_code(p.b[(int64_t)(j0 + ty) * p.ld_b + k]) : 0.f;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 16; ++e) part = fmaf(as[ty][e], bs[tx][e], part);
      __syncthreads();
    }
    if (i < p.m && j < p.n)
      sum = fmaf(part, p.a_scale[(int64_t)i * p.ld_as + k0 / 128] *
                           p.b_scale[(int64_t)(j / p.b_lines) * p.ld_bs + k0 / 128], sum);
  }
  if (i < p.m && j < p.n) ((C*)p.c)[(int64_t)i * p.ld_c + j] = (C)sum;
}

}  // namespace

cudaError_t launch_matmul_blocks(CMat a, CMat a_scale, CMat b, CMat b_scale, int b_lines, Mat c,
                                 int c_type, int m, int n, int k, cudaStream_t st) {
  const MatmulParams p{(const uint8_t*)a.p, (const uint8_t*)b.p, (const float*)a_scale.p,
                       (const float*)b_scale.p, c.p, a.ld, b.ld, a_scale.ld, b_scale.ld, c.ld,
                       b_lines, m, n, k};
  const int64_t grid = (((int64_t)m + 15) / 16) * (((int64_t)n + 15) / 16);
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (c_type == FWT_F32) matmul_blocks_kernel<float><<<(unsigned)grid, 256, 0, st>>>(p);
  else if (c_type == FWT_BF16) matmul_blocks_kernel<__nv_bfloat16><<<(unsigned)grid, 256, 0, st>>>(p);
  else matmul_blocks_kernel<__half><<<(unsigned)grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace ff
}  // namespace fwt
