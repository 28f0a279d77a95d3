// The block-scaled 8-bit product for a few lines of the first operand (tokens): see
// tokens.cuh for the scheme.  A CTA owns 16 lines of b; its warps take blocks of 128 of the
// contraction in turn.  The sums of one block stay in the matrix products' fp32 accumulators
// and are then added up in fp32, times both scales.  Bound: HBM (the bytes of b).
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "feed_forward.cuh"
#include "fwt.h"
#include "tokens.cuh"

namespace fwt {
namespace ff {
namespace {

struct TokenParams {
  const uint8_t *a, *b;
  int64_t ld_a, ld_b;
  const float *a_scale, *b_scale;
  int64_t ld_as, ld_bs;
  void* c;
  int64_t ld_c;
  int c_type, m, n, k, blocks;
};

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: groups of 8 tokens.  U: blocks whose loads a warp has in flight together.
template <int NT, int U, int LINES>
__global__ void __launch_bounds__(kTokenWarps * 32) tokens_kernel(const TokenParams p) {
  __shared__ float sums[kTokenWarps][NT][32][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int j0 = blockIdx.x * 16;
  const uint8_t* w[2];
  const float* ws[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int j = j0 + g + 8 * r;
    w[r] = j < p.n ? p.b + (int64_t)j * p.ld_b : nullptr;
    ws[r] = j < p.n ? p.b_scale + (int64_t)(LINES == 1 ? j : j / 128) * p.ld_bs : nullptr;
  }
  float sum[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[i][e] = 0.f;

  for (int first = warp; first < p.blocks; first += kTokenWarps * U) {
    uint4 wv[U][2][2], xv[U][NT][2];
    float sw[U][2], sx[U][NT][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int block = first + u * kTokenWarps;
      const bool in = block < p.blocks;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          wv[u][r][h] = load16_once<1>(w[r], (int64_t)block * 128 + 64 * h + 16 * t, p.k);
#pragma unroll
      for (int r = 0; r < 2; ++r) sw[u][r] = in && ws[r] ? __ldg(ws[r] + block) : 0.f;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int token = 8 * i + g;
        const uint8_t* x = token < p.m ? p.a + token * p.ld_a : nullptr;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          xv[u][i][h] = load16<1>(x, (int64_t)block * 128 + 64 * h + 16 * t, p.k);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          sx[u][i][e] = in && 8 * i + 2 * t + e < p.m
                            ? __ldg(p.a_scale + (8 * i + 2 * t + e) * p.ld_as + block) : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (first + u * kTokenWarps >= p.blocks) break;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 lo = wv[u][0][h], hi = wv[u][1][h], x = xv[u][i][h];
          mma_e4m3(part, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
          mma_e4m3(part, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sum[i][e] = fmaf(part[e], sw[u][e >> 1] * sx[u][i][e & 1], sum[i][e]);
      }
    }
  }

#pragma unroll
  for (int i = 0; i < NT; ++i)
    *(float4*)sums[warp][i][lane] = make_float4(sum[i][0], sum[i][1], sum[i][2], sum[i][3]);
  __syncthreads();
  // thread -> (token, line): 16 consecutive lines of a token's row of C
  for (int o = threadIdx.x; o < NT * 128; o += kTokenWarps * 32) {
    const int token = o >> 4, line = o & 15;
    if (token >= p.m || j0 + line >= p.n) continue;
    const int from = 4 * (line & 7) + ((token & 7) >> 1), e = (line >> 3) * 2 + (token & 1);
    float v = 0.f;
#pragma unroll
    for (int s = 0; s < kTokenWarps; ++s) v += sums[s][token >> 3][from][e];
    const int64_t at = token * p.ld_c + j0 + line;
    if (p.c_type == FWT_F32) ((float*)p.c)[at] = v;
    else if (p.c_type == FWT_BF16) ((__nv_bfloat16*)p.c)[at] = __float2bfloat16_rn(v);
    else ((__half*)p.c)[at] = __float2half_rn(v);
  }
}

template <int NT, int U>
cudaError_t launch(const TokenParams& p, int lines, cudaStream_t st) {
  const unsigned grid = (unsigned)((p.n + 15) / 16);
  if (lines == 1) tokens_kernel<NT, U, 1><<<grid, kTokenWarps * 32, 0, st>>>(p);
  else tokens_kernel<NT, U, 128><<<grid, kTokenWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_matmul_tokens(CMat a, CMat a_scale, CMat b, CMat b_scale, int b_lines, Mat c,
                                 int c_type, int m, int n, int k, cudaStream_t st) {
  const TokenParams p{(const uint8_t*)a.p, (const uint8_t*)b.p, a.ld, b.ld,
                      (const float*)a_scale.p, (const float*)b_scale.p, a_scale.ld, b_scale.ld,
                      c.p, c.ld, c_type, m, n, k, (int)(((int64_t)k + 127) / 128)};
  if (m <= 8) return launch<1, 4>(p, b_lines, st);
  if (m <= 16) return launch<2, 2>(p, b_lines, st);
  return launch<4, 1>(p, b_lines, st);
}

}  // namespace ff
}  // namespace fwt
