// Gated projections of a few tokens: see tokens.cuh for the scheme.  A CTA owns 16 lines of
// both weights; its warps take stretches of 64 elements of the contraction in turn, and the
// join applies the activation.  Bound: HBM (the bytes of both weights).
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "feed_forward.cuh"
#include "ff_host.cuh"
#include "fwt.h"
#include "tma.cuh"
#include "tokens.cuh"

namespace fwt {
namespace ff {
namespace {

struct GatedTokenParams {
  const uint8_t *x, *w[2];
  int64_t ld_x, ld_w[2];  // bytes
  void* h;
  int64_t ld_h;
  int act, m, f;
  int64_t bytes;  // of a line
  int stretches;  // of 128 bytes
};

template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
        " {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
        " {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: groups of 8 tokens.  U: stretches whose loads a warp has in flight together.
template <typename T, int NT, int U>
__global__ void __launch_bounds__(kTokenWarps * 32) gated_tokens_kernel(const GatedTokenParams p) {
  __shared__ float sums[kTokenWarps][2][NT][32][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int j0 = blockIdx.x * 16;
  const uint8_t* w[2][2];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int j = j0 + g + 8 * r;
      w[s][r] = j < p.f ? p.w[s] + (int64_t)j * p.ld_w[s] : nullptr;
    }
  float sum[2][NT][4];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[s][i][e] = 0.f;

  pdl_begin();
  for (int first = warp; first < p.stretches; first += kTokenWarps * U) {
    uint4 wv[U][2][2][2], xv[U][NT][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = (int64_t)(first + u * kTokenWarps) * 128 + 16 * t;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            wv[u][s][r][h] = load16_once<2>(w[s][r], at + 64 * h, p.bytes);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int token = 8 * i + g;
        const uint8_t* x = token < p.m ? p.x + token * p.ld_x : nullptr;
#pragma unroll
        for (int h = 0; h < 2; ++h) xv[u][i][h] = load16<2>(x, at + 64 * h, p.bytes);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 lo = wv[u][s][0][h], hi = wv[u][s][1][h], x = xv[u][i][h];
            mma16<T>(sum[s][i], lo.x, hi.x, lo.y, hi.y, x.x, x.y);
            mma16<T>(sum[s][i], lo.z, hi.z, lo.w, hi.w, x.z, x.w);
          }
  }

#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < NT; ++i)
      *(float4*)sums[warp][s][i][lane] =
          make_float4(sum[s][i][0], sum[s][i][1], sum[s][i][2], sum[s][i][3]);
  __syncthreads();
  // thread -> (token, line): 16 consecutive lines of a token's row of h
  for (int o = threadIdx.x; o < NT * 128; o += kTokenWarps * 32) {
    const int token = o >> 4, line = o & 15;
    if (token >= p.m || j0 + line >= p.f) continue;
    const int from = 4 * (line & 7) + ((token & 7) >> 1), e = (line >> 3) * 2 + (token & 1);
    float gate = 0.f, up = 0.f, value, slope;
#pragma unroll
    for (int s = 0; s < kTokenWarps; ++s) {
      gate += sums[s][0][token >> 3][from][e];
      up += sums[s][1][token >> 3][from][e];
    }
    activate(p.act, gate, value, slope);
    ((T*)p.h)[token * p.ld_h + j0 + line] = (T)(value * up);
  }
}

template <typename T, int NT, int U>
cudaError_t launch(const GatedTokenParams& p, cudaStream_t st) {
  return launch_overlapped(gated_tokens_kernel<T, NT, U>, (unsigned)((p.f + 15) / 16),
                           kTokenWarps * 32, 0, 1, st, p);
}
template <typename T>
cudaError_t run(const GatedTokenParams& p, cudaStream_t st) {
  if (p.m <= 8) return launch<T, 1, 2>(p, st);
  if (p.m <= 16) return launch<T, 2, 1>(p, st);
  return launch<T, 4, 1>(p, st);
}

}  // namespace

cudaError_t launch_gated_tokens(CMat x, CMat w_gate, CMat w_up, Mat h, int type, int act, int m,
                                int f, int d, cudaStream_t st) {
  const GatedTokenParams p{(const uint8_t*)x.p, {(const uint8_t*)w_gate.p, (const uint8_t*)w_up.p},
                           x.ld * 2, {w_gate.ld * 2, w_up.ld * 2}, h.p, h.ld, act, m, f,
                           (int64_t)d * 2, (int)(((int64_t)d + 63) / 64)};
  return type == FWT_BF16 ? run<__nv_bfloat16>(p, st) : run<__half>(p, st);
}

}  // namespace ff
}  // namespace fwt
