// The block-scaled 8-bit product for a few lines of the first operand (tokens): see
// tokens.cuh for the scheme.  A CTA owns 16 lines of b; its warps take blocks of 128 of the
// contraction in turn.  The sums of one block stay in the matrix products' fp32 accumulators
// and are then added up in fp32, times both scales.  Bound: HBM (the bytes of b).
//
// Each warp has a ring of its own in shared memory that asynchronous copies fill: the bytes on
// their way then cost no registers, and an SM holds enough of them.  (Loading straight to
// registers measured 12.6 us for one token by 4096 x 8192: 163 registers a thread left one
// CTA an SM, and two waves.)  One token by 4096 x 8192: 8.75 us, 3.8 TB/s, of which some 1.5 are
// the launch; 16 tokens 11.1 us.
#include <atomic>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "feed_forward.cuh"
#include "ff_host.cuh"
#include "fwt.h"
#include "scales.cuh"
#include "tma.cuh"

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

// 16 (or 4) bytes to shared memory, `valid` of them from `from`, zeros after.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, int valid) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(valid)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from, int valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(valid)
               : "memory");
}

// NT: groups of 8 tokens.  W: warps.  S: stages of a warp's ring, a block of 128 each.
template <int NT, int W, int S>
struct Ring {
  static constexpr int kTokens = 2048, kScales = kTokens + NT * 1024;  // after 16 lines of b
  static constexpr int kStage = kScales + (8 * NT + 16) * 4;
  static constexpr int kBytes = S * W * kStage;
};

template <int NT, int W, int S, int LINES>
__global__ void __launch_bounds__(W * 32) tokens_kernel(const TokenParams p) {
  using R = Ring<NT, W, S>;
  extern __shared__ __align__(16) uint8_t rings[];
  __shared__ __align__(16) float sums[W][NT][32][4];  // (float4 stores)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int j0 = blockIdx.x * 16;
  uint8_t* ring = rings + warp * (S * R::kStage);
  const uint32_t ring_at = smem_u32(ring);
  pdl_begin();

  // Rows of 128 bytes, the halves of odd ones swapped, so that the fragments' reads (64 bytes
  // of two rows at a time) meet all banks.
  auto fill = [&](int stage, int block) {
    const uint32_t at = ring_at + stage * R::kStage;
    if (block < p.blocks) {
      const int chunk = lane & 7;
      const int64_t k = (int64_t)block * 128 + 16 * chunk;
      const int valid = (int)min((int64_t)16, max((int64_t)0, p.k - k));
#pragma unroll
      for (int i = 0; i < 4 + 2 * NT; ++i) {  // of b, then of the tokens
        const int row = (i < 4 ? i : i - 4) * 4 + (lane >> 3);
        const bool in = i < 4 ? j0 + row < p.n : row < p.m;
        const uint8_t* from = i < 4 ? p.b + (int64_t)(j0 + row) * p.ld_b : p.a + (int64_t)row * p.ld_a;
        copy16(at + (i < 4 ? 0 : R::kTokens) + row * 128 + ((chunk ^ ((row & 1) << 2)) << 4),
               in && valid ? from + k : p.b, in ? valid : 0);
      }
      if (lane < 8 * NT)
        copy4(at + R::kScales + lane * 4, lane < p.m ? p.a_scale + lane * p.ld_as + block : p.a_scale,
              lane < p.m ? 4 : 0);
      if (lane < (LINES == 1 ? 16 : 1)) {
        const int line = LINES == 1 ? j0 + lane : j0 / 128;
        const bool in = LINES == 128 || line < p.n;
        copy4(at + R::kScales + (8 * NT + lane) * 4,
              in ? p.b_scale + (int64_t)line * p.ld_bs + block : p.b_scale, in ? 4 : 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < S; ++s) fill(s, warp + s * W);

  float sum[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[i][e] = 0.f;
  int stage = 0;
  for (int block = warp; block < p.blocks; block += W) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    __syncwarp();
    const uint8_t* at = ring + stage * R::kStage;
    const float* scales = (const float*)(at + R::kScales);
    uint4 w[2][2];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[r][h] = *(const uint4*)(at + (g + 8 * r) * 128 + (((4 * h + t) ^ ((g & 1) << 2)) << 4));
    const float sw[2] = {scales[8 * NT + (LINES == 1 ? g : 0)], scales[8 * NT + (LINES == 1 ? g + 8 : 0)]};
    float part[NT][4], most = 0.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      part[i][0] = part[i][1] = part[i][2] = part[i][3] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 x = *(const uint4*)(at + R::kTokens + (8 * i + g) * 128 +
                                        (((4 * h + t) ^ ((g & 1) << 2)) << 4));
        const uint4 lo = w[0][h], hi = w[1][h];
        mma_e4m3(part[i], lo.x, hi.x, lo.y, hi.y, x.x, x.y);
        mma_e4m3(part[i], lo.z, hi.z, lo.w, hi.w, x.z, x.w);
      }
      const float2 sx = *(const float2*)&scales[8 * i + 2 * t];
      most = fmaxf(most, fmaxf(fabsf(sx.x), fabsf(sx.y)));
    }
    // (one look at the block's scales, not one for each pair of them)
    if (most * fmaxf(fabsf(sw[0]), fabsf(sw[1])) < INFINITY) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float2 sx = *(const float2*)&scales[8 * i + 2 * t];
        sum[i][0] = fmaf(part[i][0], sw[0] * sx.x, sum[i][0]);
        sum[i][1] = fmaf(part[i][1], sw[0] * sx.y, sum[i][1]);
        sum[i][2] = fmaf(part[i][2], sw[1] * sx.x, sum[i][2]);
        sum[i][3] = fmaf(part[i][3], sw[1] * sx.y, sum[i][3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float2 sx = *(const float2*)&scales[8 * i + 2 * t];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sum[i][e] = add_apart(sum[i][e], part[i][e], sw[e >> 1], e & 1 ? sx.y : sx.x);
      }
    }
    __syncwarp();
    fill(stage, block + S * W);
    if (++stage == S) stage = 0;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");

#pragma unroll
  for (int i = 0; i < NT; ++i)
    *(float4*)sums[warp][i][lane] = make_float4(sum[i][0], sum[i][1], sum[i][2], sum[i][3]);
  __syncthreads();
  // thread -> (token, line): 16 consecutive lines of a token's row of C
  for (int o = threadIdx.x; o < NT * 128; o += W * 32) {
    const int token = o >> 4, line = o & 15;
    if (token >= p.m || j0 + line >= p.n) continue;
    const int from = 4 * (line & 7) + ((token & 7) >> 1), e = (line >> 3) * 2 + (token & 1);
    float v = 0.f;
#pragma unroll
    for (int s = 0; s < W; ++s) v += sums[s][token >> 3][from][e];
    const int64_t at = token * p.ld_c + j0 + line;
    if (p.c_type == FWT_F32) ((float*)p.c)[at] = v;
    else if (p.c_type == FWT_BF16) ((__nv_bfloat16*)p.c)[at] = __float2bfloat16_rn(v);
    else ((__half*)p.c)[at] = __float2half_rn(v);
  }
}

template <int NT, int W, int S, int LINES>
cudaError_t launch(const TokenParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  log_kernel("matmul_blocks m=%d n=%d k=%d scale_lines=%d | tokens=%d warps=%d", p.m, p.n, p.k, LINES,
             8 * NT, W);
  return launch_cluster(tokens_kernel<NT, W, S, LINES>, ready, (unsigned)((p.n + 15) / 16), W * 32,
                        Ring<NT, W, S>::kBytes, 1, st, p);
}
template <int NT, int W, int S>
cudaError_t launch(const TokenParams& p, int lines, cudaStream_t st) {
  return lines == 1 ? launch<NT, W, S, 1>(p, st) : launch<NT, W, S, 128>(p, st);
}
// Eight warps to 16 lines of b, or four where that many CTAs would come in a second wave.
template <int NT, int S8, int S4>
cudaError_t launch_few(const TokenParams& p, int lines, cudaStream_t st) {
  return (p.n + 15) / 16 <= 2 * multiprocessors() ? launch<NT, 8, S8>(p, lines, st)
                                                  : launch<NT, 4, S4>(p, lines, st);
}

}  // namespace

cudaError_t launch_matmul_tokens(CMat a, CMat a_scale, CMat b, CMat b_scale, int b_lines, Mat c,
                                 int c_type, int m, int n, int k, cudaStream_t st) {
  const TokenParams p{(const uint8_t*)a.p, (const uint8_t*)b.p, a.ld, b.ld,
                      (const float*)a_scale.p, (const float*)b_scale.p, a_scale.ld, b_scale.ld,
                      c.p, c.ld, c_type, m, n, k, (int)(((int64_t)k + 127) / 128)};
  if (m <= 8) return launch_few<1, 4, 4>(p, b_lines, st);
  if (m <= 16) return launch_few<2, 3, 4>(p, b_lines, st);
  return launch_few<4, 2, 3>(p, b_lines, st);
}

}  // namespace ff
}  // namespace fwt
