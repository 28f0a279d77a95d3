// Gated projections of a few tokens: see tokens.cuh for the scheme.  A CTA owns 16 lines of
// both weights; its warps take stretches of 64 elements of the contraction in turn, and the
// join applies the activation.  Bound: HBM (the bytes of both weights): one token by
// 2 x 8192 x 4096 24.6 us, 5.5 TB/s (23.8 with loads of the read-only path, which asks for weights
// that no kernel before writes).
//
// Their gradients for up to 8 tokens, three kernels: the same products again with dg and du
// left in fp32, a line of the weights after the other (8 tokens side by side); dx, which reads
// both weights once more, in strips of 64 columns that a cluster shares out along f; dw_gate
// and dw_up, up to eight multiply-adds an element, bound by writing them.  One token, 8192 x
// 2048: 47 us in three launches (the bytes' floor is 20, 30 with the weights read twice as here);
// eight 64, by the latency of dx.
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "feed_forward.cuh"
#include "ff_host.cuh"
#include "fwt.h"
#include "tcgen05.cuh"
#include "tokens.cuh"

namespace fwt {
namespace ff {
namespace {

struct GatedTokenParams {
  const uint8_t *x, *w[2];
  int64_t ld_x, ld_w[2];  // bytes
  void* h;
  int64_t ld_h;
  const void* grad;  // gradients: dh, and
  int64_t ld_grad;
  float* work;       // dg of 8 tokens for each line, then du
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
template <typename T, int NT, int U, bool GRADIENTS>
__global__ void __launch_bounds__(kTokenWarps * 32) gated_tokens_kernel(const GatedTokenParams p) {
  __shared__ __align__(16) float sums[kTokenWarps][2][NT][32][4];  // (float4 stores)
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
            wv[u][s][r][h] = load16_once(w[s][r], at + 64 * h, p.bytes);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int token = 8 * i + g;
        const uint8_t* x = token < p.m ? p.x + token * p.ld_x : nullptr;
#pragma unroll
        for (int h = 0; h < 2; ++h) xv[u][i][h] = load16(x, at + 64 * h, p.bytes);
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
    if ((!GRADIENTS && token >= p.m) || j0 + line >= p.f) continue;
    const int from = 4 * (line & 7) + ((token & 7) >> 1), e = (line >> 3) * 2 + (token & 1);
    float gate = 0.f, up = 0.f, value, slope;
#pragma unroll
    for (int s = 0; s < kTokenWarps; ++s) {
      gate += sums[s][0][token >> 3][from][e];
      up += sums[s][1][token >> 3][from][e];
    }
    activate(p.act, gate, value, slope);
    if constexpr (GRADIENTS) {
      const float dh = token < p.m ? (float)((const T*)p.grad)[token * p.ld_grad + j0 + line] : 0.f;
      float* to = p.work + (int64_t)(j0 + line) * 8 + token;
      to[0] = token < p.m ? dh * up * slope : 0.f;
      to[(int64_t)p.f * 8] = token < p.m ? dh * value : 0.f;
    } else {
      ((T*)p.h)[token * p.ld_h + j0 + line] = (T)(value * up);
    }
  }
}

struct TokenGradientParams {
  const uint8_t *x, *w[2];
  int64_t ld_x, ld_w[2];  // bytes
  void* out[2];           // dx; dw_gate, dw_up
  int64_t ld_out[2];
  const float* work;
  int m, f, d;
  int vec;  // output rows start on 16-byte boundaries
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f;
    if constexpr (std::is_same<T, __half>::value) f = __half22float2(*(const __half2*)&w[i]);
    else f = __bfloat1622float2(*(const __nv_bfloat162*)&w[i]);
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 v = __floats2half2_rn(a, b);
    return *(const uint32_t*)&v;
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *(const uint32_t*)&v;
  }
}

// dx of up to TM tokens, 64 columns: the cluster's CTAs share out the lines of both weights,
// 128 of them at a time; a thread adds up TM tokens by 8 columns over every 32nd line.  All
// loads of a turn are on their way together: the weights' to registers, dg and du to shared
// memory, where every thread of a line reads them.
constexpr int kDxCluster = 8, kDxWarps = 8, kDxLines = 128;

template <typename T, int TM>
__global__ void __launch_bounds__(kDxWarps * 32, 2) token_dx_kernel(const TokenGradientParams p) {
  __shared__ __align__(16) float work[2][2][kDxLines][8];  // in turn; dg and du
  __shared__ float sums[kDxWarps][TM][64];
  __shared__ float total[TM][64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cluster_rank();
  const int col = (int)(blockIdx.x / kDxCluster) * 64 + (lane & 7) * 8;
  const int share = (p.f + kDxCluster - 1) / kDxCluster;
  const int begin = rank * share, end = min(p.f, begin + share);
  float acc[TM][8];
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[t][c] = 0.f;
  pdl_begin();
  for (int j0 = begin, turn = 0; j0 < end; j0 += kDxLines, turn ^= 1) {
    uint4 w[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int j = j0 + u * 32 + warp * 4 + (lane >> 3);
        w[u][s] = load16_once(j < end ? p.w[s] + (int64_t)j * p.ld_w[s] : nullptr, (int64_t)col * 2,
                                 (int64_t)p.d * 2);
      }
    const int line = threadIdx.x >> 1;  // two threads a line, dg then du
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const float4* from = (const float4*)(p.work + ((int64_t)s * p.f + j0 + line) * 8) + (threadIdx.x & 1);
      const float4 v = j0 + line < end ? *from : make_float4(0.f, 0.f, 0.f, 0.f);
      *((float4*)work[turn][s][line] + (threadIdx.x & 1)) = v;
    }
    __syncthreads();  // once a turn: the other half of `work` is read until the next
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const float* g = work[turn][s][u * 32 + warp * 4 + (lane >> 3)];
        float v[8];
        unpack8<T>(w[u][s], v);
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[t][c] = fmaf(g[t], v[c], acc[t][c]);
      }
  }
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      float v = acc[t][c];
      v += __shfl_xor_sync(~0u, v, 8);
      v += __shfl_xor_sync(~0u, v, 16);
      if (lane < 8) sums[warp][t][lane * 8 + c] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < TM * 64; i += kDxWarps * 32) {
    float v = 0.f;
#pragma unroll
    for (int s = 0; s < kDxWarps; ++s) v += sums[s][i >> 6][i & 63];
    total[i >> 6][i & 63] = v;
  }
  cluster_sync();
  if (threadIdx.x < 64 && rank < TM && rank < p.m) {  // a token a CTA
    const uint32_t at = smem_u32(&total[rank][threadIdx.x]);
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < kDxCluster; ++r) v += load_cluster(map_to_rank(at, r));
    const int c = (int)(blockIdx.x / kDxCluster) * 64 + threadIdx.x;
    if (c < p.d) ((T*)p.out[0])[(int64_t)rank * p.ld_out[0] + c] = (T)v;
  }
  cluster_sync();  // no CTA leaves while another reads its sums
}

// dw_gate and dw_up: a thread holds 8 columns of up to TM tokens and goes through lines of the
// weights, a warp's 256 columns at a time.
constexpr int kDwWarps = 8, kDwLines = 8;  // lines of a warp

template <typename T, int TM>
__global__ void __launch_bounds__(kDwWarps * 32) token_dw_kernel(const TokenGradientParams p, int strips) {
  __shared__ __align__(16) float work[2][kDwWarps * kDwLines][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = (int)(blockIdx.x % strips) * 256 + lane * 8;
  const int first = (int)(blockIdx.x / strips) * (kDwWarps * kDwLines);
  pdl_begin();
  float x[TM][8];
#pragma unroll
  for (int t = 0; t < TM; ++t)
    unpack8<T>(load16(t < p.m ? p.x + t * p.ld_x : nullptr, (int64_t)col * 2, (int64_t)p.d * 2), x[t]);
  for (int i = threadIdx.x; i < 2 * kDwWarps * kDwLines * 2; i += kDwWarps * 32) {
    const int s = i / (kDwWarps * kDwLines * 2), line = i / 2 % (kDwWarps * kDwLines);
    const float4* from = (const float4*)(p.work + ((int64_t)s * p.f + first + line) * 8) + (i & 1);
    *((float4*)work[s][line] + (i & 1)) =
        first + line < p.f ? *from : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  if (col >= p.d) return;
#pragma unroll 2
  for (int i = 0; i < kDwLines; ++i) {
    const int line = warp * kDwLines + i, j = first + line;
    if (j >= p.f) break;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const float* g = work[s][line];
      float v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = g[0] * x[0][c];
#pragma unroll
      for (int t = 1; t < TM; ++t)
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = fmaf(g[t], x[t][c], v[c]);
      T* out = (T*)p.out[s] + (int64_t)j * p.ld_out[s] + col;
      if (p.vec && col + 8 <= p.d) {
        *(uint4*)out = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                                  pack2<T>(v[6], v[7]));
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (col + c < p.d) out[c] = (T)v[c];
      }
    }
  }
}

template <typename T, int TM>
cudaError_t launch_gradients(TokenGradientParams p, Mat dx, Mat dw_gate, Mat dw_up, cudaStream_t st) {
  cudaError_t err = cudaSuccess;
  constexpr const char* kType = std::is_same<T, __half>::value ? "f16" : "bf16";
  if (dx.p) {
    log_kernel("gated dx %s m=%d f=%d d=%d | tokens=%d", kType, p.m, p.f, p.d, TM);
    p.out[0] = dx.p, p.ld_out[0] = dx.ld;
    err = launch_overlapped(token_dx_kernel<T, TM>, (unsigned)((p.d + 63) / 64) * kDxCluster,
                            kDxWarps * 32, 0, kDxCluster, st, p);
  }
  if (err == cudaSuccess && dw_gate.p) {
    const Mat out[2] = {dw_gate, dw_up};
    p.vec = 1;
    for (int s = 0; s < 2; ++s) {
      p.out[s] = out[s].p, p.ld_out[s] = out[s].ld;
      p.vec &= ((uintptr_t)out[s].p & 15u) == 0 && out[s].ld % 8 == 0;
    }
    log_kernel("gated dw %s m=%d f=%d d=%d | tokens=%d", kType, p.m, p.f, p.d, TM);
    const int strips = (p.d + 255) / 256, lines = kDwWarps * kDwLines;
    const int64_t grid = (int64_t)strips * ((p.f + lines - 1) / lines);
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    err = launch_overlapped(token_dw_kernel<T, TM>, (unsigned)grid, kDwWarps * 32, 0, 1, st, p, strips);
  }
  return err;
}

template <typename T, int NT, int U, bool GRADIENTS = false>
cudaError_t launch(const GatedTokenParams& p, cudaStream_t st) {
  log_kernel("gated%s %s m=%d f=%d d=%d | tokens=%d", GRADIENTS ? " gradients" : "",
             std::is_same<T, __half>::value ? "f16" : "bf16", p.m, p.f, (int)(p.bytes / 2), 8 * NT);
  return launch_overlapped(gated_tokens_kernel<T, NT, U, GRADIENTS>, (unsigned)((p.f + 15) / 16),
                           kTokenWarps * 32, 0, 1, st, p);
}
template <typename T>
cudaError_t run(const GatedTokenParams& p, cudaStream_t st) {
  if (p.m <= 8) return launch<T, 1, 2>(p, st);
  if (p.m <= 16) return launch<T, 2, 1>(p, st);
  return launch<T, 4, 1>(p, st);
}

template <typename T>
cudaError_t run_gradients(const GatedTokenParams& g, Mat dx, Mat dw_gate, Mat dw_up, int d,
                          cudaStream_t st) {
  const cudaError_t err = launch<T, 1, 2, true>(g, st);
  if (err != cudaSuccess) return err;
  const TokenGradientParams p{g.x, {g.w[0], g.w[1]}, g.ld_x, {g.ld_w[0], g.ld_w[1]}, {}, {}, g.work,
                              g.m, g.f, d, 0};
  if (g.m <= 1) return launch_gradients<T, 1>(p, dx, dw_gate, dw_up, st);
  if (g.m <= 2) return launch_gradients<T, 2>(p, dx, dw_gate, dw_up, st);
  if (g.m <= 4) return launch_gradients<T, 4>(p, dx, dw_gate, dw_up, st);
  return launch_gradients<T, 8>(p, dx, dw_gate, dw_up, st);
}

}  // namespace

cudaError_t launch_gated_tokens(CMat x, CMat w_gate, CMat w_up, Mat h, int type, int act, int m,
                                int f, int d, cudaStream_t st) {
  const GatedTokenParams p{(const uint8_t*)x.p, {(const uint8_t*)w_gate.p, (const uint8_t*)w_up.p},
                           x.ld * 2, {w_gate.ld * 2, w_up.ld * 2}, h.p, h.ld, nullptr, 0,
                           nullptr, act, m, f,
                           (int64_t)d * 2, (int)(((int64_t)d + 63) / 64)};
  return type == FWT_BF16 ? run<__nv_bfloat16>(p, st) : run<__half>(p, st);
}

cudaError_t launch_gated_token_gradients(CMat grad, CMat x, CMat w_gate, CMat w_up, Mat dx,
                                         Mat dw_gate, Mat dw_up, void* work, int type, int act,
                                         int m, int f, int d, cudaStream_t st) {
  const GatedTokenParams p{(const uint8_t*)x.p, {(const uint8_t*)w_gate.p, (const uint8_t*)w_up.p},
                           x.ld * 2, {w_gate.ld * 2, w_up.ld * 2}, nullptr, 0, grad.p, grad.ld,
                           (float*)work, act, m, f, (int64_t)d * 2, (int)(((int64_t)d + 63) / 64)};
  return type == FWT_BF16
             ? run_gradients<__nv_bfloat16>(p, dx, dw_gate, dw_up, d, st)
             : run_gradients<__half>(p, dx, dw_gate, dw_up, d, st);
}

}  // namespace ff
}  // namespace fwt
