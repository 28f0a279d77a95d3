// Gated projections h = act(x Wg^T) * (x Wu^T) and their gradients.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "feed_forward.cuh"
#include "fwt.h"

namespace fwt {
namespace ff {
namespace {

// sum_e a[i * a_i + e * a_e] * b[j * b_j + e * b_e] over e < k, a 16 x 16 tile a CTA.
struct Strided {
  const void* p;
  int64_t line, element;
};

template <typename T>
__device__ __forceinline__ float tile_dot(Strided a, Strided b, int i0, int j0, int m, int n,
                                          int k) {
  __shared__ float as[16][17], bs[16][17];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float sum = 0.f;
  for (int s = 0; s < k; s += 16) {
    const int e = s + tx;
    as[ty][tx] = i0 + ty < m && e < k
                     ? (float)((const T*)a.p)[(int64_t)(i0 + ty) * a.line + e * a.element] : 0.f;
    bs[ty][tx] = j0 + ty < n && e < k
                     ? (float)((const T*)b.p)[(int64_t)(j0 + ty) * b.line + e * b.element] : 0.f;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 16; ++q) sum = fmaf(as[ty][q], bs[tx][q], sum);
    __syncthreads();
  }
  return sum;
}

template <typename T, int ACT, bool BACKWARD>
__global__ void __launch_bounds__(256) gated_kernel(CMat x, CMat wg, CMat wu, CMat grad, Mat out0,
                                                    Mat out1, int m, int f, int d) {
  const int tiles = (f + 15) / 16, i0 = blockIdx.x / tiles * 16, j0 = blockIdx.x % tiles * 16;
  const float g = tile_dot<T>({x.p, x.ld, 1}, {wg.p, wg.ld, 1}, i0, j0, m, f, d);
  const float u = tile_dot<T>({x.p, x.ld, 1}, {wu.p, wu.ld, 1}, i0, j0, m, f, d);
  const int i = i0 + (threadIdx.x >> 4), j = j0 + (threadIdx.x & 15);
  if (i >= m || j >= f) return;
  float value, slope;
  activation<ACT>(g, value, slope);
  if constexpr (BACKWARD) {
    const float dh = (float)((const T*)grad.p)[(int64_t)i * grad.ld + j];
    ((T*)out0.p)[(int64_t)i * out0.ld + j] = (T)(dh * u * slope);
    ((T*)out1.p)[(int64_t)i * out1.ld + j] = (T)(dh * value);
  } else {
    ((T*)out0.p)[(int64_t)i * out0.ld + j] = (T)(value * u);
  }
}

// c = a1 b1 (+ a2 b2)
template <typename T>
__global__ void __launch_bounds__(256) product_kernel(Strided a1, Strided b1, Strided a2,
                                                      Strided b2, Mat c, int m, int n, int k) {
  const int tiles = (n + 15) / 16, i0 = blockIdx.x / tiles * 16, j0 = blockIdx.x % tiles * 16;
  float sum = tile_dot<T>(a1, b1, i0, j0, m, n, k);
  if (a2.p) sum += tile_dot<T>(a2, b2, i0, j0, m, n, k);
  const int i = i0 + (threadIdx.x >> 4), j = j0 + (threadIdx.x & 15);
  if (i < m && j < n) ((T*)c.p)[(int64_t)i * c.ld + j] = (T)sum;
}

int64_t tiles16(int m, int n) { return (((int64_t)m + 15) / 16) * (((int64_t)n + 15) / 16); }

template <typename T, int ACT, bool BACKWARD>
cudaError_t run_gated(CMat x, CMat wg, CMat wu, CMat grad, Mat o0, Mat o1, int m, int f, int d,
                      cudaStream_t st) {
  if (tiles16(m, f) > 0x7fffffff) return cudaErrorInvalidConfiguration;
  gated_kernel<T, ACT, BACKWARD>
      <<<(unsigned)tiles16(m, f), 256, 0, st>>>(x, wg, wu, grad, o0, o1, m, f, d);
  return cudaGetLastError();
}

template <typename T, bool BACKWARD>
cudaError_t run_gated(int act, CMat x, CMat wg, CMat wu, CMat grad, Mat o0, Mat o1, int m, int f,
                      int d, cudaStream_t st) {
  if (act == FWT_SILU) return run_gated<T, FWT_SILU, BACKWARD>(x, wg, wu, grad, o0, o1, m, f, d, st);
  if (act == FWT_GELU) return run_gated<T, FWT_GELU, BACKWARD>(x, wg, wu, grad, o0, o1, m, f, d, st);
  return run_gated<T, FWT_RELU, BACKWARD>(x, wg, wu, grad, o0, o1, m, f, d, st);
}

cudaError_t run_product(int type, Strided a1, Strided b1, Strided a2, Strided b2, Mat c, int m,
                        int n, int k, cudaStream_t st) {
  if (tiles16(m, n) > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)tiles16(m, n);
  if (type == FWT_BF16)
    product_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a1, b1, a2, b2, c, m, n, k);
  else
    product_kernel<__half><<<grid, 256, 0, st>>>(a1, b1, a2, b2, c, m, n, k);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated(CMat x, CMat w_gate, CMat w_up, Mat h, int type, int act, int m, int f,
                         int d, cudaStream_t st) {
  if (type == FWT_BF16)
    return run_gated<__nv_bfloat16, false>(act, x, w_gate, w_up, {}, h, {}, m, f, d, st);
  return run_gated<__half, false>(act, x, w_gate, w_up, {}, h, {}, m, f, d, st);
}

cudaError_t launch_gated_gradients(CMat grad, CMat x, CMat w_gate, CMat w_up, Mat dg, Mat du,
                                   int type, int act, int m, int f, int d, cudaStream_t st) {
  if (type == FWT_BF16)
    return run_gated<__nv_bfloat16, true>(act, x, w_gate, w_up, grad, dg, du, m, f, d, st);
  return run_gated<__half, true>(act, x, w_gate, w_up, grad, dg, du, m, f, d, st);
}

cudaError_t launch_gated_dx(CMat dg, CMat du, CMat w_gate, CMat w_up, Mat dx, int type, int m,
                            int f, int d, cudaStream_t st) {
  return run_product(type, {dg.p, dg.ld, 1}, {w_gate.p, 1, w_gate.ld}, {du.p, du.ld, 1},
                     {w_up.p, 1, w_up.ld}, dx, m, d, f, st);
}

cudaError_t launch_gated_dw(CMat dg, CMat du, CMat x, Mat dw_gate, Mat dw_up, int type, int m,
                            int f, int d, cudaStream_t st) {
  cudaError_t err = run_product(type, {dg.p, 1, dg.ld}, {x.p, 1, x.ld}, {}, {}, dw_gate, f, d, m, st);
  if (err != cudaSuccess) return err;
  return run_product(type, {du.p, 1, du.ld}, {x.p, 1, x.ld}, {}, {}, dw_up, f, d, m, st);
}

}  // namespace ff
}  // namespace fwt
