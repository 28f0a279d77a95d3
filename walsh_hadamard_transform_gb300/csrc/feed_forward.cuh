// Launchers of the feed-forward operators' kernels, called by their C entries in
// ff_api.cu once the arguments are checked.  Every extent is at least 1 here unless a
// launcher says otherwise, and fits 31 bits.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace fwt {
namespace ff {

// A row-major matrix: rows of `ld` elements apart.
struct Mat {
  void* p;
  int64_t ld;
};
struct CMat {
  const void* p;
  int64_t ld;
};

cudaError_t launch_quantize(CMat x, int x_type, int rows, int cols, int rot_bits, int axis,
                            int lines, Mat q, Mat scale, cudaStream_t st);

cudaError_t launch_matmul_blocks(CMat a, CMat a_scale, CMat b, CMat b_scale, int b_lines, Mat c,
                                 int c_type, int m, int n, int k, cudaStream_t st);

cudaError_t launch_gated(CMat x, CMat w_gate, CMat w_up, Mat h, int type, int activation, int m,
                         int f, int d, cudaStream_t st);

// The same for a few lines of the first operand, at most kMostTokens.
constexpr int kMostTokens = 32;
cudaError_t launch_matmul_tokens(CMat a, CMat a_scale, CMat b, CMat b_scale, int b_lines, Mat c,
                                 int c_type, int m, int n, int k, cudaStream_t st);
cudaError_t launch_gated_tokens(CMat x, CMat w_gate, CMat w_up, Mat h, int type, int activation,
                                int m, int f, int d, cudaStream_t st);

// The gradients for at most kMostGradientTokens lines, all in fp32 up to their one rounding.
// `work`: 64 bytes for each of f.  dx, or dw_gate and dw_up, may be null.
constexpr int kMostGradientTokens = 8;
cudaError_t launch_gated_token_gradients(CMat grad, CMat x, CMat w_gate, CMat w_up, Mat dx,
                                         Mat dw_gate, Mat dw_up, void* work, int type,
                                         int activation, int m, int f, int d, cudaStream_t st);

// For float16, what dg and du are multiplied by to stay in its range: a power of two from a bound
// on them all, which is the product of the largest first and the largest second of `parts` pairs.
struct Bounds {
  float* pairs;
  int parts;
};
constexpr int kMostBounds = 512;
cudaError_t launch_gated_bounds(CMat grad, CMat x, CMat w_gate, CMat w_up, Bounds& bounds, int m,
                                int f, int d, cudaStream_t st);

// dg and du into the workspace matrices, rows of ld elements (a multiple of 8).  (The bounds of
// these three are read for float16 alone.)
cudaError_t launch_gated_gradients(CMat grad, CMat x, CMat w_gate, CMat w_up, Mat dg, Mat du,
                                   Bounds bounds, int type, int activation, int m, int f, int d,
                                   cudaStream_t st);
// dx = dg w_gate + du w_up.
cudaError_t launch_gated_dx(CMat dg, CMat du, CMat w_gate, CMat w_up, Mat dx, Bounds bounds,
                            int type, int m, int f, int d, cudaStream_t st);
// dw_gate = dg^T x, dw_up = du^T x.
cudaError_t launch_gated_dw(CMat dg, CMat du, CMat x, Mat dw_gate, Mat dw_up, Bounds bounds,
                            int type, int m, int f, int d, cudaStream_t st);

// Read and clear the device error words of the kernels that wait (synchronising).
cudaError_t read_device_error_gated(unsigned int* out);
cudaError_t read_device_error_matmul(unsigned int* out);

}  // namespace ff
}  // namespace fwt
