// C entries of the feed-forward operators: argument checks, then the launchers.
#include <algorithm>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "feed_forward.cuh"
#include "fwt.h"

namespace fwt {
void set_last_cuda_error(int err);

namespace ff {
namespace {

constexpr int64_t kMaxExtent = 0x7fffff00;  // extents are 32-bit inside the kernels

int type_size(int type) { return type == FWT_F32 ? 4 : type == FWT_BF16 || type == FWT_F16 ? 2 : 0; }

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned_to(const void* p, int size) { return ((uintptr_t)p % (unsigned)size) == 0; }

// A matrix argument in bytes, for the overlap checks.
struct Window {
  uintptr_t p;
  int64_t rows, width, pitch;
};

// False where ld or the extent cannot be: columns beyond ld, or a last byte beyond 2^62.
bool window(const void* p, int64_t rows, int64_t cols, int64_t ld, int size, Window& w) {
  if (rows < 0 || cols < 0 || rows > kMaxExtent || cols > kMaxExtent || ld < cols) return false;
  if (rows > 1 && ld > (int64_t{1} << 62) / size / rows) return false;
  if (ld > (int64_t{1} << 58)) return false;
  w = {(uintptr_t)p, rows, cols * size, ld * size};
  return !(rows > 0 && cols > 0 && !p);
}

// Whether two matrices share a byte.  Column windows of one matrix (the same pitch, or the
// one row of a window that has no other; disjoint columns) do not.
bool overlap(const Window& a, const Window& b) {
  if (!a.rows || !b.rows || !a.width || !b.width) return false;
  const uintptr_t a_end = a.p + (uintptr_t)((a.rows - 1) * a.pitch + a.width);
  const uintptr_t b_end = b.p + (uintptr_t)((b.rows - 1) * b.pitch + b.width);
  if (a.p >= b_end || b.p >= a_end) return false;
  const int64_t pitch = a.rows > 1 ? a.pitch : b.pitch;
  if ((b.rows > 1 && b.pitch != pitch) || pitch == 0 || a.width > pitch || b.width > pitch) return true;
  const int64_t d = (int64_t)((b.p >= a.p ? (b.p - a.p) % (uintptr_t)pitch
                                          : (pitch - (int64_t)((a.p - b.p) % (uintptr_t)pitch)) % pitch));
  return !(d >= a.width && d + b.width <= pitch);
}

int done(cudaError_t err) {
  if (err == cudaSuccess) return FWT_OK;
  set_last_cuda_error((int)err);
  return FWT_ERR_CUDA;
}

// rows x cols of zero; rows and cols may be 0.
cudaError_t zero(Mat c, int size, int64_t rows, int64_t cols, cudaStream_t st) {
  if (!rows || !cols) return cudaSuccess;
  return cudaMemset2DAsync(c.p, (size_t)(c.ld * size), 0, (size_t)(cols * size), (size_t)rows, st);
}

bool misaligned_rows(const void* p, int64_t ld, int size) {
  return !aligned16(p) || (ld * size) % 16 != 0;
}

}  // namespace
}  // namespace ff
}  // namespace fwt

using namespace fwt::ff;

extern "C" {

int fwt_quantize_blocks(const void* x, int x_type, int64_t rows, int64_t cols, int64_t ld_x,
                        int rot_bits, int axis, int lines, void* q, int64_t ld_q, float* scale,
                        int64_t ld_scale, fwt_stream_t stream) {
  const int size = type_size(x_type);
  if (!size || rot_bits < 0 || rot_bits > 7 || (axis != 0 && axis != 1) ||
      (lines != 1 && lines != 128))
    return FWT_ERR_INVALID_ARG;
  Window wx, wq, ws;
  if (rows < 0 || cols < 0 || rows > kMaxExtent || cols > kMaxExtent) return FWT_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return FWT_OK;
  const int64_t nl = axis ? rows : cols;
  const int64_t group = int64_t{1} << rot_bits;
  const int64_t length = ((axis ? cols : rows) + group - 1) / group * group;
  if (!window(x, rows, cols, ld_x, size, wx) || !window(q, nl, length, ld_q, 1, wq) ||
      !window(scale, (nl + lines - 1) / lines, (length + 127) / 128, ld_scale, 4, ws))
    return FWT_ERR_INVALID_ARG;
  if (!aligned_to(x, size) || misaligned_rows(q, ld_q, 1) || !aligned_to(scale, 4))
    return FWT_ERR_MISALIGNED;
  if (overlap(wx, wq) || overlap(wx, ws) || overlap(wq, ws)) return FWT_ERR_INVALID_ARG;
  return done(launch_quantize({x, ld_x}, x_type, (int)rows, (int)cols, rot_bits, axis, lines,
                              {q, ld_q}, {scale, ld_scale}, (cudaStream_t)stream));
}

int fwt_matmul_blocks(const void* a, int64_t ld_a, const float* a_scale, int64_t ld_a_scale,
                      const void* b, int64_t ld_b, const float* b_scale, int64_t ld_b_scale,
                      int b_lines, void* c, int c_type, int64_t ld_c, int64_t m, int64_t n,
                      int64_t k, fwt_stream_t stream) {
  const int size = type_size(c_type);
  if (!size || (b_lines != 1 && b_lines != 128) || m < 0 || n < 0 || k < 0)
    return FWT_ERR_INVALID_ARG;
  if (m > kMaxExtent || n > kMaxExtent || k > kMaxExtent) return FWT_ERR_INVALID_ARG;
  if (m == 0 || n == 0) return FWT_OK;
  const int64_t blocks = (k + 127) / 128;
  Window wa, wb, wc, wsa, wsb;
  if (!window(a, m, k, ld_a, 1, wa) || !window(b, n, k, ld_b, 1, wb) ||
      !window(c, m, n, ld_c, size, wc) || !window(a_scale, m, blocks, ld_a_scale, 4, wsa) ||
      !window(b_scale, (n + b_lines - 1) / b_lines, blocks, ld_b_scale, 4, wsb))
    return FWT_ERR_INVALID_ARG;
  if (!aligned_to(c, size) || !aligned_to(a_scale, 4) || !aligned_to(b_scale, 4))
    return FWT_ERR_MISALIGNED;
  if (k == 0) return done(zero({c, ld_c}, size, m, n, (cudaStream_t)stream));
  if (misaligned_rows(a, ld_a, 1) || misaligned_rows(b, ld_b, 1)) return FWT_ERR_MISALIGNED;
  if (overlap(wc, wa) || overlap(wc, wb) || overlap(wc, wsa) || overlap(wc, wsb))
    return FWT_ERR_INVALID_ARG;
  return done(launch_matmul_blocks({a, ld_a}, {a_scale, ld_a_scale}, {b, ld_b},
                                   {b_scale, ld_b_scale}, b_lines, {c, ld_c}, c_type, (int)m,
                                   (int)n, (int)k, (cudaStream_t)stream));
}

int fwt_gated(const void* x, int64_t ld_x, const void* w_gate, int64_t ld_gate, const void* w_up,
              int64_t ld_up, void* h, int64_t ld_h, int type, int activation, int64_t m,
              int64_t f, int64_t d, fwt_stream_t stream) {
  if ((type != FWT_BF16 && type != FWT_F16) || activation < FWT_SILU || activation > FWT_RELU ||
      m < 0 || f < 0 || d < 0 || m > kMaxExtent || f > kMaxExtent || d > kMaxExtent)
    return FWT_ERR_INVALID_ARG;
  if (m == 0 || f == 0) return FWT_OK;
  Window wx, wg, wu, wh;
  if (!window(x, m, d, ld_x, 2, wx) || !window(w_gate, f, d, ld_gate, 2, wg) ||
      !window(w_up, f, d, ld_up, 2, wu) || !window(h, m, f, ld_h, 2, wh))
    return FWT_ERR_INVALID_ARG;
  if (!aligned_to(h, 2)) return FWT_ERR_MISALIGNED;
  if (d == 0) return done(zero({h, ld_h}, 2, m, f, (cudaStream_t)stream));
  if (misaligned_rows(x, ld_x, 2) || misaligned_rows(w_gate, ld_gate, 2) ||
      misaligned_rows(w_up, ld_up, 2))
    return FWT_ERR_MISALIGNED;
  if (overlap(wh, wx) || overlap(wh, wg) || overlap(wh, wu)) return FWT_ERR_INVALID_ARG;
  return done(launch_gated({x, ld_x}, {w_gate, ld_gate}, {w_up, ld_up}, {h, ld_h}, type,
                           activation, (int)m, (int)f, (int)d, (cudaStream_t)stream));
}

size_t fwt_gated_backward_workspace_bytes(int64_t m, int64_t f) {
  if (m <= 0 || f <= 0 || m > kMaxExtent || f > kMaxExtent) return 0;
  const size_t line = (size_t)((f + 7) / 8 * 8);
  if (m <= kMostGradientTokens) return line * 64;  // dg and du of 8 lines in fp32
  return (size_t)m * line * 4;                     // dg and du, rows of a multiple of 8
}

size_t fwt_gated_backward_workspace_bytes_for(int type, int64_t m, int64_t f) {
  const size_t both = fwt_gated_backward_workspace_bytes(m, f);
  if (type != FWT_BF16 && type != FWT_F16) return 0;
  return both && type == FWT_F16 && m > kMostGradientTokens ? both + kMostBounds * 8 : both;
}

int fwt_gated_backward(const void* grad, int64_t ld_grad, const void* x, int64_t ld_x,
                       const void* w_gate, int64_t ld_gate, const void* w_up, int64_t ld_up,
                       void* dx, int64_t ld_dx, void* dw_gate, int64_t ld_dw_gate, void* dw_up,
                       int64_t ld_dw_up, int type, int activation, int64_t m, int64_t f,
                       int64_t d, void* workspace, size_t workspace_bytes, fwt_stream_t stream) {
  if ((type != FWT_BF16 && type != FWT_F16) || activation < FWT_SILU || activation > FWT_RELU ||
      m < 0 || f < 0 || d < 0 || m > kMaxExtent || f > kMaxExtent || d > kMaxExtent)
    return FWT_ERR_INVALID_ARG;
  const bool want_dx = dx != nullptr, want_dw = dw_gate != nullptr;
  if (want_dw != (dw_up != nullptr)) return FWT_ERR_INVALID_ARG;
  if (d == 0 || (!want_dx && !want_dw)) return FWT_OK;  // every output is empty
  Window wdy, wx, wg, wu, wdx{}, wdg{}, wdu{};
  if (!window(grad, m, f, ld_grad, 2, wdy) || !window(x, m, d, ld_x, 2, wx) ||
      !window(w_gate, f, d, ld_gate, 2, wg) || !window(w_up, f, d, ld_up, 2, wu) ||
      (want_dx && !window(dx, m, d, ld_dx, 2, wdx)) ||
      (want_dw && (!window(dw_gate, f, d, ld_dw_gate, 2, wdg) ||
                   !window(dw_up, f, d, ld_dw_up, 2, wdu))))
    return FWT_ERR_INVALID_ARG;
  if ((want_dx && !aligned_to(dx, 2)) ||
      (want_dw && (!aligned_to(dw_gate, 2) || !aligned_to(dw_up, 2))))
    return FWT_ERR_MISALIGNED;
  cudaStream_t st = (cudaStream_t)stream;
  if (m == 0 || f == 0) {  // sums over nothing
    cudaError_t err = cudaSuccess;
    if (want_dx) err = zero({dx, ld_dx}, 2, m, d, st);
    if (want_dw && err == cudaSuccess) err = zero({dw_gate, ld_dw_gate}, 2, f, d, st);
    if (want_dw && err == cudaSuccess) err = zero({dw_up, ld_dw_up}, 2, f, d, st);
    return done(err);
  }
  if (!workspace || workspace_bytes < fwt_gated_backward_workspace_bytes_for(type, m, f))
    return FWT_ERR_INVALID_ARG;
  if (misaligned_rows(grad, ld_grad, 2) || misaligned_rows(x, ld_x, 2) ||
      misaligned_rows(w_gate, ld_gate, 2) || misaligned_rows(w_up, ld_up, 2) ||
      !aligned16(workspace))
    return FWT_ERR_MISALIGNED;
  const int64_t ws_bytes = (int64_t)fwt_gated_backward_workspace_bytes_for(type, m, f);
  const Window inputs[] = {wdy, wx, wg, wu, {(uintptr_t)workspace, 1, ws_bytes, ws_bytes}};
  const Window outputs[] = {wdx, wdg, wdu};
  for (int o = 0; o < 3; ++o) {
    for (const Window& in : inputs)
      if (overlap(outputs[o], in)) return FWT_ERR_INVALID_ARG;
    for (int o2 = 0; o2 < o; ++o2)
      if (overlap(outputs[o], outputs[o2])) return FWT_ERR_INVALID_ARG;
  }
  for (int i = 0; i < 4; ++i)
    if (overlap(inputs[i], inputs[4])) return FWT_ERR_INVALID_ARG;

  if (m <= kMostGradientTokens)
    return done(launch_gated_token_gradients({grad, ld_grad}, {x, ld_x}, {w_gate, ld_gate},
                                             {w_up, ld_up}, {dx, ld_dx}, {dw_gate, ld_dw_gate},
                                             {dw_up, ld_dw_up}, workspace, type, activation, (int)m,
                                             (int)f, (int)d, st));
  const int64_t ld = (f + 7) / 8 * 8;
  Mat dg{workspace, ld}, du{(char*)workspace + (size_t)m * (size_t)ld * 2, ld};
  const CMat cx{x, ld_x}, cg{w_gate, ld_gate}, cu{w_up, ld_up}, cdg{dg.p, ld}, cdu{du.p, ld};
  Bounds bounds{(float*)((char*)workspace + (size_t)m * (size_t)ld * 4), 0};
  cudaError_t err = cudaSuccess;
  if (type == FWT_F16)
    err = launch_gated_bounds({grad, ld_grad}, cx, cg, cu, bounds, (int)m, (int)f, (int)d, st);
  if (err == cudaSuccess)
    err = launch_gated_gradients({grad, ld_grad}, cx, cg, cu, dg, du, bounds, type, activation,
                                 (int)m, (int)f, (int)d, st);
  if (err == cudaSuccess && want_dx)
    err = launch_gated_dx(cdg, cdu, cg, cu, {dx, ld_dx}, bounds, type, (int)m, (int)f, (int)d, st);
  if (err == cudaSuccess && want_dw)
    err = launch_gated_dw(cdg, cdu, cx, {dw_gate, ld_dw_gate}, {dw_up, ld_dw_up}, bounds, type,
                          (int)m, (int)f, (int)d, st);
  return done(err);
}

}  // extern "C"
