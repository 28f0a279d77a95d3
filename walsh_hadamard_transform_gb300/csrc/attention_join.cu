// Items of attention that several CTAs shared, put together from their parts: see attention_plan.cuh.
//
//   m = max m_i,  w_i = 2^(m_i - m),  out = R (sum w_i O_i) / (sum w_i l_i)
//
// A warp takes a row; its lanes first a part's maximum and total each, then all of the row's
// elements, parts in the order of the keys.  Bound: latency, a few microseconds less what the launch
// overlaps; the parts were written just before and come from L2.
#include <cstdint>

#include <cuda_runtime.h>

#include "attention_plan.cuh"
#include "cache.cuh"
#include "feed_forward.cuh"
#include "ff_host.cuh"
#include "tma.cuh"

namespace fwt {
namespace ff {
namespace {

constexpr int kWarps = 8;

template <int DIM>
__global__ void __launch_bounds__(kWarps * 32) join_kernel(const AttentionParams p, int rows_all, int workers) {
  const int lane = threadIdx.x & 31;
  const int owner = blockIdx.x % workers, r = blockIdx.x / workers * kWarps + (threadIdx.x >> 5);
  pdl_begin();
  const int4 note = p.notes[owner];
  if (!(note.x & kNoteTail)) return;
  const Sequence s = sequence(p.at, p.cache.page_tokens, note.y);
  const int64_t row = (int64_t)note.w * rows_all + r;
  if (r >= rows_all || row >= (int64_t)s.count * p.group) return;
  const int64_t floats = part_floats(rows_all, DIM);
  // parts: 2 owner + 1, then 2 i of the CTAs that follow, up to the one that ends the item
  int last = workers - 1;
  for (int i0 = owner + 1; i0 < workers; i0 += 32) {
    const uint32_t ends = __ballot_sync(~0u, i0 + lane < workers && (p.notes[min(i0 + lane, workers - 1)].x & kNoteHeadEnds));
    if (ends) {
      last = i0 + __ffs(ends) - 1;
      break;
    }
  }
  constexpr int kOwn = DIM / 32;
  float m = -INFINITY;
  for (int i = owner + lane; i <= last; i += 32)
    m = fmaxf(m, p.parts[(2 * (int64_t)i + (i == owner)) * floats + rows_all * DIM + r]);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f, v[kOwn];
#pragma unroll
  for (int j = 0; j < kOwn; ++j) v[j] = 0.f;
#pragma unroll 8
  for (int i = owner; i <= last; ++i) {
    const float* part = p.parts + (2 * (int64_t)i + (i == owner)) * floats;
    const float top = part[rows_all * DIM + r], total = part[rows_all * DIM + rows_all + r];
    // (a part with no maximum has seen nothing, or only what is not a number)
    const float w = top == -INFINITY ? 1.f : exp2f(top - base);
    l = fmaf(total, w, l);
#pragma unroll
    for (int j = 0; j < kOwn; ++j) v[j] = fmaf(part[(int64_t)r * DIM + kOwn * lane + j], w, v[j]);
  }
  turn_row<DIM>(v, p.rot_bits, lane);
  const float norm = l == 0.f ? 0.f : rotation_norm(p.rot_bits) / l;
  const int token = s.row + quotient((int)row, p.by_group), head = note.z * p.group + remainder((int)row, p.by_group);
  uint32_t* out = (uint32_t*)((uint16_t*)p.out.p + token * p.out.token + head * p.out.head + kOwn * lane);
#pragma unroll
  for (int j = 0; j < kOwn / 2; ++j) out[j] = pair_from_float(v[2 * j] * norm, v[2 * j + 1] * norm, p.type);
}

}  // namespace

cudaError_t launch_attention_join(const AttentionParams& p, int rows, int workers, cudaStream_t st) {
  const unsigned grid = (unsigned)(workers * ((rows + kWarps - 1) / kWarps));
  log_kernel("cache_attention join rows=%d workers=%d", rows, workers);
  return launch_overlapped(p.dim == 64 ? join_kernel<64> : join_kernel<128>, grid, kWarps * 32, 0, 1, st, p,
                           rows, workers);
}

}  // namespace ff
}  // namespace fwt
