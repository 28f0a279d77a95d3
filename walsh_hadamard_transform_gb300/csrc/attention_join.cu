// Items of attention that several CTAs shared, put together from their parts: see attention_plan.cuh.
//
//   m = max m_i,  w_i = 2^(m_i - m) l_i,  out = R sum (w_i / sum w_i) O_i
//
// O_i is the mean of the part's values: a sum of all their weights, and of a row for the rotation, may pass fp32 where
// the output does not.  A warp takes a row; its lanes first a part's maximum and total each, then all of the row's
// elements, parts in the order of the keys.  Bound: latency, a few microseconds less what the launch
// overlaps (of items of 8 rows: those of 16 and 256 make grids of over 2048 CTAs, which start when the
// kernel before has ended); the parts were written just before and come from L2.
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
  const int4 note = p.notes[2 * owner], at = p.notes[2 * owner + 1];
  if (!(note.x & kNoteTail)) return;
  const int row = note.w * rows_all + r;
  if (r >= rows_all || row >= at.y * p.group) return;
  const int64_t floats = part_floats(rows_all, DIM);
  const int last = min(note.y, workers - 1);  // parts: 2 owner + 1, then 2 i of the workers that follow
  constexpr int kOwn = DIM / 32;
  const auto read = [&](int i, float& top, float& total) {
    top = -INFINITY, total = 0.f;
    if (i > last) return;
    const float* part = p.parts + (2 * (int64_t)i + (i == owner)) * floats + rows_all * DIM + r;
    top = part[0], total = part[rows_all];
  };
  // (a part with no maximum has seen nothing, or only what is not a number)
  const auto weight = [](float top, float m) { return top == -INFINITY ? 1.f : exp2f(top - m); };
  float top, total;  // of the part owner + lane
  read(owner + lane, top, total);
  float m = top, l = total;
#pragma unroll 1
  for (int i = owner + lane + 32; i <= last; i += 32) {
    float other_top, other_total;
    read(i, other_top, other_total);
    const float both = fmaxf(m, other_top);
    l = l * weight(m, both) + other_total * weight(other_top, both), m = both;
  }
  const float mine = m;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  l *= weight(mine, m);
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
  const float inverse = l == 0.f ? 0.f : 1.f / l;
  float v[kOwn];
#pragma unroll
  for (int j = 0; j < kOwn; ++j) v[j] = 0.f;
  constexpr int kBatch = 8;  // parts on their way at a time
#pragma unroll 1
  for (int i0 = owner; i0 <= last; i0 += 32) {
    if (i0 != owner) read(i0 + lane, top, total);
    const float share = total * weight(top, m) * inverse;
#pragma unroll 1
    for (int k0 = 0; k0 < 32 && i0 + k0 <= last; k0 += kBatch) {
      float part_v[kBatch][kOwn];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = min(i0 + k0 + k, last);
        const float* part = p.parts + (2 * (int64_t)i + (i == owner)) * floats + r * DIM + kOwn * lane;
        if constexpr (kOwn == 4) {
          const float4 x = *(const float4*)part;
          part_v[k][0] = x.x, part_v[k][1] = x.y, part_v[k][2] = x.z, part_v[k][3] = x.w;
        } else {
          const float2 x = *(const float2*)part;
          part_v[k][0] = x.x, part_v[k][1] = x.y;
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float of_it = __shfl_sync(~0u, share, k0 + k);
        if (i0 + k0 + k <= last) {
#pragma unroll
          for (int j = 0; j < kOwn; ++j) v[j] = fmaf(part_v[k][j], of_it, v[j]);
        }
      }
    }
  }
  const float before = rotation_before(p.rot_bits), norm = rotation_after(p.rot_bits);
#pragma unroll
  for (int j = 0; j < kOwn; ++j) v[j] *= before;
  turn_row<DIM>(v, p.rot_bits, lane);
  const int token = at.x + quotient(row, p.by_group), head = note.z * p.group + remainder(row, p.by_group);
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
