// Keys and values into the cache and back: rotated, with a scale for each token and head.
//
//   append   y = 2^(-r/2) H x in fp32, s = the least 2^e with max |y| <= 448 s, codes e4m3(y / s)
//   read     x = 2^(-r/2) H (s codes)
//
// A row (a token's head) is spread over DIM / 16 lanes, 16 elements each: two runs of 8, half a
// row apart, so that the lanes of a row read and write whole sectors in one instruction.  Bits 0 to
// 2 and the top bit of the rotation are then among a lane's own elements, the others exchange
// with a neighbour lane.  Scales are powers of two: a floating-point code loses nothing by it (its
// relative step is the same at either end of a factor of two), and multiplying by one rounds nothing.
//
// Rows of several sequences lie one after the other; a CTA counts how many sequences end at or
// before its first row, and its rows go on from there.
//
// Bound, large: instructions, some 600 a thread for a key's and a value's 16 elements each, and between them waits
// that 28 warps of a multiprocessor do not cover: issue slots are 63% busy, warps that could issue and were not chosen
// wait about as long as those whose loads are on their way.  8192 x 8 x 128 bf16 18.5 us, 2.7 TB/s (every byte once
// takes 7.4); f32 18.6 us, 4.5 TB/s (12.4).  Reading back 4 x 4096 x 8 x 128 27.7 us, 3.7 TB/s (14.9), issue slots 75%
// busy; into f32 33.4 us, 5.0 TB/s (24.7).  Small: the chain of lookups, 3.3 us.
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "cache.cuh"
#include "feed_forward.cuh"
#include "ff_host.cuh"
#include "tma.cuh"

namespace fwt {
namespace ff {
namespace {

constexpr int kThreads = 256;
constexpr int kReadRows = 2;  // of a group of lanes that reads back: their places are looked up together

struct MoveParams {
  Divisor by_head;
  CacheView cache;
  Places at;
  Rows rows[2];
  int rot_bits;
};

// Sequences that end at or before packed row `row`; every thread of the CTA calls it.
__device__ __forceinline__ int sequences_before(const Places& at, int row) {
  int before = 0;
  for (int b0 = 0; b0 < at.sequences; b0 += kThreads) {
    const int b = b0 + (int)threadIdx.x;
    before += __syncthreads_count(b < at.sequences && at.starts[b + 1] <= row);
  }
  return before;
}

// Token and head of row `row` of a CTA's, which begin with row `first` of all.
struct FirstRow {
  int token, head;
};
__device__ __forceinline__ FirstRow first_row(const MoveParams& p, int64_t first) {
  FirstRow at;
  at.token = first < 0x7fffffff ? quotient((int)first, p.by_head) : (int)(first / p.cache.heads);
  at.head = (int)(first - (int64_t)at.token * p.cache.heads);
  return at;
}
__device__ __forceinline__ void row_at(const MoveParams& p, const FirstRow& at, int row, int& token, int& head) {
  const int more = quotient(at.head + row, p.by_head);
  token = at.token + more, head = at.head + row - more * p.cache.heads;
}

// The sequence of row `row`, from `b` on, and its place: the page and the slot in it, page -1 for
// none; false where the row is no sequence's.
__device__ __forceinline__ bool locate(const MoveParams& p, int row, int b, int& page, int& slot) {
  page = -1, slot = 0;
  while (b < p.at.sequences && p.at.starts[b + 1] <= row) ++b;
  if (b >= p.at.sequences) return false;
  const Sequence s = sequence(p.at, p.cache.page_tokens, b);
  if (row < s.row || row >= s.row + s.count) return false;
  const int pos = s.length - (s.row + s.count - row);
  if (pos >= 0) {
    page = page_of(p.cache, p.at, b, pos);
    slot = remainder(pos, p.cache.by_page);
  }
  return true;
}

template <typename T>
__device__ __forceinline__ void load8(const T* from, float* v) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 q = ((const float4*)from)[i];
      v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
    }
  } else {
    const uint4 q = *(const uint4*)from;
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = pair_to_float<T>(w[i]);
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* to, const float* v) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      ((float4*)to)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
    *(uint4*)to = make_uint4(pair_from_float<T>(v[0], v[1]), pair_from_float<T>(v[2], v[3]),
                             pair_from_float<T>(v[4], v[5]), pair_from_float<T>(v[6], v[7]));
  }
}

template <typename T, int DIM>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const MoveParams p) {
  constexpr int kLanes = DIM / 16, kRows = kThreads / kLanes;
  const int lane = threadIdx.x & (kLanes - 1), r = p.rot_bits;
  const FirstRow first = first_row(p, (int64_t)blockIdx.x * kRows);
  int token, head;
  row_at(p, first, threadIdx.x / kLanes, token, head);
  pdl_begin();
  // (lanes of a warp exchange: those without a row go along with zeros)
  float v[2][16];
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const T* from = (const T*)p.rows[o].p + token * p.rows[o].token + head * p.rows[o].head + 8 * lane;
    if (token < p.at.tokens) {  // on their way while the place is looked up
      load8(from, v[o]), load8(from + DIM / 2, v[o] + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[o][i] = 0.f;
    }
  }
  const int before = sequences_before(p.at, first.token);
  int page, slot;
  if (token >= p.at.tokens || !locate(p, token, before, page, slot)) page = -1;
  // 16 * 2^(-r/2) in two floats, and the product with them to the last bit but rarely: codes then differ from
  // those of exact arithmetic only where the sums do
  const float norm = rotation_after(r);
  const float norm_rest = r & 1 ? 16.f * __uint_as_float((uint32_t)(127 - r / 2) << 23) * 1.21016171e-8f : 0.f;
  const auto times = [](float2 x, float high, float rest) {
    const float2 h = make_float2(high, high), l = make_float2(rest, rest);
    const float2 p = fma_pair(x, h, make_float2(-0.f, -0.f));
    return add_pair(p, fma_pair(x, l, fma_pair(x, h, make_float2(-p.x, -p.y))));
  };
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    if (r) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[o][i] *= rotation_before(r);
      turn_spread<DIM>(v[o], r, lane);
    }
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(fabsf(v[o][i])));
    most = times(make_float2(most, most), norm, norm_rest).x;
    uint32_t top = __float_as_uint(most) & 0x7fffffffu;  // NaN is above all
#pragma unroll
    for (int step = 1; step < kLanes; step *= 2) top = max(top, __shfl_xor_sync(~0u, top, step));
    const uint32_t byte = scale_byte(__uint_as_float(top));
    // the norm and 1 / s in one product (in two where that could overflow)
    const uint32_t inverse = 254u - byte;
    const float power = __uint_as_float(min(inverse, 240u) << 23), factor = power * norm, factor_rest = power * norm_rest;
    if (inverse > 240u) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[o][i] *= __uint_as_float((127u + min(inverse - 240u, 14u)) << 23);
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = times(make_float2(v[o][4 * i], v[o][4 * i + 1]), factor, factor_rest);
      const float2 y = times(make_float2(v[o][4 * i + 2], v[o][4 * i + 3]), factor, factor_rest);
      w[i] = byte == 255u ? 0u : f32x2_to_e4m3(x.x, x.y) | f32x2_to_e4m3(y.x, y.y) << 16;
    }
    if (page >= 0) {
      const int64_t at = (int64_t)head * p.cache.page_tokens + slot;
      uint8_t* codes = p.cache.codes[o] + page * p.cache.code_stride[o] + at * DIM + 8 * lane;
      *(uint2*)codes = make_uint2(w[0], w[1]);
      *(uint2*)(codes + DIM / 2) = make_uint2(w[2], w[3]);
      if (lane == 0) p.cache.scales[o][page * p.cache.scale_stride[o] + at] = (uint8_t)byte;
    }
  }
}

template <typename T, int DIM>
__global__ void __launch_bounds__(kThreads, 4) read_kernel(const MoveParams p) {
  constexpr int kLanes = DIM / 16, kRows = kThreads / kLanes;
  const int lane = threadIdx.x & (kLanes - 1), r = p.rot_bits;
  const FirstRow first = first_row(p, (int64_t)blockIdx.x * (kRows * kReadRows));
  pdl_begin();
  const int before = sequences_before(p.at, first.token);
  int token[kReadRows], head[kReadRows];
  bool row[kReadRows];
  uint2 w[kReadRows][2][2];
  uint32_t byte[kReadRows][2];
#pragma unroll
  for (int k = 0; k < kReadRows; ++k) {
    row_at(p, first, k * kRows + threadIdx.x / kLanes, token[k], head[k]);
    int page = -1, slot = 0;
    row[k] = token[k] < p.at.tokens && locate(p, token[k], before, page, slot);
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      w[k][o][0] = w[k][o][1] = make_uint2(0, 0), byte[k][o] = 127;
      if (page >= 0) {
        const int64_t at = (int64_t)head[k] * p.cache.page_tokens + slot;
        const uint8_t* codes = p.cache.codes[o] + page * p.cache.code_stride[o] + at * DIM + 8 * lane;
        w[k][o][0] = *(const uint2*)codes, w[k][o][1] = *(const uint2*)(codes + DIM / 2);
        byte[k][o] = p.cache.scales[o][page * p.cache.scale_stride[o] + at];
      }
    }
  }
  const float norm = rotation_norm(r);
#pragma unroll
  for (int k = 0; k < kReadRows; ++k)
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t q = i & 1 ? w[k][o][i / 2].y : w[k][o][i / 2].x;
        const float2 lo = pair_to_float<__half>(e4m3_to_f16x2(q));
        const float2 hi = pair_to_float<__half>(e4m3_to_f16x2(q >> 16));
        v[4 * i] = lo.x, v[4 * i + 1] = lo.y, v[4 * i + 2] = hi.x, v[4 * i + 3] = hi.y;
      }
      turn_spread<DIM>(v, r, lane);  // of codes: their sums are exact or nearly so
      const float scale = scale_value(byte[k][o]);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = v[i] * norm * scale;
      if (row[k]) {
        T* to = (T*)p.rows[o].p + token[k] * p.rows[o].token + head[k] * p.rows[o].head + 8 * lane;
        store8(to, v), store8(to + DIM / 2, v + 8);
      }
    }
}

template <template <typename, int> class Kernel, typename T>
cudaError_t launch_dim(const MoveParams& p, int dim, const char* what, cudaStream_t st) {
  const int64_t pairs = (int64_t)p.at.tokens * p.cache.heads, rows = kThreads / (dim / 16) * Kernel<T, 64>::rows_each();
  const int64_t grid = (pairs + rows - 1) / rows;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  log_kernel("%s tokens=%d heads=%d dim=%d | rows a CTA=%lld", what, p.at.tokens, p.cache.heads, dim,
             (long long)rows);
  return launch_overlapped(dim == 64 ? Kernel<T, 64>::get() : Kernel<T, 128>::get(), (unsigned)grid,
                           kThreads, 0, 1, st, p);
}
template <typename T, int DIM>
struct Append {
  static int rows_each() { return 1; }
  static auto get() { return append_kernel<T, DIM>; }
};
template <typename T, int DIM>
struct Read {
  static int rows_each() { return kReadRows; }
  static auto get() { return read_kernel<T, DIM>; }
};
template <template <typename, int> class Kernel>
cudaError_t launch_type(const MoveParams& p, int type, int dim, const char* what, cudaStream_t st) {
  if (type == FWT_F32) return launch_dim<Kernel, float>(p, dim, what, st);
  if (type == FWT_F16) return launch_dim<Kernel, __half>(p, dim, what, st);
  return launch_dim<Kernel, __nv_bfloat16>(p, dim, what, st);
}

}  // namespace

cudaError_t launch_cache_append(Rows k, Rows v, int type, int dim, int rot_bits, const CacheView& cache,
                                const Places& at, cudaStream_t st) {
  return launch_type<Append>(MoveParams{divisor((uint32_t)cache.heads), cache, at, {k, v}, rot_bits}, type, dim, "cache_append", st);
}

cudaError_t launch_cache_read(Rows k, Rows v, int type, int dim, int rot_bits, const CacheView& cache,
                              const Places& at, cudaStream_t st) {
  return launch_type<Read>(MoveParams{divisor((uint32_t)cache.heads), cache, at, {k, v}, rot_bits}, type, dim, "cache_read", st);
}

}  // namespace ff
}  // namespace fwt
