// The cache of keys and values and how its kernels find their way in it.
//
// A page holds `page_tokens` tokens (a multiple of 16) of every head: codes as heads x tokens x dim
// bytes, so that 16 tokens of a head are one run of memory that no page boundary cuts, and scales
// as heads x tokens bytes, 16 of them one aligned 16-byte piece.
//
// Sequence b owns rows starts[b] .. starts[b + 1] of the packed operands: the last of its
// lengths[b] tokens in the cache.  Both arrays are device memory that the host never reads, so
// every kernel clamps what it takes from them: rows to the packed operand, lengths to the table,
// and a page that is not one of the cache's holds nothing.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fwt.h"

namespace fwt {
namespace ff {

// Division by a number that the host knows, of 0 <= n < 2^31: with 2^s >= d > 2^(s-1) and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (floor(n m / 2^32) + n) / 2^s, rounded down (Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994).
struct Divisor {
  uint32_t d, multiplier, shift;
};
inline Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while (s < 31 && (1u << s) < d) ++s;
  return {d, (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - d)) / d + 1), s};
}
__device__ __forceinline__ int quotient(int n, const Divisor& by) {
  return (int)((__umulhi((uint32_t)n, by.multiplier) + (uint32_t)n) >> by.shift);
}
__device__ __forceinline__ int remainder(int n, const Divisor& by) { return n - quotient(n, by) * (int)by.d; }

struct CacheView {
  uint8_t* codes[2];  // keys, values
  uint8_t* scales[2];
  int64_t code_stride[2], scale_stride[2];  // bytes from page to page
  int pages, heads, page_tokens;
  Divisor by_page;  // page_tokens
};

struct Places {
  const int32_t* table;
  int64_t ld_table;
  int most_pages;
  const int32_t *starts, *lengths;
  int sequences, tokens;  // tokens: rows of the packed operands
};

// Rows of heads apart: element strides of a (tokens, heads, dim) operand.
struct Rows {
  void* p;
  int64_t token, head;
};

struct AttentionParams {
  CacheView cache;
  Places at;
  Rows q, out;
  int type, group, dim, rot_bits;
  Divisor by_group;
  float scale;   // of the scores, times log2(e)
  int causal, window;
  float* parts;  // see attention_plan.cuh
  int4* notes;
};

// Launchers, their arguments checked (ff_api.cu's manner): every extent is at least 1.
cudaError_t launch_cache_append(Rows k, Rows v, int type, int dim, int rot_bits, const CacheView& cache,
                                const Places& at, cudaStream_t st);
cudaError_t launch_cache_read(Rows k, Rows v, int type, int dim, int rot_bits, const CacheView& cache,
                              const Places& at, cudaStream_t st);
cudaError_t launch_attention_tokens(const AttentionParams& p, int rows, cudaStream_t st);
cudaError_t launch_attention_chunk(const AttentionParams& p, cudaStream_t st);
constexpr int kChunkRows = 256;  // rows of an item there
cudaError_t launch_attention_join(const AttentionParams& p, int rows, int workers, cudaStream_t st);

constexpr int kMostCtas = 192;   // of an attention kernel
constexpr int kTokenWorkers = 8;  // of a CTA there, where rows are few; the workspace has room for their parts

// A worker's two parts: rows x dim means, then a maximum and a total for each row.
__host__ __device__ constexpr int64_t part_floats(int rows, int dim) { return (int64_t)rows * (dim + 2); }

// The tensor cores round their sums toward zero, each time by up to 2^-23 of the sum so far: over a million keys of one
// share outputs were 0.7% short.  So after this many keys a worker adds its sums to those before in fp32, to
// nearest, and begins again: outputs are then short by some 2^-13 at most.  (With many rows a share of up to twice as
// many keys goes on in one sum, and the last ones are added to all.)  Sums wait in the worker's part that they would
// be written to in the end, and those of p beside them (one fp32 number of a lane for every eighth of a million keys was off
// by 0.2%: equal numbers round alike).  4096 tokens over 32768: 1.885 ms, and 1.88 without.
constexpr int kSumKeys = 8192;

constexpr int kMostLength = 0x7fff0000;  // tokens of a sequence (sums with a tile's fit 31 bits)

struct Sequence {
  int row, count, length;  // first packed row, rows, tokens in the cache
};

__device__ __forceinline__ Sequence sequence(const Places& at, int pages_tokens, int b) {
  Sequence s;
  s.row = min(max(at.starts[b], 0), at.tokens);
  s.count = min(max(at.starts[b + 1], s.row), at.tokens) - s.row;
  const int64_t room = min((int64_t)at.most_pages * pages_tokens, (int64_t)kMostLength);
  s.length = (int)min((int64_t)max(at.lengths[b], 0), room);
  return s;
}

// The page of token `pos` (below the sequence's length), -1 where there is none.
__device__ __forceinline__ int page_of(const CacheView& c, const Places& at, int b, int pos) {
  const int page = at.table[(int64_t)b * at.ld_table + quotient(pos, c.by_page)];
  return (unsigned)page < (unsigned)c.pages ? page : -1;
}

// ---- 8-bit values ----------------------------------------------------------------------

// Two e4m3 codes (16 bits) as float16: exact.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t codes) {
  uint32_t v;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(v) : "h"((unsigned short)codes));
  return v;
}
// float32 to e4m3, to nearest even, beyond 448 to 448.
__device__ __forceinline__ uint32_t f32x2_to_e4m3(float lo, float hi) {
  unsigned short v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}

// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fc00000u) : byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);
}

// The scale byte of a row of largest magnitude `top`: the least power of two from 2^-126 on that
// takes it to 448 = 1.75 * 2^8 or below, 255 where it is not finite.  (2^-126 is the least whose
// inverse is a finite float.)
__device__ __forceinline__ uint32_t scale_byte(float top) {
  const uint32_t bits = __float_as_uint(top) & 0x7fffffffu;
  if (bits >= 0x7f800000u) return 255u;
  const int e = (int)((bits + 0x1fffffu) >> 23) - 8;  // (a mantissa above 1.75 carries)
  return (uint32_t)max(e, 1);
}

// ---- 16-bit and 32-bit rows ------------------------------------------------------------

template <typename T>
__device__ __forceinline__ float2 pair_to_float(uint32_t v) {
  if constexpr (sizeof(T) == 2) {
    if constexpr (std::is_same<T, __half>::value) return __half22float2(*(const __half2*)&v);
    else return __bfloat1622float2(*(const __nv_bfloat162*)&v);
  }
  return make_float2(0.f, 0.f);
}
template <typename T>
__device__ __forceinline__ uint32_t pair_from_float(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 v = __floats2half2_rn(a, b);
    return *(const uint32_t*)&v;
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *(const uint32_t*)&v;
  }
}
// Either 16-bit type by its code.
__device__ __forceinline__ float2 pair_to_float(uint32_t v, int type) {
  return type == FWT_F16 ? pair_to_float<__half>(v) : pair_to_float<__nv_bfloat16>(v);
}
__device__ __forceinline__ uint32_t pair_from_float(float a, float b, int type) {
  return type == FWT_F16 ? pair_from_float<__half>(a, b) : pair_from_float<__nv_bfloat16>(a, b);
}

// ---- two fp32 at a time ---------------------------------------------------------------

__device__ __forceinline__ float2 fma_pair(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add_pair(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// ---- the rotation ----------------------------------------------------------------------

// 2^(-r / 2).
__device__ __forceinline__ float rotation_norm(int r) {
  return __uint_as_float((uint32_t)(127 - r / 2) << 23) * (r & 1 ? 0.70710678118654752f : 1.f);
}

// The same around the sums: 1/16 before them and the rest after, so that no sum of 128 passes fp32 where the
// rotated row does not.
__device__ __forceinline__ float rotation_before(int r) { return r ? 0.0625f : 1.f; }
__device__ __forceinline__ float rotation_after(int r) { return r ? 16.f * rotation_norm(r) : 1.f; }

// One bit of the rotation among a thread's own values, STEP apart.
template <int N, int STEP>
__device__ __forceinline__ void turn_own(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (!(i & STEP)) {
      const float a = v[i], b = v[i + STEP];
      v[i] = a + b, v[i + STEP] = a - b;
    }
}
// One bit across lanes `step` apart.
template <int N>
__device__ __forceinline__ void turn_lanes(float (&v)[N], int step, int lane) {
  const float sign = lane & step ? -1.f : 1.f;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = fmaf(sign, v[i], __shfl_xor_sync(~0u, v[i], step));
}

// A row over DIM / 16 lanes, each with 8 elements from 8 `lane` on and 8 half a row on: without the norm.
template <int DIM>
__device__ __forceinline__ void turn_spread(float (&v)[16], int r, int lane) {
  constexpr int kBits = DIM == 128 ? 7 : 6;
  if (r > 0) turn_own<16, 1>(v);
  if (r > 1) turn_own<16, 2>(v);
  if (r > 2) turn_own<16, 4>(v);
#pragma unroll
  for (int bit = 3; bit < kBits - 1; ++bit)
    if (r > bit) turn_lanes(v, 1 << (bit - 3), lane);
  if (r == kBits) turn_own<16, 8>(v);
}

// A row of DIM over the 32 lanes of a warp, DIM / 32 consecutive elements each, without the norm.
template <int DIM>
__device__ __forceinline__ void turn_row(float (&v)[DIM / 32], int r, int lane) {
  constexpr int kOwn = DIM == 128 ? 2 : 1;  // bits of a lane's own elements
  if (r > 0) turn_own<DIM / 32, 1>(v);
  if constexpr (DIM == 128)
    if (r > 1) turn_own<DIM / 32, 2>(v);
#pragma unroll
  for (int bit = 0; bit < 5; ++bit)
    if (r > kOwn + bit) turn_lanes(v, 1 << bit, lane);
}

}  // namespace ff
}  // namespace fwt
