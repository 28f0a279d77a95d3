// C entries of the cache: argument checks, then the launchers.
#include <algorithm>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "cache.cuh"
#include "fwt.h"

namespace fwt {
void set_last_cuda_error(int err);

namespace ff {
namespace {

constexpr int64_t kMostTokens = int64_t{1} << 30;  // positions are 32-bit inside the kernels

int done(cudaError_t err) {
  if (err == cudaSuccess) return FWT_OK;
  set_last_cuda_error((int)err);
  return FWT_ERR_CUDA;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// What an operand spans, for the overlap checks; empty: begin = end.
struct Span {
  uintptr_t begin, end;
};
bool apart(const Span& a, const Span& b) {
  return a.begin == a.end || b.begin == b.end || a.end <= b.begin || b.end <= a.begin;
}

// Whether two operands of rows `pitch` bytes apart, of which they fill `width_a` and `width_b`, share
// a byte: windows side by side do not.
bool rows_apart(const Span& a, int64_t width_a, const Span& b, int64_t width_b, int64_t pitch) {
  if (apart(a, b)) return true;
  if (pitch <= 0) return false;
  const int64_t d = b.begin >= a.begin
                        ? (int64_t)((b.begin - a.begin) % (uintptr_t)pitch)
                        : (pitch - (int64_t)((a.begin - b.begin) % (uintptr_t)pitch)) % pitch;
  return d >= width_a && d + width_b <= pitch;
}

// A (tokens, heads, dim) operand of elements of `size` bytes: strides that hold a row, no negative
// ones, and rows on 16-byte boundaries.
int check_rows(const Rows& r, int64_t tokens, int64_t heads, int dim, int size, bool written, Span& span) {
  if (!r.p || r.token < 0 || r.head < 0) return FWT_ERR_INVALID_ARG;
  if (r.token > (int64_t{1} << 40) || r.head > (int64_t{1} << 40)) return FWT_ERR_INVALID_ARG;
  // rows of an output are apart: heads within tokens, or tokens within heads
  if (written) {
    const bool inner_head = (heads == 1 || r.head >= dim) && (tokens == 1 || r.token >= (heads - 1) * r.head + dim);
    const bool inner_token = (tokens == 1 || r.token >= dim) && (heads == 1 || r.head >= (tokens - 1) * r.token + dim);
    if (!inner_head && !inner_token) return FWT_ERR_INVALID_ARG;
  }
  const int64_t last = (tokens - 1) * r.token;
  if ((tokens > 1 && last / (tokens - 1) != r.token) || last > (int64_t{1} << 58)) return FWT_ERR_INVALID_ARG;
  const int64_t elements = last + (heads - 1) * r.head + dim;  // (heads at most 2^16)
  if (elements > (int64_t{1} << 59)) return FWT_ERR_INVALID_ARG;
  span = {(uintptr_t)r.p, (uintptr_t)r.p + (uintptr_t)(elements * size)};
  if (!aligned16(r.p) || (tokens > 1 && r.token * size % 16) || (heads > 1 && r.head * size % 16))
    return FWT_ERR_MISALIGNED;
  return FWT_OK;
}

// Windows of one tensor that differ in their heads, or lie anywhere apart.
bool operands_apart(const Rows& a, const Span& sa, const Rows& b, const Span& sb, int64_t tokens, int64_t heads,
                    int dim, int size) {
  if (apart(sa, sb)) return true;
  if (tokens < 2 || a.token != b.token) return false;
  return rows_apart(sa, ((heads - 1) * a.head + dim) * size, sb, ((heads - 1) * b.head + dim) * size, a.token * size);
}

struct Call {
  CacheView view;
  Places at;
  Span spans[4];  // codes and scales of keys, then of values
};

int check_cache(const fwt_cache* c, Call& call) {
  if (!c || (c->dim != 64 && c->dim != 128) || c->heads < 1 || c->heads > 65536 || c->page_tokens < 16 ||
      c->page_tokens > (1 << 20) || c->page_tokens % 16 || (int64_t)c->heads * c->page_tokens > 0x7fffffff || c->pages < 0 || c->pages > 0x7fffffff)
    return FWT_ERR_INVALID_ARG;
  uint8_t* const codes[2] = {(uint8_t*)c->k, (uint8_t*)c->v};
  uint8_t* const scales[2] = {(uint8_t*)c->k_scale, (uint8_t*)c->v_scale};
  const int64_t strides[2][2] = {{c->k_stride, c->k_scale_stride}, {c->v_stride, c->v_scale_stride}};
  const int64_t tokens = (int64_t)c->heads * c->page_tokens;
  bool straight = true;
  for (int o = 0; o < 2; ++o) {
    for (int s = 0; s < 2; ++s) {
      const int64_t page = s ? tokens : tokens * c->dim, stride = strides[o][s];
      const uint8_t* p = s ? scales[o] : codes[o];
      if (c->pages && !p) return FWT_ERR_INVALID_ARG;
      if (c->pages > 1 && (stride < page || stride > (int64_t{1} << 58) / c->pages)) return FWT_ERR_INVALID_ARG;
      if (!aligned16(p) || (c->pages > 1 && stride % 16)) straight = false;
      call.spans[2 * o + s] = {(uintptr_t)p, (uintptr_t)p + (uintptr_t)(c->pages ? (c->pages - 1) * stride + page : 0)};
    }
    call.view.codes[o] = codes[o], call.view.scales[o] = scales[o];
    call.view.code_stride[o] = strides[o][0], call.view.scale_stride[o] = strides[o][1];
  }
  call.view.pages = (int)c->pages, call.view.heads = c->heads, call.view.page_tokens = c->page_tokens;
  call.view.by_page = divisor((uint32_t)c->page_tokens);
  return straight ? FWT_OK : FWT_ERR_MISALIGNED;
}

int check_places(const fwt_sequences* s, int64_t tokens, Call& call) {
  if (!s || s->sequences < 0 || s->sequences > kMostTokens || s->most_pages < 0 ||
      s->most_pages > 0x7fffffff || tokens < 0 || tokens > kMostTokens)
    return FWT_ERR_INVALID_ARG;
  if (s->sequences && (!s->starts || !s->lengths || (s->most_pages && !s->table))) return FWT_ERR_INVALID_ARG;
  if (s->sequences > 1 && (s->ld_table < s->most_pages || s->ld_table > (int64_t{1} << 58) / s->sequences))
    return FWT_ERR_INVALID_ARG;
  if (((uintptr_t)s->starts | (uintptr_t)s->lengths | (uintptr_t)s->table) & 3u) return FWT_ERR_MISALIGNED;
  call.at = {s->table, s->ld_table, (int)s->most_pages, s->starts, s->lengths, (int)s->sequences, (int)tokens};
  return FWT_OK;
}

// The four arrays may be windows of one pool whose pages hold all of them, but share no byte.
bool cache_apart(const fwt_cache* c, const Call& call) {
  const int64_t tokens = (int64_t)c->heads * c->page_tokens;
  const int64_t widths[4] = {tokens * c->dim, tokens, tokens * c->dim, tokens};
  const int64_t strides[4] = {c->k_stride, c->k_scale_stride, c->v_stride, c->v_scale_stride};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j) {
      const int64_t pitch = c->pages > 1 && strides[i] == strides[j] ? strides[i] : 0;
      if (!rows_apart(call.spans[i], widths[i], call.spans[j], widths[j], pitch)) return false;
    }
  return true;
}

int type_size(int type) { return type == FWT_F32 ? 4 : type == FWT_BF16 || type == FWT_F16 ? 2 : 0; }

int most_rotation(int dim) { return dim == 64 ? 6 : 7; }

// Rows of an item.  A call whose sequences have few rows for each key head goes by groups of 8.  Measured by 8, by 16
// and by 256 rows, us on the device, 8 key heads of 128 over 4096 keys, bfloat16 queries:
//
//   rows of a key head        16               20              32               64
//   16 sequences        58   48  102    80   70  103    103   73  103    200  127  105
//   1 sequence          20   23   23    21   23   23     22   24   24     25   27   26
//
// So between 17 and 32 rows of many sequences the items of 16 rows would be 30% faster (float16 18%); their
// two passes over the keys then cost what the tile's chain does.
int item_rows(int64_t longest, int64_t group) {
  const int64_t rows = longest * group;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : kChunkRows;
}
int64_t workers_of(int rows) { return rows == kChunkRows ? kMostCtas : kMostCtas * kTokenWorkers; }

}  // namespace
}  // namespace ff
}  // namespace fwt

using namespace fwt::ff;

extern "C" {

int fwt_cache_append(const void* k, int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
                     int64_t v_head, int type, int64_t tokens, const fwt_cache* cache,
                     const fwt_sequences* sequences, int rot_bits, fwt_stream_t stream) {
  const int size = type_size(type);
  Call call;
  if (!size) return FWT_ERR_INVALID_ARG;
  int st = check_cache(cache, call);
  if (st == FWT_ERR_INVALID_ARG || rot_bits < 0 || rot_bits > most_rotation(cache->dim)) return FWT_ERR_INVALID_ARG;
  const int places = check_places(sequences, tokens, call);
  if (places == FWT_ERR_INVALID_ARG) return places;
  if (tokens == 0 || sequences->sequences == 0 || cache->pages == 0 || sequences->most_pages == 0) return FWT_OK;
  const Rows rows[2] = {{const_cast<void*>(k), k_token, k_head}, {const_cast<void*>(v), v_token, v_head}};
  Span spans[2];
  int worst = std::max(st, places);  // (misaligned, if anything)
  for (int o = 0; o < 2; ++o) {
    st = check_rows(rows[o], tokens, cache->heads, cache->dim, size, false, spans[o]);
    if (st == FWT_ERR_INVALID_ARG) return st;
    worst = std::max(worst, st);
  }
  if (worst) return worst;
  for (const Span& s : spans)
    for (const Span& c : call.spans)
      if (!apart(s, c)) return FWT_ERR_INVALID_ARG;
  if (!cache_apart(cache, call)) return FWT_ERR_INVALID_ARG;
  return done(launch_cache_append(rows[0], rows[1], type, cache->dim, rot_bits, call.view, call.at,
                                  (cudaStream_t)stream));
}

int fwt_cache_read(const fwt_cache* cache, const fwt_sequences* sequences, int rot_bits, void* k,
                   int64_t k_token, int64_t k_head, void* v, int64_t v_token, int64_t v_head, int type,
                   int64_t tokens, fwt_stream_t stream) {
  const int size = type_size(type);
  Call call;
  if (!size) return FWT_ERR_INVALID_ARG;
  int st = check_cache(cache, call);
  if (st == FWT_ERR_INVALID_ARG || rot_bits < 0 || rot_bits > most_rotation(cache->dim)) return FWT_ERR_INVALID_ARG;
  const int places = check_places(sequences, tokens, call);
  if (places == FWT_ERR_INVALID_ARG) return places;
  if (tokens == 0 || sequences->sequences == 0) return FWT_OK;
  const Rows rows[2] = {{k, k_token, k_head}, {v, v_token, v_head}};
  Span spans[2];
  int worst = std::max(st, places);
  for (int o = 0; o < 2; ++o) {
    st = check_rows(rows[o], tokens, cache->heads, cache->dim, size, true, spans[o]);
    if (st == FWT_ERR_INVALID_ARG) return st;
    worst = std::max(worst, st);
  }
  if (worst) return worst;
  if (!operands_apart(rows[0], spans[0], rows[1], spans[1], tokens, cache->heads, cache->dim, size))
    return FWT_ERR_INVALID_ARG;
  for (const Span& s : spans)
    for (const Span& c : call.spans)
      if (!apart(s, c)) return FWT_ERR_INVALID_ARG;
  return done(launch_cache_read(rows[0], rows[1], type, cache->dim, rot_bits, call.view, call.at,
                                (cudaStream_t)stream));
}

size_t fwt_cache_attention_workspace_bytes(int q_heads, int heads, int dim, int64_t longest) {
  if (heads < 1 || q_heads < 1 || q_heads > 65536 || q_heads % heads || (dim != 64 && dim != 128) ||
      longest < 0 || longest > kMostTokens)
    return 0;
  const int rows = item_rows(std::max<int64_t>(longest, 1), q_heads / heads);
  return (size_t)workers_of(rows) * (2 * sizeof(int4) + 2 * 4 * (size_t)part_floats(rows, dim));
}

int fwt_cache_attention(const void* q, int64_t q_token, int64_t q_head, void* out, int64_t out_token,
                        int64_t out_head, int type, int64_t tokens, int q_heads, const fwt_cache* cache,
                        const fwt_sequences* sequences, int rot_bits, float scale, int causal,
                        int64_t window, int64_t longest, void* workspace, size_t workspace_bytes,
                        fwt_stream_t stream) {
  Call call;
  scale *= 1.44269504088896341f;  // scores in powers of two
  if ((type != FWT_BF16 && type != FWT_F16) || (causal != 0 && causal != 1) || window < 0 || longest < 0 ||
      !(scale - scale == 0.f))
    return FWT_ERR_INVALID_ARG;
  int st = check_cache(cache, call);
  if (st == FWT_ERR_INVALID_ARG || rot_bits < 0 || rot_bits > most_rotation(cache->dim)) return FWT_ERR_INVALID_ARG;
  if (q_heads < 1 || q_heads > 65536 || q_heads % cache->heads) return FWT_ERR_INVALID_ARG;
  const int places = check_places(sequences, tokens, call);
  if (places == FWT_ERR_INVALID_ARG || tokens * q_heads > 0x7ffffe00) return FWT_ERR_INVALID_ARG;
  if (tokens == 0 || sequences->sequences == 0) return FWT_OK;
  const Rows rows[2] = {{const_cast<void*>(q), q_token, q_head}, {out, out_token, out_head}};
  Span spans[2];
  int worst = std::max(st, places);
  for (int o = 0; o < 2; ++o) {
    st = check_rows(rows[o], tokens, q_heads, cache->dim, 2, o == 1, spans[o]);
    if (st == FWT_ERR_INVALID_ARG) return st;
    worst = std::max(worst, st);
  }
  // (the longest sequence has no more rows than there are; 0: as if all had the same)
  if (longest == 0) longest = (tokens + sequences->sequences - 1) / sequences->sequences;
  longest = std::min(longest, tokens);
  const size_t need = fwt_cache_attention_workspace_bytes(q_heads, cache->heads, cache->dim, longest);
  if (!workspace || workspace_bytes < need) return FWT_ERR_INVALID_ARG;
  if (!aligned16(workspace)) worst = FWT_ERR_MISALIGNED;
  if (worst) return worst;
  const Span work{(uintptr_t)workspace, (uintptr_t)workspace + need};
  if (!operands_apart(rows[0], spans[0], rows[1], spans[1], tokens, q_heads, cache->dim, 2) ||
      !apart(work, spans[0]) || !apart(work, spans[1]))
    return FWT_ERR_INVALID_ARG;
  for (const Span& c : call.spans)
    if (!apart(spans[1], c) || !apart(work, c)) return FWT_ERR_INVALID_ARG;
  AttentionParams p;
  p.cache = call.view, p.at = call.at, p.q = rows[0], p.out = rows[1];
  p.type = type, p.group = q_heads / cache->heads, p.by_group = divisor((uint32_t)p.group), p.dim = cache->dim, p.rot_bits = rot_bits;
  p.scale = scale;
  p.causal = causal, p.window = window < kMostLength ? (int)window : 0;  // (as long as any sequence: none)
  const int rows_each = item_rows(longest, p.group);
  p.notes = (int4*)workspace, p.parts = (float*)((char*)workspace + workers_of(rows_each) * 2 * sizeof(int4));
  return done(rows_each == kChunkRows ? launch_attention_chunk(p, (cudaStream_t)stream)
                                      : launch_attention_tokens(p, rows_each, (cudaStream_t)stream));
}

}  // extern "C"
