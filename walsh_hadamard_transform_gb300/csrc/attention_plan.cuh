// How attention over the cache is shared out among CTAs.
//
// An item is a block of ROWS rows (new tokens x query heads of one key head) of a sequence with one
// key head; its keys, from the first that one of its rows sees, are cut into units of UNIT tokens, at
// least one.  All units of the call, in the order of sequences, key heads, blocks, are dealt out in
// equal consecutive shares, so that a CTA's work does not depend on how lengths are spread; a share
// begins and ends inside an item as it may.  The host does not know the lengths: every CTA adds
// them up for itself.
//
// What a CTA has done of an item that is not all its own goes to the workspace: part 2 i of CTA i is
// of the item that its share begins in the middle of, part 2 i + 1 of the one that it ends in the
// middle of.  notes[i] says which there are, and launch_attention_join() puts them together in the
// order of the keys, so that results depend on nothing but the arguments.
#pragma once

#include <cstdint>

#include "cache.cuh"

namespace fwt {
namespace ff {

// notes[i]: x flags, then sequence, key head and block of part 2 i + 1.
constexpr int kNoteHead = 1;      // part 2 i is there
constexpr int kNoteHeadEnds = 2;  // and reaches the item's end
constexpr int kNoteTail = 4;      // part 2 i + 1 is there

// The keys of an item: [low, high), low a multiple of 16.
struct Keys {
  int low, high;
};

template <int ROWS>
__device__ __forceinline__ int blocks_of(const AttentionParams& p, const Sequence& s) {
  return (s.count * p.group + ROWS - 1) / ROWS;
}

template <int ROWS>
__device__ __forceinline__ Keys keys_of(const AttentionParams& p, const Sequence& s, int block) {
  // (rows and a block more fit 31 bits)
  const int first = quotient(block * ROWS, p.by_group);
  const int last = min(s.count - 1, quotient(block * ROWS + ROWS - 1, p.by_group));
  const int own = s.length - s.count;  // position of the first new token
  Keys k;
  k.high = p.causal ? min(s.length, max(own + last + 1, 0)) : s.length;
  k.low = p.window ? min(max(own + first + 1 - p.window, 0), k.high) & ~15 : 0;
  return k;
}

template <int UNIT>
__device__ __forceinline__ int units_of(const Keys& k) {
  return max(1, (k.high - k.low + UNIT - 1) / UNIT);
}

// Units of one key head of the sequences of a warp's lanes (sequence b in each; count 0: none).
// (What runs once or once an item is kept out of line: a kernel's loops have to stay in the instruction
// cache.  Inlined throughout, the kernels were of 150 and 320 KB, and four times as slow.)
template <int ROWS, int UNIT>
__device__ __forceinline__ int64_t units_of_sequence(const AttentionParams& p, const Sequence& s, int lane) {
  constexpr int kAlone = 4;  // blocks that a lane counts by itself
  const int blocks = blocks_of<ROWS>(p, s);
  int64_t units = 0;
  if (blocks <= kAlone)
    for (int i = 0; i < blocks; ++i) units += units_of<UNIT>(keys_of<ROWS>(p, s, i));
  for (uint32_t many = __ballot_sync(~0u, blocks > kAlone); many; many &= many - 1) {
    const int from = __ffs(many) - 1;
    Sequence t;
    t.row = 0;
    t.count = __shfl_sync(~0u, s.count, from), t.length = __shfl_sync(~0u, s.length, from);
    const int n = __shfl_sync(~0u, blocks, from);
    int64_t sum = 0;
    for (int i = lane; i < n; i += 32) sum += units_of<UNIT>(keys_of<ROWS>(p, t, i));
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == from) units = sum;
  }
  return units;
}

// Where a share stands: the item, the unit in it, and the units that are left of the share.
struct Walk {
  int b, head, block;
  Sequence s;
  Keys keys;
  int unit, units;  // of the item: the next one, and all
  int64_t left;     // units of the share from `unit` on
};

template <int THREADS>
struct PlanScratch {
  int64_t warp_units[THREADS / 32];
  int64_t rem, per_head;
  int b;
};

// The share of CTA `cta` of `ctas`; every thread of the CTA calls it.  left = 0: there is none.
template <int ROWS, int UNIT, int THREADS>
__device__ __forceinline__ Walk find_share(const AttentionParams& p, int cta, int ctas,
                                           PlanScratch<THREADS>& scratch) {
  constexpr int kWarps = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, heads = p.cache.heads;
  auto units_at = [&](int b) {
    Sequence s{0, 0, 0};
    if (b < p.at.sequences) s = sequence(p.at, p.cache.page_tokens, b);
    return units_of_sequence<ROWS, UNIT>(p, s, lane);
  };
  int64_t first = units_at((int)threadIdx.x), mine = first;
  for (int b0 = THREADS; b0 < p.at.sequences; b0 += THREADS) mine += units_at(b0 + (int)threadIdx.x);
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(~0u, mine, o);
  if (lane == 0) scratch.warp_units[warp] = mine;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += scratch.warp_units[w];
  total *= heads;
  const int shares = (int)min((int64_t)ctas, total);
  Walk walk;
  walk.left = 0, walk.unit = walk.units = 0, walk.b = walk.head = walk.block = 0;
  walk.s = Sequence{0, 0, 0}, walk.keys = Keys{0, 0};
  if (cta >= shares) return walk;
  const int64_t begin = total * cta / shares, end = total * (cta + 1) / shares;
  // the sequence that holds unit `begin`
  int64_t before = 0;
  for (int b0 = 0; b0 < p.at.sequences; b0 += THREADS) {
    const int64_t units = b0 ? units_at(b0 + (int)threadIdx.x) : first;
    int64_t upto = units;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t other = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += other;
    }
    __syncthreads();
    if (lane == 31) scratch.warp_units[warp] = upto;
    __syncthreads();
    int64_t chunk = 0, below = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) below += scratch.warp_units[w];
      chunk += scratch.warp_units[w];
    }
    const int64_t from = (before + below + upto - units) * heads;
    if (units && from <= begin && begin < from + units * heads)
      scratch.b = b0 + (int)threadIdx.x, scratch.rem = begin - from, scratch.per_head = units;
    before += chunk;
    if (before * heads > begin) break;
  }
  __syncthreads();
  walk.b = scratch.b;
  walk.head = (int)(scratch.rem / scratch.per_head);
  int64_t rem = scratch.rem % scratch.per_head;
  walk.s = sequence(p.at, p.cache.page_tokens, walk.b);
  walk.left = end - begin;
  // the block, 32 at a time
  const int blocks = blocks_of<ROWS>(p, walk.s);
  for (int i0 = 0; i0 < blocks; i0 += 32) {
    const int i = i0 + lane;
    const Keys k = keys_of<ROWS>(p, walk.s, min(i, blocks - 1));
    const int units = i < blocks ? units_of<UNIT>(k) : 0;
    int64_t upto = units;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t other = __shfl_up_sync(~0u, upto, o);
      if (lane >= o) upto += other;
    }
    const uint32_t beyond = __ballot_sync(~0u, upto > rem);
    if (beyond) {
      const int at = __ffs(beyond) - 1;
      walk.block = i0 + at;
      walk.unit = (int)(rem - __shfl_sync(~0u, upto - units, at));
      walk.units = __shfl_sync(~0u, units, at);
      walk.keys.low = __shfl_sync(~0u, k.low, at), walk.keys.high = __shfl_sync(~0u, k.high, at);
      break;
    }
    rem -= __shfl_sync(~0u, upto, 31);
  }
  return walk;
}

// Units of the share that are the present item's.
__device__ __forceinline__ int piece_units(const Walk& w) {
  return (int)min(w.left, (int64_t)(w.units - w.unit));
}

// On to the next item of the share, if there is one.
template <int ROWS, int UNIT>
__device__ __forceinline__ void next_piece(const AttentionParams& p, Walk& w) {
  w.left -= piece_units(w);
  if (w.left <= 0) return;
  w.unit = 0;
  if (++w.block == blocks_of<ROWS>(p, w.s)) {
    w.block = 0;
    if (++w.head == p.cache.heads) {
      w.head = 0;
      do {
        if (++w.b >= p.at.sequences) {  // (not reached: the shares end with the last unit)
          w.left = 0;
          return;
        }
        w.s = sequence(p.at, p.cache.page_tokens, w.b);
      } while (w.s.count == 0);
    }
  }
  w.keys = keys_of<ROWS>(p, w.s, w.block);
  w.units = units_of<UNIT>(w.keys);
}

// What keys row `r` (a new token and query head of the sequence) sees: [low, high).
__device__ __forceinline__ Keys seen_by(const AttentionParams& p, const Sequence& s, int r) {
  const int own = s.length - s.count + quotient(r, p.by_group);
  Keys k;
  k.high = p.causal ? min(s.length, max(own + 1, 0)) : s.length;
  k.low = p.window ? max(own + 1 - p.window, 0) : 0;
  return k;
}

}  // namespace ff
}  // namespace fwt
