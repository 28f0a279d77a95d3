// How attention over the cache is shared out among CTAs.
//
// An item is a block of ROWS rows (new tokens x query heads of one key head) of a sequence with one
// key head; its keys, from the first that one of its rows sees, are cut into units of UNIT tokens, at
// least one; what an item costs besides its keys counts as EXTRA units before them.  All units of the call, in the order of sequences, key heads, blocks, are dealt out in
// equal consecutive shares, so that no worker's time depends on how lengths are spread; a share
// begins and ends inside an item as it may.  Workers are CTAs, or warps where an item has few rows.
// The host does not know the lengths: every CTA adds them up for itself.
//
// What worker i has done of an item that is not all its own goes to the workspace: part 2 i is of
// the item that its share begins in the middle of, part 2 i + 1 of the one that it ends in the
// middle of.  notes[i] says which there are, and launch_attention_join() puts them together in the
// order of the keys, so that results depend on nothing but the arguments.
#pragma once

#include <cstdint>

#include "cache.cuh"

namespace fwt {
namespace ff {

// notes[2 i]: x flags, and of part 2 i + 1 the last worker with a part of its item, the key head and
// the block; notes[2 i + 1]: its sequence's first packed row and number of rows.
constexpr int kNoteTail = 1;  // part 2 i + 1 is there

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
  k.low = p.window ? min(max(max(own + first + 1, 0) - p.window, 0), k.high) & ~15 : 0;  // (of 31 bits each)
  return k;
}

template <int UNIT>
__device__ __forceinline__ int units_of(const Keys& k) {
  return max(1, (k.high - k.low + UNIT - 1) / UNIT);
}

// The same with what stands for the item itself.
template <int UNIT, int EXTRA>
__device__ __forceinline__ int cost_of(const Keys& k) {
  return EXTRA + units_of<UNIT>(k);
}

// Units of one key head of the sequences of a warp's lanes (sequence b in each; count 0: none).
// (Loops here are not unrolled, and divisions few: code that runs once comes from memory, and with 150 and
// 320 KB of it the kernels took twice as long.)
template <int ROWS, int UNIT, int EXTRA>
__device__ __forceinline__ int64_t units_of_sequence(const AttentionParams& p, const Sequence& s, int lane) {
  constexpr int kAlone = 4;  // blocks that a lane counts by itself
  const int blocks = blocks_of<ROWS>(p, s);
  int64_t units = 0;
  if (blocks <= kAlone)
    for (int i = 0; i < blocks; ++i) units += cost_of<UNIT, EXTRA>(keys_of<ROWS>(p, s, i));
  for (uint32_t many = __ballot_sync(~0u, blocks > kAlone); many; many &= many - 1) {
    const int from = __ffs(many) - 1;
    Sequence t;
    t.row = 0;
    t.count = __shfl_sync(~0u, s.count, from), t.length = __shfl_sync(~0u, s.length, from);
    const int n = __shfl_sync(~0u, blocks, from);
    int64_t sum = 0;
    for (int i = lane; i < n; i += 32) sum += cost_of<UNIT, EXTRA>(keys_of<ROWS>(p, t, i));
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
  int unit, units;  // of the item's keys: the next one, and all
  int skip;         // units before them
  int64_t left;     // units of the share, `skip` among them; more than that, or 0 at its end
  int64_t each;     // of every share, and one more of the first `more`
  int more;
};

constexpr int kGroups = 256;  // that the sequences are added up in
struct PlanScratch {
  int64_t units[kGroups];  // of one key head
};

// The share of worker `worker` of `workers`, at least LEAST units while there are enough; every thread of
// the CTA calls it, with a worker of its warp's.  left = 0: there is none.
template <int ROWS, int UNIT, int EXTRA, int LEAST, int THREADS>
__device__ __forceinline__ Walk find_share(const AttentionParams& p, int worker, int workers, PlanScratch& scratch) {
  const int lane = threadIdx.x & 31, heads = p.cache.heads;
  const int span = (p.at.sequences + 32 * kGroups - 1) / (32 * kGroups) * 32;  // sequences of a group
  const int groups = (p.at.sequences + span - 1) / span;
  Sequence s{0, 0, 0};
  const auto units_at = [&](int b) {
    s.count = 0;
    if (b < p.at.sequences) s = sequence(p.at, p.cache.page_tokens, b);
    return units_of_sequence<ROWS, UNIT, EXTRA>(p, s, lane);
  };
  // (32 values of a warp added up from the first on)
  const auto upto = [&](int64_t v) {
#pragma unroll 1
    for (int o = 1; o < 32; o *= 2) {
      const int64_t other = __shfl_up_sync(~0u, v, o);
      if (lane >= o) v += other;
    }
    return v;
  };
#pragma unroll 1
  for (int i = threadIdx.x >> 5; i < groups; i += THREADS / 32) {
    int64_t sum = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < span; b0 += 32) sum += units_at(i * span + b0 + lane);
    sum = upto(sum);
    if (lane == 31) scratch.units[i] = sum;
  }
  __syncthreads();
  int64_t total = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < groups; i0 += 32)
    total += __shfl_sync(~0u, upto(i0 + lane < groups ? scratch.units[i0 + lane] : 0), 31);
  total *= heads;
  Walk walk;
  walk.left = walk.each = 0, walk.more = 0, walk.unit = walk.units = walk.skip = 0, walk.b = walk.head = walk.block = 0;
  walk.s = Sequence{0, 0, 0}, walk.keys = Keys{0, 0};
  const int shares = (int)min((int64_t)workers, (total + LEAST - 1) / LEAST);
  if (worker >= shares) return walk;
  const int64_t each = total < 0x7fffffff ? (int)total / shares : total / shares;
  const int more = (int)(total - each * shares);
  walk.each = each, walk.more = more;
  int64_t rem = each * worker + min(worker, more);
  walk.left = each + (worker < more);
  // its group, its sequence, its head, its block: each time 32 at once, the first beyond `rem`
  const auto find = [&](int count, int64_t times, const auto& units_of_one) {
    int at = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < count; i0 += 32) {
      const int64_t units = units_of_one(i0 + lane) * times, sum = upto(units);
      const uint32_t beyond = __ballot_sync(~0u, sum > rem);
      const int hit = beyond ? __ffs(beyond) - 1 : 31;
      at = i0 + hit;
      rem -= __shfl_sync(~0u, beyond ? sum - units : sum, hit);
      if (beyond) break;
    }
    return at;
  };
  const int group = groups == 1 ? 0 : find(groups, heads, [&](int i) { return i < groups ? scratch.units[i] : 0; });
  walk.b = group * span + find(span, heads, [&](int i) { return units_at(group * span + i); });
  walk.s = sequence(p.at, p.cache.page_tokens, walk.b);
  const int blocks = blocks_of<ROWS>(p, walk.s);
  const int64_t per_head = __shfl_sync(~0u, units_at(walk.b + lane), 0);
  walk.head = rem < 0x7fffffff && per_head < 0x7fffffff ? (int)rem / (int)per_head : (int)(rem / per_head);
  rem -= walk.head * per_head;
  walk.block = find(blocks, 1, [&](int i) {
    return (int64_t)(i < blocks ? cost_of<UNIT, EXTRA>(keys_of<ROWS>(p, walk.s, i)) : 0);
  });
  walk.skip = max(EXTRA - (int)rem, 0), walk.unit = max((int)rem - EXTRA, 0);
  if (walk.left <= walk.skip) walk.left = 0;  // (the next worker has the item)
  walk.keys = keys_of<ROWS>(p, walk.s, walk.block);
  walk.units = units_of<UNIT>(walk.keys);
  return walk;
}

// Units of the present item's keys in the share.
__device__ __forceinline__ int piece_units(const Walk& w) {
  return (int)min(w.left - w.skip, (int64_t)(w.units - w.unit));
}

// On to the next item of the share, if there is one.
template <int ROWS, int UNIT, int EXTRA>
__device__ __forceinline__ void next_piece(const AttentionParams& p, Walk& w) {
  w.left -= w.skip + piece_units(w);
  w.skip = EXTRA;
  if (w.left <= EXTRA) {
    w.left = 0;
    return;
  }
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

// The notes on the share's last piece, an item that begins in it and ends in another: `walk` stands there.
__device__ __forceinline__ void note_tail(const Walk& w, int worker, int4* notes) {
  // the item's last unit, counted from the first of all
  const int64_t end = w.each * (worker + 1) + min(worker + 1, w.more);
  const int64_t unit = end + (w.units - w.unit - piece_units(w)) - 1, longer = (w.each + 1) * w.more;
  const int64_t last = unit < longer ? unit / (w.each + 1) : w.more + (unit - longer) / w.each;
  notes[2 * worker] = make_int4(kNoteTail, (int)last, w.head, w.block);
  notes[2 * worker + 1] = make_int4(w.s.row, w.s.count, 0, 0);
}

// What keys row `r` (a new token and query head of the sequence) sees: [low, high).
__device__ __forceinline__ Keys seen_by(const AttentionParams& p, const Sequence& s, int r) {
  const int own = s.length - s.count + quotient(r, p.by_group);
  Keys k;
  k.high = p.causal ? min(s.length, max(own + 1, 0)) : s.length;
  k.low = p.window ? max(max(own + 1, 0) - p.window, 0) : 0;
  return k;
}

}  // namespace ff
}  // namespace fwt
