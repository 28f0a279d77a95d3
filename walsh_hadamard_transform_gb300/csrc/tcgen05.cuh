// Fifth-generation tensor-core helpers (sm_103a): tensor memory, matrix products of
// shared-memory tiles, their barriers, and the bounded waits around them.
//
// Operand tiles lie in shared memory as TMA writes them with 128-byte swizzle, in rows of
// 128 bytes and atoms of 8 rows (1024 bytes):
//   K-major   a row is one line of the operand, 128 bytes along the contraction;
//   MN-major  a row is one index of the contraction, 64 16-bit lines of the operand; a
//             tile of more than 64 lines is several such chunks, one after the other.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "tma.cuh"

namespace fwt {
namespace ff {

constexpr uint32_t kSwizzleAtom = 1024;  // bytes, 8 rows

// True in one thread of the (whole) warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The shared::cluster address of `addr` (shared::cta) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Says that reads of tensor memory are done (after tmem_fence_before()); orders no other
// memory, as a release at cluster scope would (measured: a thousand clocks).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr, bool one = true) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(cluster_addr),
      "r"((uint32_t)one)
      : "memory");
}

__device__ __forceinline__ float load_cluster(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// (`one`: only the threads for which it is true arrive, without a branch.)
__device__ __forceinline__ void mbar_arrive(uint64_t* bar, bool one = true) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"((uint32_t)one)
      : "memory");
}

// A box of `map` at (x, y) into this CTA's shared memory; its bytes are counted by `bar`, a
// shared::cluster address: this CTA's barrier, or for CG = 2 the barrier of the pair's first.
template <int CG>
__device__ __forceinline__ void tma_load_tile(uint32_t dst, const CUtensorMap* map, int x, int y,
                                              uint32_t bar) {
  if constexpr (CG == 1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  }
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- tensor memory -------------------------------------------------------------------

// One whole warp each; `columns` is a power of two from 32 to 512.
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t columns) {
  if constexpr (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(dst)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(dst)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}

__device__ __forceinline__ void tmem_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_loads() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 32 consecutive columns of the warp's 32 lanes, one lane a thread.  The values are there
// after tmem_wait_loads().
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11,"
      " %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29,"
      " %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr));
}

// The same for stores of 16 columns, which are done after tmem_wait_stores().
__device__ __forceinline__ void tmem_wait_stores() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11,"
      " %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// ---- matrix products -----------------------------------------------------------------

// Shared-memory operand descriptor, 128-byte swizzle.  K-major: atoms of 8 lines 1024 bytes
// apart.  MN-major: atoms of 8 contraction indices 1024 bytes apart, chunks of 64 lines
// `chunk_bytes` apart.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t chunk_bytes) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(chunk_bytes >> 4) << 16) |
         ((uint64_t)(kSwizzleAtom >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: fp32 accumulator, operand formats a and b (16-bit: 0 f16, 1 bf16;
// 8-bit: 0 e4m3), MN-major flags, tile of m x n.
__host__ __device__ constexpr uint32_t instruction(uint32_t format, bool a_mn, bool b_mn, uint32_t m, uint32_t n) {
  return (1u << 4) | (format << 7) | (format << 10) | ((uint32_t)a_mn << 15) |
         ((uint32_t)b_mn << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// D (tensor memory) = A B^T, plus D where `add`; one thread.  BYTES: of an operand element.
template <int CG, int BYTES>
__device__ __forceinline__ void mma_tile(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t add) {
  if constexpr (CG == 1 && BYTES == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  else if constexpr (CG == 2 && BYTES == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  else if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

// The same with A in tensor memory, two 16-bit elements a column, a line a lane.
__device__ __forceinline__ void mma_tile_from_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                                   uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}

// Writes of this thread to shared memory, seen by products issued after what it signals next.
__device__ __forceinline__ void fence_to_products() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// `bar` (at the same place in each CTA of the pair) gets one arrival when the products
// issued so far by this thread are done.
template <int CG>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if constexpr (CG == 1)
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_u32(bar))
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// ---- waits ---------------------------------------------------------------------------

// Whether the phase is complete, without waiting (try_wait may suspend the thread for a while).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// The global timer in steps of 2^20 ns, about a millisecond.
__device__ __forceinline__ uint32_t global_ms() { return (uint32_t)(global_ns() >> 20); }

// A wait of a whole warp: at most about a second in which nothing comes forward, and over at once
// when another role of the CTA has given up.  false, in every lane: leave the role's loop.
// `seen`: what an earlier mbar_test of the same phase said (asked ahead, its answer is there
// by now).  `progress`: what the role waited for counts its steps with, where one wait spans many
// of them.  A device that other processes have had for a while in between has its clock go on
// without the warp: no gap between two looks at it counts as more than a tenth of a second.
template <typename... Progress>
__device__ __forceinline__ bool wait_or_leave(uint64_t* bar, uint32_t parity, volatile int* gave_up,
                                              bool seen = false, Progress... progress) {
  bool done = seen || mbar_poll(bar, parity);
  for (int i = 0; i < 32 && !done; ++i) done = mbar_poll(bar, parity);
  if (!done) {  // the timer is slow to read: not before it is needed
    uint32_t last = global_ms(), spent = 0, steps = (0u + ... + *progress);
    for (uint32_t i = 1; i < (1u << 28); ++i) {
      done = mbar_poll(bar, parity);
      if (done) break;
      if ((i & 63u) == 0) {
        const uint32_t now = global_ms();
        spent += min(now - last, 100u), last = now;
        if constexpr (sizeof...(Progress) > 0) {
          const uint32_t at = (0u + ... + *progress);
          if (at != steps) steps = at, spent = 0, i = 0;
        }
        if (*gave_up || spent > 1000u) break;
      }
    }
    if (!done && !*gave_up) {
      atomicOr(&g_device_error, kErrTmaTimeout);
      *gave_up = 1;
    }
  }
  return __all_sync(~0u, done);
}

// After a wait that gave up: time for copies and products in flight to end before the
// shared memory and the tensor memory are given back (they take microseconds).
__device__ __forceinline__ void drain() {
  const unsigned long long t0 = global_ns();
  for (int i = 0; i < (1 << 20) && global_ns() - t0 < 5000000ull; ++i) __nanosleep(1000);
}

}  // namespace ff
}  // namespace fwt
