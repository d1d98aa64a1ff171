// mma.cuh -- tensor-core plumbing of the experts' products: mbarriers across a
// pair of CTAs, tiled TMA copies, tcgen05 products and TMEM loads, as inline
// PTX, and the descriptors they take.
//
// A pair of CTAs (cta_group::2) works on one tile of M = 256: CTA 0 holds the
// operand rows and the accumulator lanes 0..127 of it in its own shared memory
// and TMEM, CTA 1 those of 128..255; of the N columns' operand each holds half.
// One thread of CTA 0 issues the products for both.
#pragma once

#include "moe_device.cuh"

#include <cuda.h>

namespace {

constexpr long long kMmaWaitCycles = 2000000000LL;  // ~1 s: a wait this long is an error

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The address of the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" :::
                   "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}

// ------------------------------------------------------------ mbarriers --
__device__ __forceinline__ void bar_init(uint32_t bar, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_init_done() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void bar_arrive_here(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Arrivals on a barrier of any CTA of the cluster (`bar`: a cluster address).
// Without publishing this thread's writes: a release at this scope waits for
// its global stores (4,000 cycles of every tile's epilogue, measured).  For
// arrivals after which others overwrite what this thread has finished reading.
__device__ __forceinline__ void bar_arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// (announcing a copy publishes no writes of this thread: a release here waits
// for nothing useful)
__device__ __forceinline__ void bar_arrive_tx(uint32_t bar, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar),
               "r"(bytes)
               : "memory");
}

// Whether a phase of a barrier of this CTA is complete (waits a little for it).
__device__ __forceinline__ bool bar_try(uint32_t bar, unsigned parity) {
  unsigned done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// The same without waiting.
__device__ __forceinline__ bool bar_test(uint32_t bar, unsigned parity) {
  unsigned done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// Waits for a phase of a barrier of this CTA; false after about a second.
__device__ __forceinline__ bool bar_wait(uint32_t bar, unsigned parity) {
  if (bar_try(bar, parity)) return true;
  const long long start = clock64();
  while (!bar_try(bar, parity))
    if (clock64() - start > kMmaWaitCycles) return false;
  return true;
}

// The same for what takes as long as a whole tile, which may be longer than that (a
// weights' gradient over hundreds of millions of rows): false after about a second
// in which `ring`, the barrier of one of the stages that the tile's operands go
// through, has not turned over either.  It turns over as often as the tile's
// contraction has blocks, so this wait ends too.
__device__ __forceinline__ bool bar_wait_tile(uint32_t bar, unsigned parity, uint32_t ring) {
  if (bar_try(bar, parity)) return true;
  bool seen = bar_test(ring, 0);
  long long start = clock64();
  while (!bar_try(bar, parity)) {
    const bool now = bar_test(ring, 0);
    if (now != seen) {
      seen = now;
      start = clock64();
    } else if (clock64() - start > kMmaWaitCycles) {
      return false;
    }
  }
  return true;
}

// ------------------------------------------------------------------ TMA --
// One box of a tiled tensor to this CTA's shared memory; its bytes are counted
// on `bar`, which may be in the other CTA of the pair.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load5(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                          int u, int v, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(bar)
      : "memory");
}

// -------------------------------------------------------------- tcgen05 --
__device__ __forceinline__ void tmem_alloc(uint32_t to, unsigned columns) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t tmem, unsigned columns) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
}

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add,
                                    bool issue) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((unsigned)add), "r"((unsigned)issue)
      : "memory");
}

// Arrives on the barrier at this offset in both CTAs once the products issued
// so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar, bool issue) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;\n\t}" ::"r"(bar),
      "h"((unsigned short)3), "r"((unsigned)issue)
      : "memory");
}

__device__ __forceinline__ void fence_before_sync() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after_sync() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 16 lanes x 32 columns of 32 bits: register 4 i + 2 h + c of lane l is lane
// l / 4 + 8 h, column 8 i + 2 (l % 4) + c.
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}

__device__ __forceinline__ void tmem_load_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Shared-memory operand with 128-byte swizzle.  K-major rows of 64 elements:
// eight rows are 1024 bytes (the stride offset).  MN-major: a box of 64
// elements x 64 steps of K, eight steps 1024 bytes (the stride offset), the
// next 64 elements one box (8192 bytes, the leading offset) further.
__device__ __forceinline__ uint64_t operand(uint32_t addr, unsigned leading) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3ffff) >> 4);
  d |= (uint64_t)(leading >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version of this architecture
  d |= (uint64_t)2 << 61;  // 128-byte swizzle
  return d;
}

// 16-bit operands of one type, 32-bit sums.
__device__ __forceinline__ uint32_t product(bool bf16, bool a_mn, bool b_mn, int m, int n) {
  uint32_t d = 0;
  d |= 1u << 4;                       // accumulate in f32
  d |= (bf16 ? 1u : 0u) << 7;         // A
  d |= (bf16 ? 1u : 0u) << 10;        // B
  d |= (a_mn ? 1u : 0u) << 15;
  d |= (b_mn ? 1u : 0u) << 16;
  d |= (uint32_t)(n >> 3) << 17;
  d |= (uint32_t)(m >> 4) << 24;
  return d;
}

// 8 x 8 matrices of 16-bit elements between registers (lane l: row l / 4,
// columns 2 (l % 4) and the next) and shared-memory rows of 16 bytes, the row
// addresses given by lanes 8 m + row; transposed: memory rows are columns.
__device__ __forceinline__ void put4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x),
               "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void put4_t(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a),
               "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void get4_t(uint32_t a, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(a)
               : "memory");
}

}  // namespace
