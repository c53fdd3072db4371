// kvcs_tcgen.cuh -- thin inline-PTX wrappers of the fifth-generation tensor
// cores (sm_103a): tensor memory, descriptors, products, tiled TMA loads, and
// packed pairs of floats.
#pragma once

#include <cuda.h>

#include "kvcs_ptx.cuh"

namespace kvcs {
namespace tc {

using ptx::u32;
using ptx::u64;

__device__ __forceinline__ void tmem_alloc(u32 smem_slot, u32 columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_slot),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(u32 addr, u32 columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns)
               : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Writes to shared memory become visible to the tensor cores and TMA.
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect() {
  u32 r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Arrives on `bar` once every product this thread issued before is done.
__device__ __forceinline__ void commit(u32 bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

// Shared-memory matrix descriptors, 128-byte swizzle.  K-major operands: rows
// of 128 bytes, 8-row groups `group` bytes apart (`lbo` unused).  MN-major
// operands: 64 contiguous elements along M or N, blocks of 64 `lbo` bytes
// apart, 8-deep groups along K `group` apart.  Moving the operand by n bytes
// adds n / 16 to the low word (the products' issue rate hangs on how little
// is computed between two of them).
__host__ __device__ constexpr u32 desc_high(u32 group) { return group >> 4 | 1u << 14 | 2u << 29; }
__device__ __forceinline__ u32 desc_low(u32 addr, u32 lbo) {
  return (addr & 0x3ffffu) >> 4 | (lbo >> 4) << 16;
}
template <u32 kGroup>
__device__ __forceinline__ u64 desc(u32 low) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(low), "r"(desc_high(kGroup)));
  return r;
}

// Instruction descriptor of kind::f16 with 32-bit accumulators.
__host__ __device__ constexpr u32 instr_desc(bool bf16, int m, int n, bool b_mn_major) {
  return 1u << 4 | (bf16 ? 1u : 0u) << 7 | (bf16 ? 1u : 0u) << 10 | (b_mn_major ? 1u : 0u) << 16 |
         static_cast<u32>(n >> 3) << 17 | static_cast<u32>(m >> 4) << 24;
}

// D (tensor memory) = A (shared) B (shared) [+ D]
__device__ __forceinline__ void mma_ss(u32 d, u64 a, u64 b, u32 idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
      : "memory");
}
// D = A (tensor memory) B (shared) [+ D]
__device__ __forceinline__ void mma_ts(u32 d, u32 a, u64 b, u32 idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
      : "memory");
}

#define KVCS_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), \
                      "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define KVCS_I8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), \
                      "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])

// As ptx::mbar_wait_bounded, with a look at the global timer (a read of about a
// microsecond) after every 1024 probes only: the waits of a product pipeline
// are shorter than that, and on its critical path.
// The first probe stands apart: one that succeeds costs about 15 cycles, the
// loop's bookkeeping about 100 more.  A warp calls it converged and leaves it
// with one answer, so that none of its lanes goes on alone: lanes give up by a
// vote of those that are still there, after a last probe that goes for all of
// them, and a phase that a lane has seen before is there at that probe.  (Votes
// on every wait cost 3 to 9% of a product pipeline's time, in the loop 5%.)
// The limit lies below 2^32 ns: the timer's low word is enough.
__device__ __forceinline__ bool wait(u32 bar, u32 parity, u64 limit_ns) {
  if (__builtin_expect(ptx::mbar_try_wait(bar, parity), 1)) return true;
  u32 t0 = 0;
#pragma unroll 1
  for (u32 i = 1; i < (1u << 28); ++i) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((i & 1023u) == 0) {
      const u32 now = ptx::globaltimer_low();
      if (i == 1024) t0 = now;
      const u32 late = __activemask();
      if (__any_sync(late, now - t0 > static_cast<u32>(limit_ns))) {
        const bool there = __any_sync(late, ptx::mbar_try_wait(bar, parity));
        __syncwarp(late);   // (orders what follows for the lanes that did not see it themselves)
        return there;
      }
    }
  }
  return false;
}
// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void ld32(u32 addr, u32 *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : KVCS_R8(v, 0), KVCS_R8(v, 8), KVCS_R8(v, 16), KVCS_R8(v, 24)
      : "r"(addr));
}
__device__ __forceinline__ void st32(u32 addr, const u32 *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::KVCS_I8(v, 0),
      KVCS_I8(v, 8), KVCS_I8(v, 16), KVCS_I8(v, 24), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void ld16(u32 addr, u32 *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : KVCS_R8(v, 0), KVCS_R8(v, 8)
      : "r"(addr));
}
__device__ __forceinline__ void st16(u32 addr, const u32 *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::KVCS_I8(v, 0),
      KVCS_I8(v, 8), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// One box of a 5-dimensional tensor into shared memory.
__device__ __forceinline__ void tma_load(u32 dst, const CUtensorMap *map, int c0, int c1, int c2,
                                         int c3, int c4, u32 bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// Packed pairs of floats.
__device__ __forceinline__ u64 pair(float a, float b) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(u64 v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

}  // namespace tc
}  // namespace kvcs
