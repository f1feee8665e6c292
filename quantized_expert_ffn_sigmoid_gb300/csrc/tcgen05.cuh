// Inline-PTX wrappers of the tcgen05 kernels (many-position and MX4 expert
// paths): matrix descriptors, tensor-memory loads and stores, commits, small
// asynchronous copies and the bounded pipeline waits.
#pragma once
#include "colimoe_internal.cuh"

namespace colimoe {

constexpr uint32_t PF_WAIT_HINT_NS = 100000;  // suspend-time hint of one wait (100 us)
constexpr uint32_t PF_WAIT_TRIES = 10000;      // hinted waits before a wait gives up (about 1 s)

// Shared-memory matrix descriptor of a K-major operand in the 128-byte
// swizzled layout: 8-row atoms 1024 bytes apart (stride byte offset), the
// leading byte offset unused (1), descriptor version 1, layout type 2 (128-byte
// swizzle).  A K16 slice at byte offset 32 k inside the 128-byte span is
// addressed by adding that offset to the start address (the swizzle is applied
// to the address bits, so the atom must be 1024-byte aligned).
__device__ __forceinline__ uint64_t umma_desc_sw128(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 consecutive 32-bit columns of this warp's 32 TMEM lanes (no wait)
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 16 consecutive 32-bit columns of this warp's 32 TMEM lanes from registers
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// try_wait with a suspend-time hint: the thread sleeps in hardware until the
// phase completes (or the hint expires) instead of polling, so twenty warps
// waiting on their barriers do not flood the shared-memory pipe that the
// MMA issuer's own waits and the TMA writes go through.
__device__ __forceinline__ bool mbar_try_wait_sleep(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "r"(PF_WAIT_HINT_NS) : "memory");
  return ok != 0;
}

// Bounded wait (PF_WAIT_TRIES hinted waits, about a second in all) that
// gives up at once after any wait of the CTA has expired (the shared abort
// flag, read only when a wait fails), so that a broken pipeline drains in a
// fraction of a second instead of expiring every later wait in turn.
__device__ __forceinline__ bool pf_wait(uint64_t* bar, uint32_t parity, uint32_t* status, volatile int* abort) {
  for (uint32_t i = 0; i < PF_WAIT_TRIES; ++i) {
    if (mbar_try_wait_sleep(bar, parity)) return true;
    if (*abort) return false;
  }
  *abort = 1;
  atomicOr(status, COLI_STATUS_TIMEOUT);
  return false;
}

// The same bounded wait polling without suspending (mbarrier.test_wait, ~2^26
// polls, about half a second), for the two roles on the pipeline's critical
// path, the MMA issuer and the converters: a suspended thread's wake-up after
// the phase completes costs more than their polls (measured: 7.37 -> 6.84 ms
// at 2048 positions), while the eight epilogue warps keep the hinted wait.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool pf_wait_poll(uint64_t* bar, uint32_t parity, uint32_t* status, volatile int* abort) {
  for (uint32_t i = 0; i < (1u << 26); ++i) {
    if (mbar_test_wait(bar, parity)) return true;
    if ((i & 1023u) == 1023u && *abort) return false;
  }
  *abort = 1;
  atomicOr(status, COLI_STATUS_TIMEOUT);
  return false;
}

}  // namespace colimoe
