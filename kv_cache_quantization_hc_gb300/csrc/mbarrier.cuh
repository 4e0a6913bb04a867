// mbarriers of a CTA's own, with waits that end: after two seconds (or what a
// kernel gives for its longest), or once another of the CTA's waits has run out.
#pragma once

#include <stdint.h>

namespace hc {
namespace {

__device__ __forceinline__ uint32_t mbar_addr(const void* b) { return static_cast<uint32_t>(__cvta_generic_to_shared(b)); }
__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(mbar_addr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(mbar_addr(b)) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t a, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\nselp.u32 %0, 1, 0, p;\n}"
      : "=r"(done) : "r"(a), "r"(parity) : "memory");
  return done != 0;
}
// Waits for the phase of this parity to end; false when the wait ran out
// (after `limit` ns), here or elsewhere in the CTA.
constexpr uint64_t kWaitLimit = 2000000000;
__device__ __forceinline__ bool mbar_wait_timed(uint32_t a, uint32_t parity, int32_t* dead, uint64_t limit = kWaitLimit) {
  uint64_t start, now;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(start));
  do {
    if (mbar_try(a, parity)) return true;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
  } while (now - start < limit && !*static_cast<volatile int32_t*>(dead));
  *static_cast<volatile int32_t*>(dead) = 1;
  return false;
}
__device__ __noinline__ bool mbar_wait_long(uint32_t a, uint32_t parity, int32_t* dead) {
  return mbar_wait_timed(a, parity, dead);
}
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity, int32_t* dead) {
  const uint32_t a = mbar_addr(b);
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (mbar_try(a, parity)) return true;
  return mbar_wait_long(a, parity, dead);
}
// The same without a call, for kernels that share registers out anew
// (setmaxnreg), in which there may be none.
__device__ __forceinline__ bool mbar_wait_inline(uint64_t* b, uint32_t parity, int32_t* dead, uint64_t limit = kWaitLimit) {
  const uint32_t a = mbar_addr(b);
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (mbar_try(a, parity)) return true;
  return mbar_wait_timed(a, parity, dead, limit);
}

}  // namespace
}  // namespace hc
