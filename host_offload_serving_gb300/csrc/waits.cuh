// waits.cuh -- barriers in shared memory, with waits that end.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {  // suspended for up to 100 us
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, 100000;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
constexpr long long kWaitCycles = 1ll << 30;  // half a second
// Waits have a limit (against microseconds in use).  One that runs out sets
// *fail, after which no wait of the CTA waits any more: every loop still makes
// its turns, so barriers stay matched, TMEM is freed and the kernel ends, with
// HISPARSE_ERR_WAIT in the status and NaN in its outputs.  They return whether the phase came:
// the warps that copy rows stop where it did not, as the addresses would be those of no row.
__device__ __noinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, volatile int *fail) {
  const long long start = clock64();
  while (!*fail) {
    if (bar_try(bar, parity)) return true;
    if (clock64() - start > kWaitCycles) *fail = 1;
  }
  return false;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *fail) {
  return bar_try(bar, parity) || bar_wait_long(bar, parity, fail);
}
