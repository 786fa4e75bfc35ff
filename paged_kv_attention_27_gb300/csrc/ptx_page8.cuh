// PTX of the kernels over a page-scaled FP8 cache: sleeping mbarrier waits,
// kind::f8f6f4 MMAs with e4m3 operands, and 4-byte asynchronous copies.
#pragma once
#include "ptx.cuh"

namespace fi {
namespace dev {

// mbar_wait_bounded with a suspend-time hint of 20 us: the thread sleeps until the
// phase completes instead of polling, which leaves the issue slots to the
// warps beside it. The abort flag and the limit are looked at between sleeps.
__device__ __forceinline__ bool mbar_sleep_bounded(uint32_t bar, uint32_t parity,
                                                   uint64_t limit_ns,
                                                   const volatile int* abort) {
  auto attempt = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
  };
  if (attempt()) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (attempt()) return true;
    if (abort && *abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) return false;
  }
}

__device__ __forceinline__ bool mbar_sleep_warp(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                                const volatile int* abort) {
  const bool ok = mbar_sleep_bounded(bar, parity, limit_ns, abort);
  return __all_sync(0xffffffffu, ok);
}

// The descriptor of sdesc_sw128 for any swizzle: `mode` is 0 (none), 2 (128-byte), 4
// (64-byte) or 6 (32-byte). 64-byte swizzle: rows of 64 B, 8-row atoms of
// 512 B; MN-major without swizzle: 16 B along MN per row of K, 8 rows
// adjacent, `lbo` between 8-row groups along K and `sbo` between 16-byte
// groups along MN.
__device__ __forceinline__ uint64_t sdesc_swz(uint32_t smem_addr, uint32_t lbo, uint32_t sbo,
                                              uint32_t mode) {
  uint64_t d = 0;
  d |= uint64_t((smem_addr >> 4) & 0x3FFFu);
  d |= uint64_t((lbo >> 4) & 0x3FFFu) << 16;
  d |= uint64_t((sbo >> 4) & 0x3FFFu) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(mode) << 61;
  return d;
}

// D[tmem] (+)= A[smem] * B[smem], kind::f8f6f4 (here e4m3 inputs, 32 elements
// of K per instruction, fp32 accumulate).
__device__ __forceinline__ void tc_mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4 with e4m3 A and B, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) |
         (uint32_t(M >> 4) << 24);
}

// Programmatic dependent launch: the kernel behind this one may start (if its
// launch says so) once every block has called pdl_trigger; what it reads of
// earlier kernels' results it reads after pdl_wait, which returns when those
// have completed (at once in an ordinary launch).
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Four bytes from global to shared memory, completing asynchronously; the
// calling thread's copies so far arrive on an mbarrier when they have landed.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace dev
}  // namespace fi
