// attn_pipe.cuh -- pieces of a warp-specialised attention pipeline: votes over some of a
// CTA's warps, asynchronous copies, tcgen05.mma issued from a converged warp, registers moved
// between warpgroups and bounded waits that need no function call.
#pragma once

#include "common.cuh"

namespace dsv4sa {
namespace attn {

__device__ __forceinline__ bool any_of(bool v, uint32_t id, uint32_t n) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(v ? 1u : 0u), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

// 16-byte asynchronous copy into shared memory; bytes = 0 writes zeros.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// A contiguous range into L2 (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// tcgen05.mma and its commit by one elected lane of a converged warp: the
// operands then stay in uniform registers (60 cycles an MMA against 68 to 80 from
// a single-lane branch).
// The low words of the descriptors (address and leading offset) vary, the high words
// are the same for every operand here.
__device__ __forceinline__ void mma_f16_elect(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "mov.b64 a, {%1, %3};\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
template <int kRegs>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

// mbar_wait without a function call: a kernel that moves registers between its
// warpgroups cannot make one (the register allocation fails).
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity) {
  if (mbar_test_parity(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  for (uint32_t it = 1;; ++it) {
    if (mbar_test_parity(bar, parity)) return true;
    if ((it & 63u) == 0u && global_timer_ns() - t0 > kWaitLimitNs) {
      raise_error(kErrTimeout);
      return false;
    }
  }
}
// The whole (converged) warp waits and stays converged: every branch is on a vote.
// (Were one lane to wait for the others, the warp would go on in two parts, and each
// elect.sync after it would have to bring them together: 280 cycles an MMA.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_test_parity(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, mbar_test_parity(bar, parity))) return true;
    if ((it & 63u) == 0u && __any_sync(0xffffffffu, global_timer_ns() - t0 > kWaitLimitNs)) {
      raise_error(kErrTimeout);
      return false;
    }
  }
}

}  // namespace attn
}  // namespace dsv4sa
