// pipe.cuh -- pieces shared by linear.cu and logprobs.cu: bounded mbarrier waits
// that sleep in the barrier unit, single-lane issue from a converged warp, paired
// fp32 arithmetic, and bf16 pairs and byte shifts of 16-byte pieces.  (The
// self-test of the waits in lmhead.cu runs them out.)
#pragma once

#include "tcgen05.cuh"

namespace sga {
namespace {

// Bounded wait (as mbar_wait) that sleeps in the barrier unit (try_wait with a
// time hint) between looks at the clock and the abort flag.
__device__ __forceinline__ bool pipe_wait(uint32_t bar, uint32_t parity,
                                          const volatile int *abort_flag,
                                          unsigned long long limit_ns = kWaitLimitNs) {
  if (mbar_try_wait(bar, parity)) return true;
  unsigned long long t0 = 0;
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(100000u)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
    const unsigned long long t = global_timer_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > limit_ns) return false;
  }
}

// The same, agreed on by the whole (converged) warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity,
                                          const volatile int *abort_flag,
                                          unsigned long long limit_ns = kWaitLimitNs) {
  return __all_sync(0xffffffffu, pipe_wait(bar, parity, abort_flag, limit_ns)) != 0;
}

// True in one lane of a converged warp.  Producer and MMA warps run their
// loops with all lanes and elect one around each issue, so that the operands
// of TMA and MMA instructions stay in uniform registers: issued from a branch
// on the lane number, the two copies and four MMAs of a K block took about 650
// cycles of their warps, more than the tensor core needs for them.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// The abort flag as the whole warp sees it.
__device__ __forceinline__ bool aborted(const volatile int *abort_flag) {
  return __any_sync(0xffffffffu, *abort_flag != 0) != 0;
}

__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ void raise_abort(int *flag, uint32_t *err) {
  *reinterpret_cast<volatile int *>(flag) = 1;
  atomicOr(err, SGA_DEVERR_TIMEOUT);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack_f32(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack_f32(uint64_t v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Two values rounded to bf16, lo in the low half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Bytes s .. s + 15 (s even, 0 .. 16) of two 16-byte pieces that follow each other.
__device__ __forceinline__ uint4 bytes_of(const uint4 a, const uint4 b, int s) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = (s & 8) ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = (s & 4) ? w[i + 1] : w[i];
  uint4 r;
  r.x = __funnelshift_r(w[0], w[1], (s & 2) * 8);
  r.y = __funnelshift_r(w[1], w[2], (s & 2) * 8);
  r.z = __funnelshift_r(w[2], w[3], (s & 2) * 8);
  r.w = __funnelshift_r(w[3], w[4], (s & 2) * 8);
  return (s & 16) ? b : r;
}

// Untiled copy of global memory into shared memory (16-byte aligned, size a
// multiple of 16), counted on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

}  // namespace
}  // namespace sga
