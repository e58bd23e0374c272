// mbar_poll.cuh — waits that poll an mbarrier among other things, or without a timer in
// their first tries (the absorbed latent kernel).
#pragma once

#include "pa_device.cuh"

namespace pa {

// mbar_try_wait's question without the wait that it may spend in hardware: for
// polling several barriers in turn.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, unsigned parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounds a wait: asked after every kTries failed tries, it says when to give up, which
// is kWaitLimitNs after the first time or, with an `abort` flag, as soon as that is set
// (another role has given up and raised the error). Reading the timer only then keeps it
// out of the waits of a GPU at work: a cold line of instructions costs microseconds
// once all SMs stream, and a timer's loop is one that every first wait would fetch. (A
// loop of tries inside a loop of these, not one that counts: up to 1.5 %.)
constexpr unsigned kTries = 4096;
class WaitLimit {
 public:
  __device__ __forceinline__ bool over(const int* abort, unsigned* err) {
    since_ = check(since_, abort, err);
    return since_ == 0;
  }

 private:
  // The time of the first check (low half of the timer, odd), or 0: over.
  __device__ __noinline__ static uint32_t check(uint32_t since, const int* abort, unsigned* err) {
    if (abort && *static_cast<const volatile int*>(abort) != 0) return 0;
    const uint32_t now = (uint32_t)global_timer_ns() | 1u;
    if (since == 0) return now;
    if (now - since <= (uint32_t)kWaitLimitNs) return since;
    raise_error(err, kErrTimeout);
    return 0;
  }
  uint32_t since_ = 0;
};
static_assert(kWaitLimitNs < 0xFFFFFFFFull - 1000000000ull, "the limit has to fit 32 bits of time");

// pa::mbar_wait with WaitLimit's bound: a try suspends the thread for about kTryNs at
// most, so the limit is passed by about kTries * kTryNs (4 ms) at most.
constexpr unsigned kTryNs = 1000;
__device__ __forceinline__ bool mbar_wait_quiet(uint64_t* bar, unsigned parity, const int* abort,
                                                unsigned* err) {
  const uint32_t addr = smem_u32(bar);
  WaitLimit limit;
#pragma unroll 1
  do {
#pragma unroll 1
    for (unsigned i = 0; i < kTries; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(addr), "r"(parity), "r"(kTryNs)
          : "memory");
      if (ok) return true;
    }
  } while (!limit.over(abort, err));
  return false;
}

}  // namespace pa
