// mbar_poll.cuh — polling an mbarrier among other things (the latent kernels).
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

}  // namespace pa
