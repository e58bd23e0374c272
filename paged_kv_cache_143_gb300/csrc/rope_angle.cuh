// rope_angle.cuh — the cosine and sine of a rotary pair, shared by the rotary
// kernel and the latent cache write.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// factor * cos and factor * sin of pos * freq radians, pos any int32.
// A product in fp32 would be off by 2^-24 of the whole angle (0.06 rad at
// position 10^6), and FP64 runs at 1/60 of the fp32 rate here. Positions are whole
// numbers and whole turns may be dropped at any point, so the angle is kept in turns
// as a 64-bit fraction: F = freq / (2 pi) * 2^64 modulo 2^64, off by 1 + freq / 4, and
// pos * F modulo 2^64 is pos times as far off, whatever the position. What is left
// is cut to 32 bits and rounded to fp32 at half a turn or less: the angle is off by
// 2^-26 + 2^-32 + |pos| (1 + freq / 4) 2^-64 turns, below 2^-25 for frequencies up to
// 256 at any position. (Sums of two fp32 numbers keep 2^-24 up to position 2^24, but
// 2^-18 at 2^31.)
__device__ __forceinline__ void rope_cos_sin(int32_t pos, float freq, float factor, float& c,
                                             float& s) {
  constexpr uint64_t kInvTwoPi = 11743562013128004905ull;  // 2^66 / (2 pi), rounded down
  const uint32_t bits = __float_as_uint(freq);
  const int e = (int)(bits >> 23 & 0xFFu);
  // |freq| = m 2^(e - 150), so F = m kInvTwoPi 2^(e - 152), from the 96 bits of the product
  const uint32_t m = (bits & 0x7FFFFFu) | (e > 0 ? 0x800000u : 0u);
  const int shift = 152 - max(e, 1);
  const uint64_t low = (uint64_t)m * (uint32_t)kInvTwoPi;
  const uint64_t high = (uint64_t)m * (uint32_t)(kInvTwoPi >> 32) + (low >> 32);
  uint32_t w0 = (uint32_t)low, w1 = (uint32_t)high, w2 = (uint32_t)(high >> 32);
  if (shift >= 32) {
    const bool far = shift >= 64;  // (frequencies below 2^-39)
    w0 = far ? w2 : w1;
    w1 = far ? 0u : w2;
    w2 = 0u;
  }
  uint32_t f0 = __funnelshift_r(w0, w1, shift), f1 = __funnelshift_r(w1, w2, shift);
  if (shift < 0 || shift >= 96) {  // frequencies from 2^26 on, and below 2^-71
    const uint64_t f = shift >= 0 || shift <= -64 ? 0ull : ((uint64_t)w1 << 32 | w0) << -shift;
    f0 = (uint32_t)f;
    f1 = (uint32_t)(f >> 32);
  }
  // the upper half of pos * F
  const uint32_t turns = (uint32_t)pos * f1 + __umulhi((uint32_t)pos, f0) - (pos < 0 ? f0 : 0u);
  sincospif((float)(int32_t)turns * 0x1p-31f, &s, &c);
  c *= factor;
  s *= (bits >> 31) ? -factor : factor;
  if (e == 255) c = s = __uint_as_float(0x7FC00000u);  // a frequency that is no number
}

// One pair turned: (x, y) -> (x c - y s, y c + x s), in fp32.
__device__ __forceinline__ void rope_turn(float& x, float& y, float c, float s) {
  const float u = x * c - y * s;
  y = y * c + x * s;
  x = u;
}

}  // namespace pa
