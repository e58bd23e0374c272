// rope_angle.cuh — the cosine and sine of a rotary pair, shared by the rotary
// kernel and the latent cache write.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// factor * cos and factor * sin of pos * freq radians, pos any int32.
// A product in fp32 would be off by 2^-24 of the whole angle (0.06 rad at
// position 10^6), so the angle is kept in turns as an unevaluated sum: freq /
// (2 pi) = fh + fl to ~2^-48, pos = hi * 2^16 + lo (both exact in fp32), every
// partial product split by an fma into its rounding and its remainder. Whole
// turns are dropped from the large terms exactly before the small ones are
// added; what is left is below half a turn, off by about 2^-25 turns (plus
// 2^-48 of the angle). FP64, which would do, runs at 1/60 of the fp32 rate here.
__device__ __forceinline__ void rope_cos_sin(int32_t pos, float freq, float factor, float& c,
                                             float& s) {
  constexpr double kInvTwoPi = 0.15915494309189533577;  // 1 / (2 pi)
  constexpr float kHi = static_cast<float>(kInvTwoPi);
  constexpr float kLo = static_cast<float>(kInvTwoPi - static_cast<double>(kHi));
  const float fh = freq * kHi;
  const float fl = fmaf(freq, kHi, -fh) + freq * kLo;
  const float a = static_cast<float>(pos >> 16) * 65536.f;
  const float b = static_cast<float>(pos & 0xFFFF);
  const float pa = a * fh, pb = b * fh;
  float t = (pa - rintf(pa)) + (pb - rintf(pb));
  t -= rintf(t);
  t += fmaf(a, fh, -pa) + fmaf(b, fh, -pb) + a * fl + b * fl;
  t -= rintf(t);
  sincospif(2.f * t, &s, &c);
  c *= factor;
  s *= factor;
}

// One pair turned: (x, y) -> (x c - y s, y c + x s), in fp32.
__device__ __forceinline__ void rope_turn(float& x, float& y, float c, float s) {
  const float u = x * c - y * s;
  y = y * c + x * s;
  x = u;
}

}  // namespace pa
