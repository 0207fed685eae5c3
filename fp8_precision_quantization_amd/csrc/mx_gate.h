// The gate functions of the gated activation and the value of a scale byte,
// shared by the kernel that takes the activation from memory and those that
// form it from their accumulators.
#pragma once

#include "mx_device.h"

namespace mx {

// s = s(t) = 1 / (1 + e^-t), and dt = g t'(g).  Both terms of the denominator
// are taken times 2^-32: 1 / x would otherwise come out as 0 for x above
// 2^126, where s is still a (subnormal) binary32 that a large factor can
// bring back.  e^-t 2^-32 overflows to Inf for t below about -110, whose
// reciprocal is 0, as s rounds to.  In the GELU s is exactly
// 0 or 1 in binary32 long before |g| = 32; beyond that t and dt are those of
// +-32, so that g^3 cannot overflow into 0 * Inf (a NaN stays one).
template <bool GELU>
__device__ __forceinline__ void gate(float g, float& s, float& dt) {
  constexpr float kA = 1.5957691216057308f, kB = 0.044715f;
  float t = g;
  dt = g;
  if constexpr (GELU) {
    g = __builtin_fabsf(g) > 32.0f ? __builtin_copysignf(32.0f, g) : g;
    const float g2 = g * g;
    t = kA * g * (1.0f + kB * g2);
    dt = kA * g * (1.0f + 3.0f * kB * g2);
  }
  const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(t, -1.44269504088896341f, -32.0f));
  s = __builtin_amdgcn_rcpf(0x1p-32f + e) * 0x1p-32f;
}

// act(g); a gate far on the negative side gives 0 (s is 0 there).
template <bool GELU>
__device__ __forceinline__ float act_of(float g) {
  float s, dt;
  gate<GELU>(g, s, dt);
  return g * s;
}

// 2^(byte - 127) as a binary32: byte 0 is the subnormal 2^-127, 0xFF NaN.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  const uint32_t bits = byte << 23;
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 0xFF ? 0x7FC00000u : bits);
}

}  // namespace mx
