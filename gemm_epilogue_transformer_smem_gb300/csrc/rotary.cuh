// rotary.cuh -- positions as angles, and the rotation of a pair by them.
//
// A pair i turns by freq[i] radians per position.  An angle only matters
// modulo one turn, so a frequency is kept as the 64-bit fraction of a turn it
// advances per position, step = freq / (2 pi) * 2^64 mod 2^64, and the phase
// of a position is the low 64 bits of position * step.  That product is exact
// for every 64-bit position (negative ones too), where an fp32 product
// position * freq is off by up to half an ulp of the angle -- 0.03 radians at
// position 1e6.  The step is not: freq and freq / (2 pi) are doubles, so that for
// frequencies up to 1 it is off by up to 2^-55 of a turn and the phase of a
// position by that many times the position: 2^-32 of a turn, the last bit used,
// at position 2^23; 2^-24, what bf16 results keep, at 2^31; 2^-15 at 2^40.  The
// phase's top 32 bits are read as a signed fraction of a turn in [-1/2, 1/2).
#pragma once

#include <stdint.h>

namespace ge {

// Phase of `position`, its top 32 bits: a signed fraction of a turn times 2^32.
__device__ __forceinline__ int32_t phase_bits(int64_t position, uint64_t step) {
  return static_cast<int32_t>((static_cast<uint64_t>(position) * step) >> 32);
}

// cos and sin of a phase by the special-function unit: for bf16 tensors, which
// keep 8 bits, and what is summed from them.  The unit is off by up to 2^-21.2 on [-pi, pi]; the phase, rounded
// to its top 23 bits and placed in the mantissa of a float in [2, 4) (an
// int-to-float conversion would take the same unit as sin and cos), by 2 pi
// 2^-24 = 2^-21.3, and its product with pi by 2^-23: 2^-20 together (2^-20.4 the
// largest of 51200 angles, their mean 3e-10; 23 bits cut off instead of rounded
// 2^-19.8 and a mean of 4e-7).
__device__ __forceinline__ void phase_cos_sin_fast(int32_t phase, float& c, float& s) {
  // half a turn on, unsigned; a round past the whole turn is -1/2
  const uint32_t top = (static_cast<uint32_t>(phase) + 0x80000100u) >> 9;
  const float half_turns = __uint_as_float(0x40000000u | top) - 3.0f;      // [-1, 1)
  const float angle = half_turns * 3.14159265358979f;
  c = __cosf(angle);
  s = __sinf(angle);
}

// The same to fp32's accuracy.  The phase splits exactly, in integers, into
// the nearest quarter turn and a rest of at most an eighth of a turn either
// side: x in [-pi/4, pi/4], where the Taylor series of sin to x^9 and of cos
// to x^10 are within 2^-29 (their next terms are below 2e-9 and 2e-10).
__device__ __forceinline__ void phase_cos_sin(int32_t phase, float& c, float& s) {
  const uint32_t quarter = (static_cast<uint32_t>(phase) + 0x20000000u) >> 30;
  const int32_t rest = static_cast<int32_t>(static_cast<uint32_t>(phase) - (quarter << 30));
  const float x = static_cast<float>(rest) * 1.4629180792671596e-9f;
  const float z = x * x;
  float sp = fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f);
  sp = fmaf(z, sp, 1.0f / 120.0f);
  sp = fmaf(z, sp, -1.0f / 6.0f);
  const float sx = fmaf(x * z, sp, x);
  float cp = fmaf(z, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  cp = fmaf(z, cp, -1.0f / 720.0f);
  cp = fmaf(z, cp, 1.0f / 24.0f);
  cp = fmaf(z, cp, -0.5f);
  const float cx = fmaf(z, cp, 1.0f);
  const float u = (quarter & 1u) ? sx : cx, v = (quarter & 1u) ? cx : sx;
  // quarter turns 0..3: cos = cx, -sx, -cx, sx; sin = sx, cx, -sx, -cx
  c = ((quarter + 1u) & 2u) ? -u : u;
  s = (quarter & 2u) ? -v : v;
}

template <bool FAST>
__device__ __forceinline__ void turn_cos_sin(int32_t phase, float& c, float& s) {
  if constexpr (FAST)
    phase_cos_sin_fast(phase, c, s);
  else
    phase_cos_sin(phase, c, s);
}

}  // namespace ge
