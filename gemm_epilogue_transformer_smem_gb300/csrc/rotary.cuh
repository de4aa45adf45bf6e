// rotary.cuh -- positions as angles, and the rotation of a pair by them.
//
// A pair i turns by freq[i] radians per position.  An angle only matters
// modulo one turn, so a frequency is kept as the 64-bit fraction of a turn it
// advances per position, step = freq / (2 pi) * 2^64 mod 2^64, and the phase
// of a position is the low 64 bits of position * step: exact for every 64-bit
// position (negative ones too), where an fp32 product position * freq is off
// by up to half an ulp of the angle -- 0.03 radians at position 1e6.  The
// phase's top 32 bits are read as a signed fraction of a turn in [-1/2, 1/2).
#pragma once

#include <stdint.h>

namespace ge {

// Signed turns of phase `position * step`: the top 32 of its 64 bits.
__device__ __forceinline__ float phase_turns(int64_t position, uint64_t step) {
  const uint64_t phase = static_cast<uint64_t>(position) * step;
  return static_cast<float>(static_cast<int32_t>(phase >> 32)) * 2.3283064365386963e-10f;  // 2^-32
}

// cos and sin of `turns` in [-1/2, 1/2).  FAST: the special-function unit, off
// by about 2^-21; a bf16 result keeps 8 bits, so its rounding hides that.
// fp32 results take the accurate functions.
template <bool FAST>
__device__ __forceinline__ void turn_cos_sin(float turns, float& c, float& s) {
  if constexpr (FAST) {
    const float angle = turns * 6.2831853071795865f;
    c = __cosf(angle);
    s = __sinf(angle);
  } else {
    sincospif(2.0f * turns, &s, &c);
  }
}

}  // namespace ge
