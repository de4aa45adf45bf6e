// dropout.cuh -- the dropout mask, drawn anew wherever it is needed.
//
// Philox 4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", 2011) turns a 128-bit counter and a 64-bit key into four 32-bit
// words.  Key: the seed.  Counter: (column / 8, row, site, step), so that an
// element's number depends on nothing but its place, the call's site, the seed
// and the step in device memory: the forward and the backward pass, a kernel over
// stored rows and an output tile of a GEMM all draw the same mask.  Each of a
// counter's eight columns takes 16 of the 128 bits (columns 2i and 2i + 1 the
// low and the high half of word i), which cost 5 integer instructions an element
// in place of the 10 of 32-bit numbers; probabilities are then multiples of
// 2^-16, and the scale of what is kept is the inverse of that multiple.
#pragma once

#include <stdint.h>

#include "gemm_epi.h"

namespace ge {

// An element whose number is below `threshold` is dropped, one that stays is
// multiplied by 65536 / (65536 - threshold); threshold in [1, 65536] (without
// dropout, step is NULL).  The rounds' keys come with the launch: as operands in
// the constant bank they cost the kernels neither registers nor additions.
struct Dropout {
  const uint64_t* step;  // device
  uint32_t site;
  uint32_t above;  // (threshold << 16) - 1: a number n stays if n << 16 is above it
  float scale;
  uint32_t keys[10][2];
};

inline Dropout dropout_of(const gemm_epi_mask& m) {
  Dropout d{};
  if (m.threshold == 0) return d;
  d.step = m.step;
  d.site = m.site;
  d.above = static_cast<uint32_t>((static_cast<uint64_t>(m.threshold) << 16) - 1);
  d.scale = m.threshold == 65536 ? 0.0f : static_cast<float>(65536.0 / (65536 - m.threshold));
  for (uint32_t i = 0; i < 10; ++i) {
    d.keys[i][0] = static_cast<uint32_t>(m.seed) + i * 0x9E3779B9u;
    d.keys[i][1] = static_cast<uint32_t>(m.seed >> 32) + i * 0xBB67AE85u;
  }
  return d;
}

__device__ __forceinline__ uint32_t drop_step(const Dropout& d) { return static_cast<uint32_t>(__ldg(d.step)); }

// The words of columns 8 group .. 8 group + 7 of G rows' groups: the rounds in
// step, so that G chains of multiplications run side by side and share the keys.
template <int G>
__device__ __forceinline__ void drop_words(const Dropout& d, uint32_t step, const uint32_t (&row)[G], const uint32_t (&group)[G],
                                           uint32_t (&w)[G][4]) {
#pragma unroll
  for (int g = 0; g < G; ++g) w[g][0] = group[g], w[g][1] = row[g], w[g][2] = d.site, w[g][3] = step;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint64_t x = static_cast<uint64_t>(w[g][0]) * 0xD2511F53u, y = static_cast<uint64_t>(w[g][2]) * 0xCD9E8D57u;
      w[g][0] = static_cast<uint32_t>(y >> 32) ^ w[g][1] ^ d.keys[i][0];
      w[g][2] = static_cast<uint32_t>(x >> 32) ^ w[g][3] ^ d.keys[i][1];
      w[g][1] = static_cast<uint32_t>(y);
      w[g][3] = static_cast<uint32_t>(x);
    }
  }
}

// Whether the column of that number among the eight stays.
__device__ __forceinline__ bool drop_keeps(const uint32_t (&w)[4], int column, uint32_t above) {
  return (column & 1 ? w[column / 2] : w[column / 2] << 16) > above;
}

}  // namespace ge
