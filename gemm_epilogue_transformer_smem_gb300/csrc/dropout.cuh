// dropout.cuh -- the dropout mask, drawn anew wherever it is needed.
//
// Philox 4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", 2011) turns a 128-bit counter and a 64-bit key into four 32-bit
// words.  Key: the seed.  Counter: (column / 8, row, site, step), so that an
// element's number depends on nothing but its place, the call's site and the
// state in device memory: the forward and the backward pass, a kernel over
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
// dropout, state is NULL).
struct Dropout {
  const uint64_t* state;  // device: seed, step
  uint32_t site;
  uint32_t above;  // (threshold << 16) - 1: a number n stays if n << 16 is above it
  float scale;
};

inline Dropout dropout_of(const gemm_epi_mask& m) {
  if (m.threshold == 0) return Dropout{};
  return Dropout{m.state, m.site, static_cast<uint32_t>((static_cast<uint64_t>(m.threshold) << 16) - 1),
                 m.threshold == 65536 ? 0.0f : static_cast<float>(65536.0 / (65536 - m.threshold))};
}

struct DropKey {
  uint32_t k0, k1, site, step;
};

__device__ __forceinline__ DropKey drop_key(const Dropout& d) {
  const uint64_t seed = __ldg(d.state), step = __ldg(d.state + 1);
  return DropKey{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), d.site, static_cast<uint32_t>(step)};
}

// The words of columns 8 group .. 8 group + 7 of a row.
__device__ __forceinline__ void drop_words(const DropKey& key, uint32_t row, uint32_t group, uint32_t (&w)[4]) {
  uint32_t a = group, b = row, c = key.site, d = key.step;
#pragma unroll
  for (uint32_t i = 0; i < 10; ++i) {
    const uint64_t x = static_cast<uint64_t>(a) * 0xD2511F53u, y = static_cast<uint64_t>(c) * 0xCD9E8D57u;
    a = static_cast<uint32_t>(y >> 32) ^ b ^ (key.k0 + i * 0x9E3779B9u);
    c = static_cast<uint32_t>(x >> 32) ^ d ^ (key.k1 + i * 0xBB67AE85u);
    b = static_cast<uint32_t>(y);
    d = static_cast<uint32_t>(x);
  }
  w[0] = a, w[1] = b, w[2] = c, w[3] = d;
}

// Whether the column of that number among the eight stays.
__device__ __forceinline__ bool drop_keeps(const uint32_t (&w)[4], int column, uint32_t above) {
  return (column & 1 ? w[column / 2] : w[column / 2] << 16) > above;
}

// Eight columns of a row in place.  What is dropped is zero whatever it held.
__device__ __forceinline__ void drop8(const Dropout& d, const DropKey& key, uint32_t row, uint32_t group, float (&v)[8]) {
  uint32_t w[4];
  drop_words(key, row, group, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = drop_keeps(w, j, d.above) ? v[j] * d.scale : 0.0f;
}

}  // namespace ge
