// layer_norm_kernels.h -- which kernel serves a call of the layer norm passes:
// shared by their translation units.
#pragma once

#include <stdint.h>

#include "layer_norm.cuh"

namespace ge_norm {

// The kernels of a pass, by what they are compiled for.
struct Kernel {
  void (*fn)(ge::NormParams);
  int warp_bytes;  // dynamic shared memory of a warp
};

enum Form { NARROW, HELD, LONG };  // teams within a warp; rows held by warps; rows read again

// How a row is dealt out and by what kernel.
struct Shape {
  Form form;
  int k;          // HELD: pieces of 256 columns per warp
  int warps;      // of a team
  int teams;      // of a block
  int log_lanes;  // NARROW: of a team
  int rows;       // a team works on at once
  bool staged;    // HELD: weights through shared memory
  int index() const { return form == HELD ? k : form == NARROW ? 0 : 9; }
};

// What the kernels of either pass are chosen by.
struct Choice {
  bool f32, drop, add, wide;
  int index() const { return f32 | drop << 1 | add << 2 | wide << 3; }
};

Kernel forward_kernel(const Shape& s, const Choice& c);
Kernel backward_kernel(const Shape& s, const Choice& c);

// The sum of the blocks' partial sums of dw and db.
extern void (*const weight_grad_kernel)(const float* partials, int blocks, int width, int staged, int N, float* dw, float* db);

}  // namespace ge_norm
