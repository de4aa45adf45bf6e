// heads.cuh -- rotary positions on the heads of q and k, the RMS norm of each
// head in the same pass, and that pass's backward.
//
// For a head x of D values at position p (r = 1/sqrt(mean x^2 + eps), w the
// norm's weight, R(p) the rotation of each pair (a, b) of the first
// rotary_dim values by its angle, A the amplitude of the rotated part):
//   rotary     y  = A R(p) x                     (inverse: A R(p)^T x)
//   norm       y  = A R(p) (x r w)
//   backward   g  = A R(p)^T dy
//              dx = r (g w - x r mean(g w x r)),  dw = sum over rows of g x r
// Everything is fp32 between one load and one store of each value.
//
// All three are memory-bound (x in, y out; or dy and x in, dx out), so the
// layout serves wide accesses: a lane holds, for every head it works on, pairs
// of 16-byte chunks chosen so that both halves of a pair are in the same lane
// -- chunks i and i + n, n chunks to half the rotated part (half layout) or to
// half the head -- and that neighbouring lanes read neighbouring chunks, so
// that an access of a warp covers whole sectors.  Values are kept as arrays
// of first and of second halves of pairs whatever the layout, so the rotation
// needs no exchange between lanes and runs on packed fp32 pairs.  G = 2^g
// lanes hold a head and reduce its sums with g shuffles; each of a warp's 32 / G
// groups of lanes takes a token of its own and walks through that token's
// heads, so that few heads leave no lane idle and the groups work out their
// angles at once.
#pragma once

#include <stdint.h>

#include "gemm_epi.h"
#include "ptx.cuh"
#include "rotary.cuh"

namespace ge {

constexpr int HD_WARPS = 8;
constexpr int HD_THREADS = 32 * HD_WARPS;
constexpr int HD_MAX_DIM = 512;  // 16 values per lane x 32 lanes
// Resident blocks per SM that the register budget allows, and iterations a
// warp keeps in flight.  Measured on one GB300 with 32 + 8 heads of 128 (bf16):
//   norm, 16384 tokens (336 MB): 56.4 us = 6.0 TB/s, 0.88 of the measured copy;
//     64.3 us with 3 blocks (80 registers, which spill), 59.4 at depth 2, 62.1 at 4;
//     fp32, 8192 tokens (336 MB) 60.2 us, 0.82
//   rotary, 65536 tokens (1.34 GB): 209.3 us = 6.4 TB/s, 0.94; 8192 tokens 28.8
//     us = 0.86; with 4 blocks 212.9 and 30.3, with 2 208.4 and 30.4
//   backward, 16384 tokens (503 MB): 85.5 us = 5.9 TB/s, 0.87; 104.6 us at
//     depth 1, 88.6 at 3, 93.9 at 4
// The norm and the backward pass use 0.42 of the issue slots: beside HBM it is
// latency that is left, of each head's sums over its lanes, hidden by the 16
// warps of an SM that the registers (a norm's weights, angles and one head's
// values) allow.
constexpr int HD_ROTARY_BLOCKS = 3, HD_NORM_BLOCKS = 2, HD_BWD_BLOCKS = 2;
constexpr int HD_FWD_DEPTH = 3, HD_BWD_DEPTH = 2;
// Partial dw rows of the backward pass: one per block, added up by
// head_weight_grad_kernel in a fixed order.
constexpr int HD_MAX_PARTIALS = 512;

enum HeadMode { HEAD_ROTARY = 0, HEAD_NORM = 1, HEAD_NORM_BWD = 2 };

// One of q and k: its tensors' strides are in elements.
struct HeadPart {
  const void* x;
  int64_t x_b, x_t, x_h;
  const void* dy;  // HEAD_NORM_BWD
  int64_t dy_b, dy_t, dy_h;
  void* y;  // output (dx in the backward pass); NULL: not written
  int64_t y_b, y_t, y_h;
  const float* w;  // NULL: 1
  int32_t heads;
};

// How sets of tokens (one to each lane group of a warp) of per_row iterations
// (heads) are shared out to `warps` warps: `rounds` whole sets each, warp by
// warp, and the iterations of the sets left over in order, `base` to each warp
// and one more to each of the first `rest`.
struct HeadShare {
  int32_t warps, per_row, rounds, base, rest;
};

struct HeadParams {
  HeadPart part[2];  // q, k
  int32_t tokens;    // per sequence
  int32_t rows;      // batch * tokens
  int32_t dim, rot_pairs;
  // A head's chunks in pairs: half layout, first_plain pairs of rotated chunks,
  // then the chunks that do not rotate; interleaved, first_plain = 0.
  int32_t first_plain, num_pc;
  int32_t reach;  // values of a head that are worked on: dim, or the rotated ones
  int32_t log_g;        // lanes per head
  HeadShare share[2];   // forward: [0]; backward: of q's and of k's warps
  int32_t q_blocks;     // backward: blocks [0, q_blocks) work on q, the rest on k
  const uint64_t* steps;
  const void* positions;  // NULL: the token's index in its sequence
  int32_t positions_64;
  int64_t pos_b;
  float amplitude, sin_sign, eps, inv_dim;
  float* partials;  // [blocks][dim]
};

// A chunk of V values of type T in memory.
template <class T, int V>
struct HeadChunk;

template <>
struct HeadChunk<uint16_t, 8> {
  uint4 q;
  __device__ __forceinline__ void load(const uint16_t* p) { q = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      v[2 * h] = __uint_as_float(w[h] << 16);
      v[2 * h + 1] = __uint_as_float(w[h] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(ptx::pack_bf16x2(v[0], v[1]), ptx::pack_bf16x2(v[2], v[3]),
                                              ptx::pack_bf16x2(v[4], v[5]), ptx::pack_bf16x2(v[6], v[7]));
  }
};

template <>
struct HeadChunk<float, 4> {
  float4 q;
  __device__ __forceinline__ void load(const float* p) { q = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void unpack(float (&v)[4]) const { v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w; }
  static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};

// Sizes and alignments that 16-byte accesses do not serve: single elements.
template <>
struct HeadChunk<uint16_t, 2> {
  uint32_t q;
  __device__ __forceinline__ void load(const uint16_t* p) {
    q = static_cast<uint32_t>(p[0]) | (static_cast<uint32_t>(p[1]) << 16);
  }
  __device__ __forceinline__ void unpack(float (&v)[2]) const {
    v[0] = __uint_as_float(q << 16);
    v[1] = __uint_as_float(q & 0xFFFF0000u);
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&v)[2]) {
    const uint32_t w = ptx::pack_bf16x2(v[0], v[1]);
    p[0] = static_cast<uint16_t>(w & 0xFFFFu);
    p[1] = static_cast<uint16_t>(w >> 16);
  }
};

template <>
struct HeadChunk<float, 2> {
  float2 q;
  __device__ __forceinline__ void load(const float* p) { q = make_float2(p[0], p[1]); }
  __device__ __forceinline__ void unpack(float (&v)[2]) const { v[0] = q.x, v[1] = q.y; }
  static __device__ __forceinline__ void store(float* p, const float (&v)[2]) { p[0] = v[0], p[1] = v[1]; }
};

// Sum over the 2^log_g lanes of a head.
__device__ __forceinline__ float head_sum(float v, int log_g) {
#pragma unroll
  for (int g = 4; g >= 0; --g)
    if (g < log_g) v += __shfl_xor_sync(0xffffffffu, v, 1 << g);
  return v;
}

// The values of one head in a lane: first and second halves of its 8 pairs,
// two pairs to a float2.
struct HeadPairs {
  float2 a[4], b[4];
};

// Where a lane's values lie in a head: S slots of two chunks of V values.
template <class T, int VALUES, bool HALF>
struct HeadLane {
  using Type = T;
  static constexpr int V = VALUES;
  static constexpr bool HALVES = HALF;
  using Chunk = HeadChunk<T, V>;
  static constexpr int S = 8 / V;
  int off0[S], off1[S];    // element offsets of the two chunks
  bool in0[S], in1[S];     // inside the head
  uint32_t turning;        // bit k: the lane's pair k (k % V of slot k / V) rotates

  // The raw chunks of one head.
  struct Raw {
    Chunk c0[S], c1[S];
  };

  __device__ __forceinline__ void place(const HeadParams& p, int lane_in_group) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int pc = (i << p.log_g) + lane_in_group;
      const int part = HALF && pc < p.first_plain ? 0 : p.first_plain;  // pair-chunks in front of this one's kind
      const int a = 2 * V * part + V * (pc - part);
      const int b = a + V * ((part == 0 && HALF && p.first_plain > 0 ? p.first_plain : p.num_pc) - part);
      in0[i] = pc < p.num_pc && a < p.reach;
      in1[i] = pc < p.num_pc && b < p.reach;
      off0[i] = in0[i] ? a : 0;
      off1[i] = in1[i] ? b : 0;
    }
    turning = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      turning |= static_cast<uint32_t>(pair_of(p, lane_in_group, k / V, k % V) < p.rot_pairs) << k;
  }
  // Index of the head's rotated pair in place j of slot i; past the rotated
  // pairs where there is none.
  __device__ __forceinline__ int pair_of(const HeadParams& p, int lane_in_group, int i, int j) const {
    if (HALF) return ((i << p.log_g) + lane_in_group) * V + j;
    const bool second_chunk = 2 * j >= V;
    return (second_chunk ? in1[i] : in0[i]) ? (second_chunk ? off1[i] : off0[i]) / 2 + j - (second_chunk ? V / 2 : 0)
                                             : p.rot_pairs;
  }

  // Pair j of slot i from the values of the slot's two chunks, and back.
  static __device__ __forceinline__ float& first(float (&v0)[V], float (&v1)[V], int j) {
    return HALF ? v0[j] : 2 * j < V ? v0[(2 * j) % V] : v1[(2 * j) % V];
  }
  static __device__ __forceinline__ float& second(float (&v0)[V], float (&v1)[V], int j) {
    return HALF ? v1[j] : 2 * j < V ? v0[(2 * j + 1) % V] : v1[(2 * j + 1) % V];
  }
  static __device__ __forceinline__ void gather(HeadPairs& x, int i, float (&v0)[V], float (&v1)[V]) {
#pragma unroll
    for (int h = 0; h < V / 2; ++h) {
      x.a[i * V / 2 + h] = make_float2(first(v0, v1, 2 * h), first(v0, v1, 2 * h + 1));
      x.b[i * V / 2 + h] = make_float2(second(v0, v1, 2 * h), second(v0, v1, 2 * h + 1));
    }
  }
  static __device__ __forceinline__ void scatter(const HeadPairs& x, int i, float (&v0)[V], float (&v1)[V]) {
#pragma unroll
    for (int h = 0; h < V / 2; ++h) {
      first(v0, v1, 2 * h) = x.a[i * V / 2 + h].x;
      first(v0, v1, 2 * h + 1) = x.a[i * V / 2 + h].y;
      second(v0, v1, 2 * h) = x.b[i * V / 2 + h].x;
      second(v0, v1, 2 * h + 1) = x.b[i * V / 2 + h].y;
    }
  }

  // Zeros outside the head, and everywhere unless `ok`.
  __device__ __forceinline__ void load(Raw& r, const T* head, bool ok) const {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      r.c0[i] = {};
      r.c1[i] = {};
      if (ok && in0[i]) r.c0[i].load(head + off0[i]);
      if (ok && in1[i]) r.c1[i].load(head + off1[i]);
    }
  }
  static __device__ __forceinline__ void unpack(const Raw& r, HeadPairs& x) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      float v0[V], v1[V];
      r.c0[i].unpack(v0);
      r.c1[i].unpack(v1);
      gather(x, i, v0, v1);
    }
  }
  __device__ __forceinline__ void store(T* head, const HeadPairs& x) const {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      float v0[V], v1[V];
      scatter(x, i, v0, v1);
      if (in0[i]) Chunk::store(head + off0[i], v0);
      if (in1[i]) Chunk::store(head + off1[i], v1);
    }
  }
  // Weights laid out in shared memory, 16-byte aligned.  A chunk outside the
  // head reads the first one: its values are zeros.
  __device__ __forceinline__ void weights_shared(const float* w, HeadPairs& x) const {
    static_assert(V % 4 == 0, "16-byte pieces of weights");
#pragma unroll
    for (int i = 0; i < S; ++i) {
      float v0[V], v1[V];
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const float4 a = *reinterpret_cast<const float4*>(w + off0[i] + j);
        const float4 b = *reinterpret_cast<const float4*>(w + off1[i] + j);
        v0[j] = a.x, v0[j + 1] = a.y, v0[j + 2] = a.z, v0[j + 3] = a.w;
        v1[j] = b.x, v1[j + 1] = b.y, v1[j + 2] = b.z, v1[j + 3] = b.w;
      }
      gather(x, i, v0, v1);
    }
  }
  // The norm's weights in global memory (1 outside the head, or without weights).
  __device__ __forceinline__ void weights(const float* w, HeadPairs& x) const {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      float v0[V], v1[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v0[j] = w != nullptr && in0[i] ? __ldg(w + off0[i] + j) : 1.0f;
        v1[j] = w != nullptr && in1[i] ? __ldg(w + off1[i] + j) : 1.0f;
      }
      gather(x, i, v0, v1);
    }
  }
};

// The rotation of a lane's 8 pairs at one position.  PART: some values of a head
// do not rotate.  Their pairs keep them untouched: c = 1 and s = 0 would let an
// infinity or NaN of one value make its partner NaN.  Kernels of their own, as
// the test costs them up to 3 % (32 + 8 heads of 128, half of each rotated:
// rotary 29.1 -> 29.6 us, norm 55.8 in both, backward 84.5 -> 86.8).
template <class Lane, bool PART>
struct HeadAngles {
  float2 c[4], s[4];  // cos and sin, times the amplitude
  uint32_t turning;   // PART: bit k: pair k rotates

  __device__ __forceinline__ void set(const HeadParams& p, const Lane& l, int lane_in_group, int64_t position) {
    const float as = p.amplitude * p.sin_sign;
    turning = l.turning;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int pair = l.pair_of(p, lane_in_group, k / Lane::V, k % Lane::V);
      float cc = 1.0f, ss = 0.0f;
      if (pair < p.rot_pairs) {
        turn_cos_sin<sizeof(typename Lane::Type) == 2>(phase_bits(position, __ldg(p.steps + pair)), cc, ss);
        cc *= p.amplitude;
        ss *= as;
      }
      if (k & 1)
        c[k / 2].y = cc, s[k / 2].y = ss;
      else
        c[k / 2].x = cc, s[k / 2].x = ss;
    }
  }

  // (a, b) -> (a c - b s, b c + a s).
  __device__ __forceinline__ void rotate(HeadPairs& x) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (!PART) {
        turn(i, x.a[i], x.b[i]);
      } else if constexpr (Lane::HALVES) {  // a slot's pairs rotate all or none
        if ((turning >> (2 * i / Lane::V * Lane::V)) & 1u) turn(i, x.a[i], x.b[i]);
      } else {
        float2 a = x.a[i], b = x.b[i];
        turn(i, a, b);
        if ((turning >> (2 * i)) & 1u) x.a[i].x = a.x, x.b[i].x = b.x;
        if ((turning >> (2 * i + 1)) & 1u) x.a[i].y = a.y, x.b[i].y = b.y;
      }
    }
  }
  __device__ __forceinline__ void turn(int i, float2& a, float2& b) const {
    const float2 x = a, bs = __fmul2_rn(b, s[i]);
    a = make_float2(fmaf(x.x, c[i].x, -bs.x), fmaf(x.y, c[i].y, -bs.y));
    b = __ffma2_rn(x, s[i], __fmul2_rn(b, c[i]));
  }
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Sum of x y over a lane's pairs.
__device__ __forceinline__ float head_dot(const HeadPairs& x, const HeadPairs& y) {
  float2 t = __fmul2_rn(x.a[0], y.a[0]), u = __fmul2_rn(x.b[0], y.b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    t = __ffma2_rn(x.a[i], y.a[i], t);
    u = __ffma2_rn(x.b[i], y.b[i], u);
  }
  t = __fadd2_rn(t, u);
  return t.x + t.y;
}

// 1 / sqrt(mean x^2 + eps) of a head.
__device__ __forceinline__ float head_rms(const HeadPairs& x, const HeadParams& p) {
  return rsqrtf(fmaf(head_sum(head_dot(x, x), p.log_g), p.inv_dim, p.eps));
}

__device__ __forceinline__ int64_t head_position(const HeadParams& p, int b, int t) {
  if (p.positions == nullptr) return t;
  const int64_t at = b * p.pos_b + t;
  return p.positions_64 ? __ldg(static_cast<const long long*>(p.positions) + at)
                        : __ldg(static_cast<const int*>(p.positions) + at);
}

// The token of lane group `group` in set `set` of tokens: its sequence, its
// place there, and whether there is one.
struct HeadRow {
  uint32_t b, t;
  bool ok;
  __device__ __forceinline__ HeadRow(const HeadParams& p, uint32_t set, int group) {
    const uint32_t at = (set << (5 - p.log_g)) + group, rows = static_cast<uint32_t>(p.rows);
    ok = at < rows;
    const uint32_t row = ok ? at : rows - 1;
    b = p.rows == p.tokens ? 0u : row / static_cast<uint32_t>(p.tokens);
    t = row - b * static_cast<uint32_t>(p.tokens);
  }
};

// ---------------------------------------------------------------- arithmetic

// One head forward: norm (r, w) and rotation.
template <bool NORM, class Angles>
__device__ __forceinline__ void head_forward(HeadPairs& v, const HeadPairs& w, const Angles& ang,
                                             const HeadParams& p) {
  if constexpr (NORM) {
    const float2 r = both(head_rms(v, p));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v.a[i] = __fmul2_rn(__fmul2_rn(v.a[i], r), w.a[i]);
      v.b[i] = __fmul2_rn(__fmul2_rn(v.b[i], r), w.b[i]);
    }
  }
  ang.rotate(v);
}

// One head backward: v = x, g = dy in; v = dx out, dw added to where `ok` (a
// lane group without a token adds nothing).  A lane adds its share's terms one
// after the other in fp32, 67 of them with 32 + 8 heads of 128 and 16384 tokens;
// then lane groups, warps and blocks are added up.  The error grows with the
// length of a share; fp64 sums would take 16 registers more.  Against 64 bits dw is
// off by 1.5e-7 of its size (fp32, 999 tokens) and 3.6e-7 (bf16 tensors, whose
// cos and sin are the special-function unit's; 16384 tokens).
template <class Angles>
__device__ __forceinline__ void head_backward(HeadPairs& v, HeadPairs& g, const HeadPairs& w, HeadPairs& dw,
                                              const Angles& ang, const HeadParams& p, bool ok) {
  const float r = head_rms(v, p);
  ang.rotate(g);  // sin_sign = -1: the transpose
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.a[i] = __fmul2_rn(v.a[i], both(r));  // x r
    v.b[i] = __fmul2_rn(v.b[i], both(r));
    if (ok) {
      dw.a[i] = __ffma2_rn(g.a[i], v.a[i], dw.a[i]);
      dw.b[i] = __ffma2_rn(g.b[i], v.b[i], dw.b[i]);
    }
    g.a[i] = __fmul2_rn(g.a[i], w.a[i]);
    g.b[i] = __fmul2_rn(g.b[i], w.b[i]);
  }
  const float m = -head_sum(head_dot(g, v), p.log_g) * p.inv_dim;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.a[i] = __fmul2_rn(both(r), __ffma2_rn(v.a[i], both(m), g.a[i]));
    v.b[i] = __fmul2_rn(both(r), __ffma2_rn(v.b[i], both(m), g.b[i]));
  }
}

// The block's share of one weight gradient: lanes of the same place in their
// group, then warps, in a fixed order.
template <class Lane, int V>
__device__ __forceinline__ void store_partial(const Lane& l, HeadPairs& dw, const HeadParams& p, int group, int warp) {
  __shared__ float part[HD_WARPS][HD_MAX_DIM];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    for (int o = 16; o >= (1 << p.log_g); o >>= 1) {
      dw.a[i].x += __shfl_xor_sync(0xffffffffu, dw.a[i].x, o);
      dw.a[i].y += __shfl_xor_sync(0xffffffffu, dw.a[i].y, o);
      dw.b[i].x += __shfl_xor_sync(0xffffffffu, dw.b[i].x, o);
      dw.b[i].y += __shfl_xor_sync(0xffffffffu, dw.b[i].y, o);
    }
  if (group == 0) {
#pragma unroll
    for (int i = 0; i < Lane::S; ++i) {
      float v0[V], v1[V];
      Lane::scatter(dw, i, v0, v1);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (l.in0[i]) part[warp][l.off0[i] + j] = v0[j];
        if (l.in1[i]) part[warp][l.off1[i] + j] = v1[j];
      }
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < p.dim; d += HD_THREADS) {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < HD_WARPS; ++k) sum += part[k][d];
    p.partials[static_cast<int64_t>(blockIdx.x) * p.dim + d] = sum;
  }
}

// A warp's share, set by set of tokens: iterations [it, end) of set `row`.  All
// warps get the same number of iterations, give or take one, so they end
// together whatever the number of tokens.
struct HeadSpan {
  uint32_t row;
  int it, end, rounds, left;

  __device__ __forceinline__ HeadSpan(const HeadShare& s, int warp) {
    row = warp;
    rounds = s.rounds;
    it = 0;
    end = s.per_row;
    left = 0;
    if (rounds == 0) tail(s, warp);
  }
  __device__ __forceinline__ void tail(const HeadShare& s, int warp) {
    left = s.base + (warp < s.rest ? 1 : 0);
    const uint32_t start = static_cast<uint32_t>(s.base) * warp + min(warp, s.rest);
    row = start / static_cast<uint32_t>(s.per_row);
    it = static_cast<int>(start - row * s.per_row);
    row += static_cast<uint32_t>(s.rounds) * s.warps;
    end = min(s.per_row, it + left);
    left -= end - it;
  }
  __device__ __forceinline__ bool any() const { return it < end; }
  // To the next set of the share, once this one's iterations are done.
  __device__ __forceinline__ void next(const HeadShare& s, int warp) {
    if (rounds > 1) {
      --rounds;
      row += s.warps;
      it = 0;
    } else if (rounds == 1) {
      rounds = 0;
      tail(s, warp);
    } else {
      ++row;
      it = 0;
      end = min(s.per_row, left);
      left -= end;
    }
  }
};

// This lane group's token in one tensor, from head `head` on: one head further
// each iteration.
template <class T>
struct HeadRun {
  T* at;
  int64_t step;

  __device__ __forceinline__ void set(const void* base, int64_t sb, int64_t st, int64_t sh, const HeadRow& r, int head) {
    at = static_cast<T*>(const_cast<void*>(base)) + r.b * sb + r.t * st + head * sh;
    step = sh;
  }
};

// ---------------------------------------------------------------- 16-byte kernels
//
// A warp walks its iterations -- heads of a token, then of the next token it
// has -- and keeps DEPTH of them in flight: per-thread asynchronous copies
// (cp.async) put its chunks into shared-memory slots that only it reads, so
// nothing is held in registers while it travels, there is no block barrier,
// and the loads of the next token run ahead of this one's angles.  Pointers
// step from iteration to iteration; what a token needs (its row, angles) is
// worked out once.

template <class T, bool HALF, int TENSORS>
struct HeadRing {
  static constexpr int V = 16 / sizeof(T);  // a chunk is 16 bytes
  using Lane = HeadLane<T, V, HALF>;
  static constexpr int PER_TENSOR = 2 * Lane::S;       // a lane's chunks of a head
  static constexpr int SLOT = TENSORS * PER_TENSOR;
  static constexpr int DEPTH = TENSORS == 1 ? HD_FWD_DEPTH : HD_BWD_DEPTH;
  static constexpr uint32_t SLOT_BYTES = SLOT * HD_THREADS * 16;
  static constexpr int BYTES = DEPTH * SLOT_BYTES;

  // A chunk outside the head is never copied: zeros, once.
  static __device__ __forceinline__ void clear(uint4* mine, const Lane& l) {
#pragma unroll
    for (int i = 0; i < Lane::S; ++i)
      for (int k = 0; k < DEPTH * TENSORS; ++k) {
        if (!l.in0[i]) mine[(k * PER_TENSOR + 2 * i) * HD_THREADS] = make_uint4(0, 0, 0, 0);
        if (!l.in1[i]) mine[(k * PER_TENSOR + 2 * i + 1) * HD_THREADS] = make_uint4(0, 0, 0, 0);
      }
  }
  // Copies tensor `which`'s chunks of a head into the slot at `slot`.
  static __device__ __forceinline__ void fetch(uint32_t slot, int which, const Lane& l, const T* head) {
    const uint32_t dst = slot + static_cast<uint32_t>(which * PER_TENSOR) * (HD_THREADS * 16u);
#pragma unroll
    for (int i = 0; i < Lane::S; ++i) {
      if (l.in0[i]) ptx::cp_async16(dst + (2 * i) * (HD_THREADS * 16u), head + l.off0[i], 16u);
      if (l.in1[i]) ptx::cp_async16(dst + (2 * i + 1) * (HD_THREADS * 16u), head + l.off1[i], 16u);
    }
  }
  static __device__ __forceinline__ void read(const uint8_t* slot, int which, HeadPairs& x) {
    const uint4* src = reinterpret_cast<const uint4*>(slot) + which * PER_TENSOR * HD_THREADS;
    typename Lane::Raw r;
#pragma unroll
    for (int i = 0; i < Lane::S; ++i) {
      r.c0[i].load(reinterpret_cast<const T*>(src + (2 * i) * HD_THREADS));
      r.c1[i].load(reinterpret_cast<const T*>(src + (2 * i + 1) * HD_THREADS));
    }
    Lane::unpack(r, x);
  }
  static __device__ __forceinline__ uint32_t next(uint32_t at) { return at + SLOT_BYTES == BYTES ? 0u : at + SLOT_BYTES; }
};

template <class T, bool HALF, bool NORM, bool PART>
__global__ void __launch_bounds__(HD_THREADS, NORM ? HD_NORM_BLOCKS : HD_ROTARY_BLOCKS)
    heads_kernel(const __grid_constant__ HeadParams p) {
  using Ring = HeadRing<T, HALF, 1>;
  using Lane = typename Ring::Lane;
  extern __shared__ uint4 head_ring[];  // [DEPTH][SLOT][HD_THREADS]
  __shared__ __align__(16) float weights[2][NORM ? HD_MAX_DIM : 4];
  const int lane = threadIdx.x & 31, warp = blockIdx.x * HD_WARPS + (threadIdx.x >> 5);
  const int group = lane >> p.log_g, in_group = lane & ((1 << p.log_g) - 1);
  const int q_heads = p.part[0].heads;
  const HeadShare& share = p.share[0];
  Lane l;
  l.place(p, in_group);
  uint8_t* mine = reinterpret_cast<uint8_t*>(head_ring + threadIdx.x);
  const uint32_t ring = ptx::smem_addr(mine);
  Ring::clear(head_ring + threadIdx.x, l);

  HeadSpan ahead(share, warp);  // what is fetched next: `n` iterations of run `src`
  HeadRun<T> src;
  int n = 0;
  bool copies = false;
  auto open = [&]() {
    const int k = ahead.it >= q_heads;
    const HeadPart& h = p.part[k];
    const HeadRow r(p, ahead.row, group);
    src.set(h.x, h.x_b, h.x_t, h.x_h, r, ahead.it - (k ? q_heads : 0));
    copies = r.ok;
    const int to = k ? ahead.end : min(ahead.end, q_heads);
    n = to - ahead.it;
    ahead.it = to;
  };
  auto fetch = [&](uint32_t at) {
    if (n > 0) {
      if (copies) Ring::fetch(ring + at, 0, l, src.at);
      src.at += src.step;
      if (--n == 0) {
        if (!ahead.any()) ahead.next(share, warp);
        if (ahead.any()) open();
      }
    }
    // one copy group per iteration, empty past the last, so that "at most
    // DEPTH - 1 groups pending" always means "this iteration landed"
    ptx::cp_async_commit();
  };
  if (ahead.any()) open();
#pragma unroll
  for (int d = 0; d < Ring::DEPTH; ++d) fetch(d * Ring::SLOT_BYTES);

  if constexpr (NORM) {
    for (int i = threadIdx.x; i < 2 * p.dim; i += HD_THREADS) {
      const int k = i >= p.dim, d = i - k * p.dim;
      weights[k][d] = p.part[k].w != nullptr ? __ldg(p.part[k].w + d) : 1.0f;
    }
    __syncthreads();
  }

  uint32_t at = 0;
#pragma unroll 1
  for (HeadSpan now(share, warp); now.any(); now.next(share, warp)) {
    const HeadRow r(p, now.row, group);
    HeadAngles<Lane, PART> ang;
    ang.set(p, l, in_group, head_position(p, r.b, r.t));
#pragma unroll 1
    while (now.any()) {
      const int k = now.it >= q_heads;
      const HeadPart& h = p.part[k];
      const int to = k ? now.end : min(now.end, q_heads);
      HeadRun<T> dst;
      dst.set(h.y, h.y_b, h.y_t, h.y_h, r, now.it - (k ? q_heads : 0));
      HeadPairs w;
      if constexpr (NORM) l.weights_shared(weights[k], w);
#pragma unroll 1
      for (; now.it < to; ++now.it) {
        ptx::cp_async_wait<Ring::DEPTH - 1>();
        HeadPairs v;
        Ring::read(mine + at, 0, v);
        head_forward<NORM>(v, w, ang, p);
        if (r.ok) l.store(dst.at, v);
        dst.at += dst.step;
        fetch(at);  // the slot's values are in registers
        at = Ring::next(at);
      }
    }
  }
  ptx::cp_async_wait<0>();
}

// Backward pass of the norm and rotation.  A block works on q or on k, so that
// its warps keep one weight gradient in registers over all of their share;
// each block leaves one partial row.
template <class T, bool HALF, bool PART>
__global__ void __launch_bounds__(HD_THREADS, HD_BWD_BLOCKS) heads_backward_kernel(const __grid_constant__ HeadParams p) {
  using Ring = HeadRing<T, HALF, 2>;
  using Lane = typename Ring::Lane;
  extern __shared__ uint4 head_ring[];  // [DEPTH][SLOT][HD_THREADS]
  ptx::launch_dependents();
  const int k = static_cast<int>(blockIdx.x) >= p.q_blocks;
  const int lane = threadIdx.x & 31, warp = (blockIdx.x - (k ? p.q_blocks : 0)) * HD_WARPS + (threadIdx.x >> 5);
  const int group = lane >> p.log_g, in_group = lane & ((1 << p.log_g) - 1);
  const HeadPart& h = p.part[k];
  const HeadShare& share = p.share[k];
  Lane l;
  l.place(p, in_group);
  uint8_t* mine = reinterpret_cast<uint8_t*>(head_ring + threadIdx.x);
  const uint32_t ring = ptx::smem_addr(mine);
  Ring::clear(head_ring + threadIdx.x, l);

  HeadSpan ahead(share, warp);  // what is fetched next: `n` iterations of runs `x` and `dy`
  HeadRun<T> x, dy;
  int n = 0;
  bool copies = false;
  auto open = [&]() {
    const HeadRow r(p, ahead.row, group);
    x.set(h.x, h.x_b, h.x_t, h.x_h, r, ahead.it);
    dy.set(h.dy, h.dy_b, h.dy_t, h.dy_h, r, ahead.it);
    copies = r.ok;
    n = ahead.end - ahead.it;
  };
  auto fetch = [&](uint32_t at) {
    if (n > 0) {
      if (copies) {
        Ring::fetch(ring + at, 0, l, x.at);
        Ring::fetch(ring + at, 1, l, dy.at);
      }
      x.at += x.step;
      dy.at += dy.step;
      if (--n == 0) {
        ahead.next(share, warp);
        if (ahead.any()) open();
      }
    }
    ptx::cp_async_commit();
  };
  if (ahead.any()) open();
#pragma unroll
  for (int d = 0; d < Ring::DEPTH; ++d) fetch(d * Ring::SLOT_BYTES);

  __shared__ __align__(16) float weights[HD_MAX_DIM];
  for (int i = threadIdx.x; i < p.dim; i += HD_THREADS) weights[i] = h.w != nullptr ? __ldg(h.w + i) : 1.0f;
  __syncthreads();
  HeadPairs w, dw;
  l.weights_shared(weights, w);
#pragma unroll
  for (int i = 0; i < 4; ++i) dw.a[i] = dw.b[i] = both(0.0f);
  uint32_t at = 0;
#pragma unroll 1
  for (HeadSpan now(share, warp); now.any(); now.next(share, warp)) {
    const HeadRow r(p, now.row, group);
    HeadAngles<Lane, PART> ang;
    ang.set(p, l, in_group, head_position(p, r.b, r.t));
    HeadRun<T> dx;
    dx.set(h.y, h.y_b, h.y_t, h.y_h, r, now.it);
#pragma unroll 1
    for (; now.it < now.end; ++now.it) {
      ptx::cp_async_wait<Ring::DEPTH - 1>();
      HeadPairs v, g;
      Ring::read(mine + at, 0, v);
      Ring::read(mine + at, 1, g);
      head_backward(v, g, w, dw, ang, p, r.ok);
      if (r.ok && h.y != nullptr) l.store(dx.at, v);
      dx.at += dx.step;
      fetch(at);
      at = Ring::next(at);
    }
  }
  ptx::cp_async_wait<0>();
  if (p.partials != nullptr) store_partial<Lane, Ring::V>(l, dw, p, group, threadIdx.x >> 5);
}

// ---------------------------------------------------------------- any alignment
//
// The same passes with single-element accesses, for sizes, strides and
// addresses that 16-byte ones do not serve.  bf16, 8192 tokens of 32 + 8 heads
// of 96 with 24 values rotated in the half layout: rotary 63.9 us (0.29 of the
// measured copy), norm 69.9, backward 138.5 (0.20).

template <class T, bool HALF, bool NORM, bool PART>
__global__ void __launch_bounds__(HD_THREADS, 2) heads_any_kernel(const __grid_constant__ HeadParams p) {
  using Lane = HeadLane<T, 2, HALF>;
  const int lane = threadIdx.x & 31, warp = blockIdx.x * HD_WARPS + (threadIdx.x >> 5);
  const int group = lane >> p.log_g, in_group = lane & ((1 << p.log_g) - 1);
  const int q_heads = p.part[0].heads;
  Lane l;
  l.place(p, in_group);
#pragma unroll 1
  for (HeadSpan now(p.share[0], warp); now.any(); now.next(p.share[0], warp)) {
    const HeadRow r(p, now.row, group);
    HeadAngles<Lane, PART> ang;
    ang.set(p, l, in_group, head_position(p, r.b, r.t));
#pragma unroll 1
    while (now.any()) {
      const int k = now.it >= q_heads;
      const HeadPart& h = p.part[k];
      const int first = now.it - (k ? q_heads : 0);
      const int to = k ? now.end : min(now.end, q_heads);
      HeadRun<T> x, y;
      x.set(h.x, h.x_b, h.x_t, h.x_h, r, first);
      y.set(h.y, h.y_b, h.y_t, h.y_h, r, first);
      HeadPairs w;
      if constexpr (NORM) l.weights(h.w, w);
#pragma unroll 1
      for (; now.it < to; ++now.it) {
        typename Lane::Raw raw;
        l.load(raw, x.at, r.ok);
        HeadPairs v;
        Lane::unpack(raw, v);
        head_forward<NORM>(v, w, ang, p);
        if (r.ok) l.store(y.at, v);
        x.at += x.step;
        y.at += y.step;
      }
    }
  }
}

template <class T, bool HALF, bool PART>
__global__ void __launch_bounds__(HD_THREADS, HD_BWD_BLOCKS)
    heads_backward_any_kernel(const __grid_constant__ HeadParams p) {
  using Lane = HeadLane<T, 2, HALF>;
  ptx::launch_dependents();
  const int k = static_cast<int>(blockIdx.x) >= p.q_blocks;
  const int lane = threadIdx.x & 31, warp = (blockIdx.x - (k ? p.q_blocks : 0)) * HD_WARPS + (threadIdx.x >> 5);
  const int group = lane >> p.log_g, in_group = lane & ((1 << p.log_g) - 1);
  const HeadPart& h = p.part[k];
  Lane l;
  l.place(p, in_group);
  HeadPairs w, dw;
  l.weights(h.w, w);
#pragma unroll
  for (int i = 0; i < 4; ++i) dw.a[i] = dw.b[i] = both(0.0f);
#pragma unroll 1
  for (HeadSpan now(p.share[k], warp); now.any(); now.next(p.share[k], warp)) {
    const HeadRow r(p, now.row, group);
    HeadAngles<Lane, PART> ang;
    ang.set(p, l, in_group, head_position(p, r.b, r.t));
    HeadRun<T> x, dy, dx;
    x.set(h.x, h.x_b, h.x_t, h.x_h, r, now.it);
    dy.set(h.dy, h.dy_b, h.dy_t, h.dy_h, r, now.it);
    dx.set(h.y, h.y_b, h.y_t, h.y_h, r, now.it);
#pragma unroll 1
    for (; now.it < now.end; ++now.it) {
      typename Lane::Raw rx, rg;
      l.load(rx, x.at, r.ok);
      l.load(rg, dy.at, r.ok);
      HeadPairs v, g;
      Lane::unpack(rx, v);
      Lane::unpack(rg, g);
      head_backward(v, g, w, dw, ang, p, r.ok);
      if (r.ok && h.y != nullptr) l.store(dx.at, v);
      x.at += x.step;
      dy.at += dy.step;
      dx.at += dx.step;
    }
  }
  if (p.partials != nullptr) store_partial<Lane, 2>(l, dw, p, group, threadIdx.x >> 5);
}

// dw[d] = sum over the blocks' partial rows, q's before q_blocks and k's after
// it, in a fixed order (the result does not depend on which block finished
// first).  Launched as a dependent of the backward kernel.  Block: 32 columns x 32 row groups; grid y 0: q, 1: k.  A gradient
// that is NULL is not wanted.
__global__ void __launch_bounds__(1024) head_weight_grad_kernel(const float* partials, int q_blocks, int blocks,
                                                                int dim, float* dw_q, float* dw_k) {
  __shared__ float part[32][33];
  ptx::wait_dependencies();  // launched beside the backward kernel's end
  const int col = blockIdx.x * 32 + threadIdx.x;
  float* dst = blockIdx.y == 0 ? dw_q : dw_k;
  if (dst == nullptr) return;
  const int begin = blockIdx.y == 0 ? 0 : q_blocks, end = blockIdx.y == 0 ? q_blocks : blocks;
  float sum = 0.0f;
  if (col < dim)
    for (int r = begin + threadIdx.y; r < end; r += 32) sum += partials[static_cast<int64_t>(r) * dim + col];
  part[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0 && col < dim) {
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < 32; ++r) t += part[r][threadIdx.x];
    dst[col] = t;
  }
}

}  // namespace ge
