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
// layout serves wide accesses: a lane holds, for every head it works on, two
// chunks of V consecutive values chosen so that both halves of a pair are in
// the same lane -- chunks i and i + half / V when pairs are (i, i + half),
// neighbouring chunks when they are (2i, 2i + 1).  The rotation then needs no
// exchange between lanes.  G = 2^g lanes hold a head and reduce its sums with
// g shuffles; a warp works on 32 / G heads of one token at a time, and computes
// that token's angles once for all of them.
#pragma once

#include <stdint.h>

#include "gemm_epi.h"
#include "ptx.cuh"
#include "rotary.cuh"

namespace ge {

constexpr int HD_WARPS = 8;
constexpr int HD_BWD_BLOCKS = 2;  // resident blocks per SM of the backward pass
constexpr int HD_THREADS = 32 * HD_WARPS;
constexpr int HD_MAX_DIM = 512;  // 16 values per lane x 32 lanes
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
  int32_t iters;  // ceil(heads / (32 / G))
};

struct HeadParams {
  HeadPart part[2];  // q, k
  int32_t tokens;    // per sequence
  int32_t rows;      // batch * tokens
  int32_t dim, rot_pairs;
  int32_t first_plain;  // pair-chunk index of the first chunks that do not rotate
  int32_t num_pc;       // pair-chunks per head
  int32_t log_g;        // lanes per head
  int32_t iters_per_unit, units_per_row;
  const uint64_t* steps;
  const void* positions;  // NULL: the token's index in its sequence
  int32_t positions_64;
  int64_t pos_b;
  float amplitude, sin_sign, eps, inv_dim;
  float* partials;  // [blocks][2][dim]
};

// V values of type T at p, as floats.
template <class T, int V>
struct HeadIO;

template <>
struct HeadIO<uint16_t, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ Raw load(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }
  static __device__ __forceinline__ void unpack(const Raw& q, float (&v)[8]) {
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
struct HeadIO<float, 8> {
  struct Raw {
    float4 a, b;
  };
  static __device__ __forceinline__ Raw load(const float* p) {
    return Raw{reinterpret_cast<const float4*>(p)[0], reinterpret_cast<const float4*>(p)[1]};
  }
  static __device__ __forceinline__ void unpack(const Raw& q, float (&v)[8]) {
    v[0] = q.a.x, v[1] = q.a.y, v[2] = q.a.z, v[3] = q.a.w;
    v[4] = q.b.x, v[5] = q.b.y, v[6] = q.b.z, v[7] = q.b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// Sizes and alignments that 16-byte accesses do not serve: single elements.
template <>
struct HeadIO<uint16_t, 2> {
  using Raw = uint32_t;
  static __device__ __forceinline__ Raw load(const uint16_t* p) {
    return static_cast<uint32_t>(p[0]) | (static_cast<uint32_t>(p[1]) << 16);
  }
  static __device__ __forceinline__ void unpack(const Raw& q, float (&v)[2]) {
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
struct HeadIO<float, 2> {
  using Raw = float2;
  static __device__ __forceinline__ Raw load(const float* p) { return make_float2(p[0], p[1]); }
  static __device__ __forceinline__ void unpack(const Raw& q, float (&v)[2]) { v[0] = q.x, v[1] = q.y; }
  static __device__ __forceinline__ void store(float* p, const float (&v)[2]) { p[0] = v[0], p[1] = v[1]; }
};

// Sum over the 2^log_g lanes of a head.
__device__ __forceinline__ float head_sum(float v, int log_g) {
  for (int o = (1 << log_g) >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The pair-chunks of one lane: 2 V values in each of S slots.
template <class T, int V, bool HALF>
struct HeadLane {
  using IO = HeadIO<T, V>;
  static constexpr int S = 8 / V;  // slots: 16 values per lane
  int off0[S], off1[S];            // element offsets of the two chunks; -1: outside the head
  float c[S][V], s[S][V];

  __device__ __forceinline__ void place(const HeadParams& p, int lane_in_group) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int pc = (i << p.log_g) + lane_in_group;
      int a = 2 * V * pc, b = a + V;
      if (HALF && pc < p.first_plain) {
        a = V * pc;
        b = p.rot_pairs + V * pc;
      }
      off0[i] = pc < p.num_pc ? a : -1;
      off1[i] = pc < p.num_pc && b < p.dim ? b : -1;
    }
  }

  // cos and sin of each pair at `position`; 1 and 0 where nothing rotates.
  __device__ __forceinline__ void angles(const HeadParams& p, int lane_in_group, int64_t position) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int pair0 = ((i << p.log_g) + lane_in_group) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        c[i][j] = 1.0f;
        s[i][j] = 0.0f;
        if (pair0 + j < p.rot_pairs) {
          float cc, ss;
          turn_cos_sin<sizeof(T) == 2>(phase_turns(position, __ldg(p.steps + pair0 + j)), cc, ss);
          c[i][j] = cc * p.amplitude;
          s[i][j] = ss * (p.amplitude * p.sin_sign);
        }
      }
    }
  }

  // (a, b) -> (a c - b s, b c + a s) on every pair of slot i.
  __device__ __forceinline__ void rotate(int i, float (&v0)[V], float (&v1)[V]) const {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float& a = HALF ? v0[j] : 2 * j < V ? v0[(2 * j) % V] : v1[(2 * j) % V];
      float& b = HALF ? v1[j] : 2 * j < V ? v0[(2 * j + 1) % V] : v1[(2 * j + 1) % V];
      const float x = a, y = b;
      a = fmaf(x, c[i][j], -(y * s[i][j]));
      b = fmaf(y, c[i][j], x * s[i][j]);
    }
  }
};

// The values of one head in a lane.
template <class T, int V, bool HALF>
struct HeadValues {
  using Lane = HeadLane<T, V, HALF>;
  using IO = HeadIO<T, V>;
  typename IO::Raw r0[Lane::S], r1[Lane::S];

  __device__ __forceinline__ void load(const Lane& l, const T* head, bool ok) {
#pragma unroll
    for (int i = 0; i < Lane::S; ++i) {
      r0[i] = {};
      r1[i] = {};
      if (ok && l.off0[i] >= 0) r0[i] = IO::load(head + l.off0[i]);
      if (ok && l.off1[i] >= 0) r1[i] = IO::load(head + l.off1[i]);
    }
  }
  __device__ __forceinline__ void unpack(float (&v0)[Lane::S][V], float (&v1)[Lane::S][V]) const {
#pragma unroll
    for (int i = 0; i < Lane::S; ++i) {
      IO::unpack(r0[i], v0[i]);
      IO::unpack(r1[i], v1[i]);
    }
  }
};

template <class T, int V, bool HALF, int MODE>
__global__ void __launch_bounds__(HD_THREADS, MODE == HEAD_NORM_BWD ? HD_BWD_BLOCKS : 3) heads_kernel(const __grid_constant__ HeadParams p) {
  using Lane = HeadLane<T, V, HALF>;
  using Values = HeadValues<T, V, HALF>;
  using IO = HeadIO<T, V>;
  constexpr int S = Lane::S;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = lane >> p.log_g, in_group = lane & ((1 << p.log_g) - 1);
  const int heads_per_iter = 32 >> p.log_g;
  Lane l;
  l.place(p, in_group);

  float dw[2][S][2][V];  // HEAD_NORM_BWD: this lane's share of each weight gradient
  if constexpr (MODE == HEAD_NORM_BWD) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) dw[k][i][0][j] = dw[k][i][1][j] = 0.0f;
  }

  const int64_t units = static_cast<int64_t>(p.rows) * p.units_per_row;
  const int64_t unit_stride = static_cast<int64_t>(gridDim.x) * HD_WARPS;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * HD_WARPS + warp; u < units; u += unit_stride) {
    const int row = static_cast<int>(u / p.units_per_row);
    const int first = static_cast<int>(u - static_cast<int64_t>(row) * p.units_per_row) * p.iters_per_unit;
    const int b = row / p.tokens, t = row - b * p.tokens;
    int64_t position = t;
    if (p.positions != nullptr) {
      const int64_t at = b * p.pos_b + t;
      position = p.positions_64 ? static_cast<const int64_t*>(p.positions)[at]
                                : static_cast<const int32_t*>(p.positions)[at];
    }
    l.angles(p, in_group, position);

    int begin = first, end = first + p.iters_per_unit;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const HeadPart& h = p.part[k];
      const int from = max(begin, 0), to = min(end, h.iters);
      begin -= h.iters;
      end -= h.iters;
      if (from >= to) continue;
      const T* x = static_cast<const T*>(h.x) + b * h.x_b + t * h.x_t;
      const T* dy = MODE == HEAD_NORM_BWD ? static_cast<const T*>(h.dy) + b * h.dy_b + t * h.dy_t : nullptr;
      T* y = static_cast<T*>(h.y);
      if (y != nullptr) y += b * h.y_b + t * h.y_t;
      float w0[S][V], w1[S][V];
      if constexpr (MODE != HEAD_ROTARY) {
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            w0[i][j] = h.w != nullptr && l.off0[i] >= 0 ? __ldg(h.w + l.off0[i] + j) : 1.0f;
            w1[i][j] = h.w != nullptr && l.off1[i] >= 0 ? __ldg(h.w + l.off1[i] + j) : 1.0f;
          }
      }
      Values nx, ng;  // the next iteration's values, in flight
      const int head0 = from * heads_per_iter + group;
      nx.load(l, x + head0 * h.x_h, head0 < h.heads);
      if constexpr (MODE == HEAD_NORM_BWD) ng.load(l, dy + head0 * h.dy_h, head0 < h.heads);
      for (int it = from; it < to; ++it) {
        const int head = it * heads_per_iter + group;
        const bool ok = head < h.heads;
        float v0[S][V], v1[S][V], g0[S][V], g1[S][V];
        nx.unpack(v0, v1);
        if constexpr (MODE == HEAD_NORM_BWD) ng.unpack(g0, g1);
        if (it + 1 < to) {
          const int nh = head + heads_per_iter;
          nx.load(l, x + nh * h.x_h, nh < h.heads);
          if constexpr (MODE == HEAD_NORM_BWD) ng.load(l, dy + nh * h.dy_h, nh < h.heads);
        }
        if constexpr (MODE != HEAD_ROTARY) {
          float ss = 0.0f;
#pragma unroll
          for (int i = 0; i < S; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(v0[i][j], v0[i][j], fmaf(v1[i][j], v1[i][j], ss));
          // A lane group past the last head holds zeros: r = 0 keeps them zero
          // whatever eps is.
          const float mean = head_sum(ss, p.log_g) * p.inv_dim;
          const float r = ok ? 1.0f / sqrtf(mean + p.eps) : 0.0f;
          if constexpr (MODE == HEAD_NORM) {
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
              for (int j = 0; j < V; ++j) {
                v0[i][j] *= r * w0[i][j];
                v1[i][j] *= r * w1[i][j];
              }
          } else {
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < S; ++i) {
              l.rotate(i, g0[i], g1[i]);  // sin_sign = -1: the transpose
#pragma unroll
              for (int j = 0; j < V; ++j) {
                v0[i][j] *= r;  // x r
                v1[i][j] *= r;
                dw[k][i][0][j] = fmaf(g0[i][j], v0[i][j], dw[k][i][0][j]);
                dw[k][i][1][j] = fmaf(g1[i][j], v1[i][j], dw[k][i][1][j]);
                g0[i][j] *= w0[i][j];
                g1[i][j] *= w1[i][j];
                dot = fmaf(g0[i][j], v0[i][j], fmaf(g1[i][j], v1[i][j], dot));
              }
            }
            const float m = head_sum(dot, p.log_g) * p.inv_dim;
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
              for (int j = 0; j < V; ++j) {
                v0[i][j] = r * fmaf(-v0[i][j], m, g0[i][j]);
                v1[i][j] = r * fmaf(-v1[i][j], m, g1[i][j]);
              }
          }
        }
#pragma unroll
        for (int i = 0; i < S; ++i) {
          if constexpr (MODE != HEAD_NORM_BWD) l.rotate(i, v0[i], v1[i]);
          if (ok && y != nullptr) {
            T* yh = y + head * h.y_h;
            if (l.off0[i] >= 0) IO::store(yh + l.off0[i], v0[i]);
            if (l.off1[i] >= 0) IO::store(yh + l.off1[i], v1[i]);
          }
        }
      }
    }
  }

  if constexpr (MODE == HEAD_NORM_BWD) {
    if (p.partials != nullptr) {
      // Lanes of the same place in their group, then warps, in a fixed order.
      __shared__ float part[HD_WARPS][HD_MAX_DIM];
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            float a = k == 0 ? dw[0][i][0][j] : dw[1][i][0][j], e = k == 0 ? dw[0][i][1][j] : dw[1][i][1][j];
            for (int o = 16; o >= (1 << p.log_g); o >>= 1) {
              a += __shfl_xor_sync(0xffffffffu, a, o);
              e += __shfl_xor_sync(0xffffffffu, e, o);
            }
            if (group == 0) {
              if (l.off0[i] >= 0) part[warp][l.off0[i] + j] = a;
              if (l.off1[i] >= 0) part[warp][l.off1[i] + j] = e;
            }
          }
        __syncthreads();
        for (int d = threadIdx.x; d < p.dim; d += HD_THREADS) {
          float sum = 0.0f;
#pragma unroll
          for (int w = 0; w < HD_WARPS; ++w) sum += part[w][d];
          p.partials[(static_cast<int64_t>(blockIdx.x) * 2 + k) * p.dim + d] = sum;
        }
        __syncthreads();
      }
    }
  }
}

// dw[d] = sum over the blocks' partial rows, in a fixed order (the result does
// not depend on which block finished first).  Block: 32 columns x 32 row
// groups.  dw_q / dw_k NULL: that gradient is not wanted.
__global__ void __launch_bounds__(1024) head_weight_grad_kernel(const float* partials, int n, int dim, float* dw_q,
                                                                float* dw_k) {
  __shared__ float part[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;  // of 2 * dim
  float sum = 0.0f;
  if (col < 2 * dim)
    for (int r = threadIdx.y; r < n; r += 32) sum += partials[static_cast<int64_t>(r) * 2 * dim + col];
  part[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0 && col < 2 * dim) {
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < 32; ++r) t += part[r][threadIdx.x];
    float* dst = col < dim ? dw_q : dw_k;
    if (dst != nullptr) dst[col < dim ? col : col - dim] = t;
  }
}

}  // namespace ge
