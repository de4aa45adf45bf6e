// layer_norm.cuh -- dropout, and layer norm with the dropout and the residual
// add in front of it in the same pass, and that pass's backward.
//
// For a row x of N values (D: dropout, w and b the norm's weight and bias):
//   dropout    y  = D(x) + residual
//   norm       h  = D(x) + residual,  mean and variance of h,
//              r  = 1 / sqrt(variance + eps),  y = (h - mean) r w + b
//   backward   n  = (h - mean) r,  a = dy w
//              g  = r (a - mean(a) - n mean(a n)) + add     (the gradient of h)
//              d_residual = g,  dx = D(g),  dw = sum of dy n,  db = sum of dy
// Everything is fp32 between one load and one store of each value.  The
// variance is that of the differences from a mean taken first, never a
// difference of squares.
//
// All of it is memory-bound, so a row is read once: a team of threads -- part of
// a warp, a warp, or a block, as the width asks for -- holds a row in registers
// while its sums are taken, each thread K groups of 8 neighbouring columns
// (16-byte accesses, neighbouring threads neighbouring groups).  The teams stay
// for all rows, so that the next rows are on their way while one is worked on:
// per-thread asynchronous copies bring them into shared-memory slots that only
// that thread reads, without a barrier and without registers.
#pragma once

#include <stdint.h>

#include "dropout.cuh"
#include "ptx.cuh"

namespace ge {

// ------------------------------------------------------------------ values

// Eight neighbouring values of a row as they lie in memory.
template <class T>
struct Group;

template <>
struct Group<uint16_t> {
  static constexpr int PIECES = 1;  // of 16 bytes
  uint4 q[1];
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      v[2 * h] = __uint_as_float(w[h] << 16);
      v[2 * h + 1] = __uint_as_float(w[h] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void pack(const float (&v)[8]) {
    q[0] = make_uint4(ptx::pack_bf16x2(v[0], v[1]), ptx::pack_bf16x2(v[2], v[3]), ptx::pack_bf16x2(v[4], v[5]),
                      ptx::pack_bf16x2(v[6], v[7]));
  }
  static __device__ __forceinline__ float load_one(const uint16_t* p) {
    return __uint_as_float(static_cast<uint32_t>(*p) << 16);
  }
  static __device__ __forceinline__ void store_one(uint16_t* p, float v) {
    *p = static_cast<uint16_t>(ptx::pack_bf16x2(v, 0.0f) & 0xFFFFu);
  }
};

template <>
struct Group<float> {
  static constexpr int PIECES = 2;
  uint4 q[2];
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[4 * i] = __uint_as_float(q[i].x);
      v[4 * i + 1] = __uint_as_float(q[i].y);
      v[4 * i + 2] = __uint_as_float(q[i].z);
      v[4 * i + 3] = __uint_as_float(q[i].w);
    }
  }
  __device__ __forceinline__ void pack(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      q[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                        __float_as_uint(v[4 * i + 3]));
  }
  static __device__ __forceinline__ float load_one(const float* p) { return *p; }
  static __device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
};

// The first `valid` (up to 8) of a group's values, zeros behind them.  `wide`:
// the group starts on 16 bytes.
template <class T>
__device__ __forceinline__ void load_group(const T* p, int valid, bool wide, float (&v)[8]) {
  if (wide && valid >= 8) {
    Group<T> g;
#pragma unroll
    for (int i = 0; i < Group<T>::PIECES; ++i) g.q[i] = reinterpret_cast<const uint4*>(p)[i];
    g.unpack(v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < valid ? Group<T>::load_one(p + j) : 0.0f;
  }
}

template <class T>
__device__ __forceinline__ void store_group(T* p, int valid, bool wide, const float (&v)[8]) {
  if (wide && valid >= 8) {
    Group<T> g;
    g.pack(v);
#pragma unroll
    for (int i = 0; i < Group<T>::PIECES; ++i) reinterpret_cast<uint4*>(p)[i] = g.q[i];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) Group<T>::store_one(p + j, v[j]);
  }
}

// Weights of a group's columns, `none` without any.
__device__ __forceinline__ void load_weights(const float* w, int col, int valid, bool wide, float none, float (&v)[8]) {
  if (w != nullptr && wide && valid >= 8) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w + col));
    const float4 b = __ldg(reinterpret_cast<const float4*>(w + col) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = w != nullptr && j < valid ? __ldg(w + col + j) : none;
  }
}

// ------------------------------------------------------------------ dropout

constexpr int DO_THREADS = 256;
constexpr int DO_BLOCKS = 4;   // resident per SM
constexpr int DO_UNROLL = 4;   // groups of a thread in flight

struct DropoutParams {
  int32_t N, groups;  // groups of 8 columns per row
  int64_t total;      // rows * groups
  int64_t step_rows;  // gridDim.x * DO_THREADS groups further on: rows and groups
  int32_t step_groups;
  const void* x;
  int64_t ld_x;
  const void* residual;  // or NULL
  int64_t ld_residual;
  void* y;
  int64_t ld_y;
  int32_t wide_in, wide_out;
  Dropout drop;
};

template <class T>
__global__ void __launch_bounds__(DO_THREADS, DO_BLOCKS) dropout_kernel(const __grid_constant__ DropoutParams p) {
  int64_t i = static_cast<int64_t>(blockIdx.x) * DO_THREADS + threadIdx.x;
  if (i >= p.total) return;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * DO_THREADS;
  int64_t row = i / p.groups;
  int32_t group = static_cast<int32_t>(i - row * p.groups);
  const bool drops = p.drop.state != nullptr;
  const DropKey key = drops ? drop_key(p.drop) : DropKey{};
  while (i < p.total) {
    int64_t rows[DO_UNROLL];
    int32_t at[DO_UNROLL];
    float x[DO_UNROLL][8], r[DO_UNROLL][8];
#pragma unroll
    for (int u = 0; u < DO_UNROLL; ++u) {
      rows[u] = row, at[u] = group;
      if (i + u * stride < p.total) {
        const int col = group * 8;
        load_group(static_cast<const T*>(p.x) + row * p.ld_x + col, p.N - col, p.wide_in, x[u]);
        if (p.residual != nullptr)
          load_group(static_cast<const T*>(p.residual) + row * p.ld_residual + col, p.N - col, p.wide_in, r[u]);
      }
      row += p.step_rows, group += p.step_groups;
      if (group >= p.groups) group -= p.groups, ++row;
    }
#pragma unroll
    for (int u = 0; u < DO_UNROLL; ++u) {
      if (i + u * stride >= p.total) break;
      uint32_t w[4];
      if (drops) drop_words(key, static_cast<uint32_t>(rows[u]), static_cast<uint32_t>(at[u]), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float add = p.residual != nullptr ? r[u][j] : 0.0f;
        x[u][j] = !drops ? x[u][j] + add : drop_keeps(w, j, p.drop.above) ? fmaf(x[u][j], p.drop.scale, add) : add;
      }
      const int col = at[u] * 8;
      store_group(static_cast<T*>(p.y) + rows[u] * p.ld_y + col, p.N - col, p.wide_out, x[u]);
    }
    i += DO_UNROLL * stride;
  }
}

// ------------------------------------------------------------------ teams

// Rows the ring holds for each thread.
template <class T, int K>
constexpr int LN_DEPTH = sizeof(T) == 4 && K == 4 ? 1 : 2;
constexpr int LN_MAX_WARPS = 16;
constexpr int LN_WARP_TEAMS = 8;  // warps of a block whose teams are within a warp
constexpr int LN_MAX_GROUPS = LN_MAX_WARPS * 32 * 4;  // wider rows run on the re-reading kernels

struct NormParams {
  int32_t M, N, groups;
  int32_t log_lanes;  // teams within a warp: 2^log_lanes threads each
  const void* x;      // backward: h, the forward pass's normalised sum
  int64_t ld_x;
  const void* other;  // residual; backward: dy
  int64_t ld_other;
  const void* add;    // backward only; or NULL
  int64_t ld_add;
  void* y;            // backward: dx; or NULL
  int64_t ld_y;
  void* sum;          // h; backward: d_residual; or NULL
  int64_t ld_sum;
  const float* w;
  const float* b;
  float* mean;  // outputs; backward: read
  float* rstd;
  float* partials;    // backward: [blocks][2][N], dw and db; or NULL
  float eps, inv_n;
  int32_t wide_in, wide_out, wide_w;
  Dropout drop;
};

// Copies of a thread's groups of the next rows on their way into its slots.
template <class T, int K, int TENSORS>
struct RowRing {
  static constexpr int PIECES = Group<T>::PIECES;
  static constexpr int DEPTH = LN_DEPTH<T, K>;
  static constexpr int bytes(int threads) { return DEPTH * TENSORS * K * PIECES * threads * 16; }

  const uint4* slots;  // this thread's column of the block's slots
  uint32_t at;
  int threads;

  __device__ __forceinline__ RowRing(const uint4* smem, int tid, int threads_)
      : slots(smem + tid), at(ptx::smem_addr(smem + tid)), threads(threads_) {}
  __device__ __forceinline__ int index(int d, int t, int k, int piece) const {
    return (((d * TENSORS + t) * K + k) * PIECES + piece) * threads;
  }
  // The first `valid` of 8 values at p, which starts on 16 bytes.
  __device__ __forceinline__ void fetch(int d, int t, int k, const T* p, int valid) const {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      constexpr int EACH = 8 / PIECES;
      const int n = min(max(valid - i * EACH, 0), EACH);
      ptx::cp_async16(at + static_cast<uint32_t>(index(d, t, k, i)) * 16u, n > 0 ? p + i * EACH : p,
                      static_cast<uint32_t>(n) * sizeof(T));
    }
  }
  __device__ __forceinline__ void take(int d, int t, int k, float (&v)[8]) const {
    Group<T> g;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) g.q[i] = slots[index(d, t, k, i)];
    g.unpack(v);
  }
};

// Sum over the 2^log_lanes lanes of a team within a warp.
__device__ __forceinline__ float team_sum(float v, int log_lanes) {
#pragma unroll
  for (int g = 4; g >= 0; --g)
    if (g < log_lanes) v += __shfl_xor_sync(0xffffffffu, v, 1 << g);
  return v;
}

__device__ __forceinline__ float warp_sum(float v) { return team_sum(v, 5); }

// Sum of (v - m)^2 over the thread's values inside the row.
template <int K>
__device__ __forceinline__ float squares_from(const float (&v)[K][8], const int (&valid)[K], float m) {
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (valid[k] >= 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(v[k][j] - m, v[k][j] - m, s);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid[k]) s = fmaf(v[k][j] - m, v[k][j] - m, s);
    }
  }
  return s;
}

// A thread's place: its team's rows and its groups of columns.
template <int K, bool BLOCK>
struct TeamPlace {
  int tid;             // within the team
  int64_t row, stride; // first row of the team, and to the next
  int64_t leader;      // the loop's row: the same for all threads that share a barrier or a shuffle
  int col[K], valid[K];

  __device__ __forceinline__ explicit TeamPlace(const NormParams& p) {
    const int lanes = BLOCK ? blockDim.x : 1 << p.log_lanes;
    tid = threadIdx.x & (BLOCK ? ~0 : lanes - 1);
    if (BLOCK) {
      row = leader = blockIdx.x;
      stride = gridDim.x;
    } else {
      const int teams = 32 >> p.log_lanes;  // of a warp
      const int64_t warp = static_cast<int64_t>(blockIdx.x) * LN_WARP_TEAMS + (threadIdx.x >> 5);
      leader = warp * teams;
      row = leader + ((threadIdx.x & 31) >> p.log_lanes);
      stride = static_cast<int64_t>(gridDim.x) * LN_WARP_TEAMS * teams;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int g = tid + k * lanes;
      valid[k] = g < p.groups ? min(8, p.N - g * 8) : 0;
      col[k] = g < p.groups ? g * 8 : 0;
    }
  }
};

// ------------------------------------------------------------------ forward

template <class T, bool DROP, int K, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 32 * LN_MAX_WARPS : 32 * LN_WARP_TEAMS)
    layer_norm_kernel(const __grid_constant__ NormParams p) {
  using Ring = RowRing<T, K, 2>;
  extern __shared__ uint4 ln_smem[];
  __shared__ float4 part[2][LN_MAX_WARPS];  // a warp's mean, sum of squares from it, count
  const TeamPlace<K, BLOCK> place(p);
  const Ring ring(ln_smem, threadIdx.x, blockDim.x);
  const T* x = static_cast<const T*>(p.x);
  const T* residual = static_cast<const T*>(p.other);

  auto fetch = [&](int d, int64_t row) {
    if (p.wide_in && row < p.M) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (place.valid[k] == 0) continue;
        ring.fetch(d, 0, k, x + row * p.ld_x + place.col[k], place.valid[k]);
        if (residual != nullptr) ring.fetch(d, 1, k, residual + row * p.ld_other + place.col[k], place.valid[k]);
      }
    }
    ptx::cp_async_commit();
  };
#pragma unroll
  for (int d = 0; d < Ring::DEPTH; ++d) fetch(d, place.row + d * place.stride);

  DropKey key{};
  if constexpr (DROP) key = drop_key(p.drop);
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  float count = 0.0f, inv_count = 0.0f;  // BLOCK: values of this warp
  if constexpr (BLOCK) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) n += min(max(p.N - 8 * (warp * 32 + k * static_cast<int>(blockDim.x)), 0), 256);
    count = static_cast<float>(n);
    inv_count = n > 0 ? 1.0f / count : 0.0f;
  }

  int d = 0, parity = 0;
  int64_t row = place.row;
  for (int64_t at = place.leader; at < p.M; at += place.stride, row += place.stride) {
    const bool ok = BLOCK || row < p.M;
    ptx::cp_async_wait<Ring::DEPTH - 1>();
    float h[K][8];
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[k][j] = r[j] = 0.0f;
      if (ok && place.valid[k] > 0) {
        if (p.wide_in) {
          ring.take(d, 0, k, h[k]);
          if (residual != nullptr) ring.take(d, 1, k, r);
        } else {
          load_group(x + row * p.ld_x + place.col[k], place.valid[k], false, h[k]);
          if (residual != nullptr)
            load_group(residual + row * p.ld_other + place.col[k], place.valid[k], false, r);
        }
      }
      if constexpr (DROP) {
        uint32_t w[4];
        drop_words(key, static_cast<uint32_t>(row), static_cast<uint32_t>(place.col[k] >> 3), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[k][j] = drop_keeps(w, j, p.drop.above) ? fmaf(h[k][j], p.drop.scale, r[j]) : r[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[k][j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s += h[k][j];
    }
    // The slot's values are in registers.
    fetch(d, row + Ring::DEPTH * place.stride);
    d = d + 1 == Ring::DEPTH ? 0 : d + 1;

    float mean, square;  // sum of squares from the mean
    if constexpr (BLOCK) {
      const float m = warp_sum(s) * inv_count;
      const float q = warp_sum(squares_from(h, place.valid, m));
      if ((threadIdx.x & 31) == 0) part[parity][warp] = make_float4(m, q, count, 0.0f);
      __syncthreads();  // the other buffer is read before the next row's barrier
      // Sums of the warps' means and squares, both from the first warp's mean.
      const float4 first = part[parity][0];
      float shift = 0.0f;
      square = first.y;
      for (int i = 1; i < warps; ++i) {
        const float4 v = part[parity][i];
        const float delta = v.x - first.x;
        shift = fmaf(v.z, delta, shift);
        square += fmaf(v.z * delta, delta, v.y);
      }
      shift *= p.inv_n;
      mean = first.x + shift;
      square = fmaf(-shift * shift, static_cast<float>(p.N), square);
      square = square < 0.0f ? 0.0f : square;  // a NaN stays
      parity ^= 1;
    } else {
      mean = team_sum(s, p.log_lanes) * p.inv_n;
      square = team_sum(squares_from(h, place.valid, mean), p.log_lanes);
    }
    const float rstd = 1.0f / sqrtf(fmaf(square, p.inv_n, p.eps));
    if (!ok) continue;
    if (place.tid == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (place.valid[k] == 0) continue;
      if (p.sum != nullptr)
        store_group(static_cast<T*>(p.sum) + row * p.ld_sum + place.col[k], place.valid[k], p.wide_out, h[k]);
      float w[8], b[8];
      load_weights(p.w, place.col[k], place.valid[k], p.wide_w, 1.0f, w);
      load_weights(p.b, place.col[k], place.valid[k], p.wide_w, 0.0f, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = fmaf((h[k][j] - mean) * rstd, w[j], b[j]);
      store_group(static_cast<T*>(p.y) + row * p.ld_y + place.col[k], place.valid[k], p.wide_out, w);
    }
  }
  ptx::cp_async_wait<0>();
}

// ------------------------------------------------------------------ backward

template <class T, bool DROP, int K, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? (K == 1 ? 256 : 512) : 32 * LN_WARP_TEAMS)
    layer_norm_backward_kernel(const __grid_constant__ NormParams p) {
  using Ring = RowRing<T, K, 3>;
  extern __shared__ uint4 ln_smem[];
  __shared__ float2 part[2][LN_MAX_WARPS];  // a warp's sums of a and a n
  const TeamPlace<K, BLOCK> place(p);
  const Ring ring(ln_smem, threadIdx.x, blockDim.x);
  const T* x = static_cast<const T*>(p.x);
  const T* dy = static_cast<const T*>(p.other);
  const T* add = static_cast<const T*>(p.add);
  const bool wants_g = p.y != nullptr || p.sum != nullptr;

  auto fetch = [&](int d, int64_t row) {
    if (p.wide_in && row < p.M) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (place.valid[k] == 0) continue;
        ring.fetch(d, 0, k, dy + row * p.ld_other + place.col[k], place.valid[k]);
        ring.fetch(d, 1, k, x + row * p.ld_x + place.col[k], place.valid[k]);
        if (add != nullptr) ring.fetch(d, 2, k, add + row * p.ld_add + place.col[k], place.valid[k]);
      }
    }
    ptx::cp_async_commit();
  };
#pragma unroll
  for (int d = 0; d < Ring::DEPTH; ++d) fetch(d, place.row + d * place.stride);

  DropKey key{};
  if constexpr (DROP) key = drop_key(p.drop);
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  float dw[K][8], db[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[k][j] = db[k][j] = 0.0f;

  // dy and x of group k of a row, zeros outside it.
  auto take = [&](int d, int64_t row, bool ok, int k, float (&g)[8], float (&h)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = h[j] = 0.0f;
    if (!ok || place.valid[k] == 0) return;
    if (p.wide_in) {
      ring.take(d, 0, k, g);
      ring.take(d, 1, k, h);
    } else {
      load_group(dy + row * p.ld_other + place.col[k], place.valid[k], false, g);
      load_group(x + row * p.ld_x + place.col[k], place.valid[k], false, h);
    }
  };

  int d = 0, parity = 0;
  int64_t row = place.row;
  for (int64_t at = place.leader; at < p.M; at += place.stride, row += place.stride) {
    const bool ok = BLOCK || row < p.M;
    const float mean = ok ? __ldg(p.mean + row) : 0.0f, rstd = ok ? __ldg(p.rstd + row) : 0.0f;
    ptx::cp_async_wait<Ring::DEPTH - 1>();
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float g[8], n[8], w[8];
      take(d, row, ok, k, g, n);
      load_weights(p.w, place.col[k], place.valid[k], p.wide_w, 1.0f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[j] = (n[j] - mean) * rstd;
        dw[k][j] = fmaf(g[j], n[j], dw[k][j]);
        db[k][j] += g[j];
        const float a = g[j] * w[j];
        s1 += a;
        s2 = fmaf(a, n[j], s2);
      }
    }
    if (wants_g) {
      if constexpr (BLOCK) {
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if ((threadIdx.x & 31) == 0) part[parity][warp] = make_float2(s1, s2);
        __syncthreads();  // the other buffer is read before the next row's barrier
        s1 = s2 = 0.0f;
        for (int i = 0; i < warps; ++i) {
          const float2 v = part[parity][i];
          s1 += v.x;
          s2 += v.y;
        }
        parity ^= 1;
      } else {
        s1 = team_sum(s1, p.log_lanes);
        s2 = team_sum(s2, p.log_lanes);
      }
      s1 *= p.inv_n;
      s2 *= p.inv_n;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!ok || place.valid[k] == 0) continue;
        float g[8], n[8], w[8];
        take(d, row, ok, k, g, n);
        load_weights(p.w, place.col[k], place.valid[k], p.wide_w, 1.0f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          n[j] = (n[j] - mean) * rstd;
          g[j] = rstd * (fmaf(g[j], w[j], -s1) - n[j] * s2);
        }
        if (add != nullptr) {
          if (p.wide_in)
            ring.take(d, 2, k, w);
          else
            load_group(add + row * p.ld_add + place.col[k], place.valid[k], false, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] += w[j];
        }
        if (p.sum != nullptr)
          store_group(static_cast<T*>(p.sum) + row * p.ld_sum + place.col[k], place.valid[k], p.wide_out, g);
        if (p.y != nullptr) {
          if constexpr (DROP)
            drop8(p.drop, key, static_cast<uint32_t>(row), static_cast<uint32_t>(place.col[k] >> 3), g);
          store_group(static_cast<T*>(p.y) + row * p.ld_y + place.col[k], place.valid[k], p.wide_out, g);
        }
      }
    }
    fetch(d, row + Ring::DEPTH * place.stride);
    d = d + 1 == Ring::DEPTH ? 0 : d + 1;
  }
  ptx::cp_async_wait<0>();
  if (p.partials == nullptr) return;
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.N;
  if constexpr (BLOCK) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < place.valid[k]) {
          out[place.col[k] + j] = dw[k][j];
          out[p.N + place.col[k] + j] = db[k][j];
        }
  } else {
    // A warp's teams by shuffles, then the warps in shared memory: [warp][dw, db][column].
    float* sums = reinterpret_cast<float*>(ln_smem);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        for (int s = 1 << p.log_lanes; s < 32; s <<= 1) {
          dw[k][j] += __shfl_xor_sync(0xffffffffu, dw[k][j], s);
          db[k][j] += __shfl_xor_sync(0xffffffffu, db[k][j], s);
        }
        if ((threadIdx.x & 31) == place.tid && j < place.valid[k]) {
          sums[(warp * 2) * p.N + place.col[k] + j] = dw[k][j];
          sums[(warp * 2 + 1) * p.N + place.col[k] + j] = db[k][j];
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.N; i += blockDim.x) {
      float t = 0.0f;
#pragma unroll
      for (int v = 0; v < LN_WARP_TEAMS; ++v) t += sums[v * 2 * p.N + i];
      out[i] = t;
    }
  }
}

// dw (blockIdx.y 0) and db (1): the sum of the blocks' partial sums in a fixed order.
__global__ void __launch_bounds__(1024) layer_norm_weight_grad_kernel(const float* partials, int blocks, int N, float* dw,
                                                                      float* db) {
  __shared__ float part[32][33];
  ptx::wait_dependencies();  // launched beside the backward kernel's end
  const int col = blockIdx.x * 32 + threadIdx.x;
  float* dst = blockIdx.y == 0 ? dw : db;
  if (dst == nullptr) return;
  float sum = 0.0f;
  if (col < N)
    for (int r = threadIdx.y; r < blocks; r += 32) sum += partials[(static_cast<int64_t>(r) * 2 + blockIdx.y) * N + col];
  part[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0 && col < N) {
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < 32; ++r) t += part[r][threadIdx.x];
    dst[col] = t;
  }
}

// ------------------------------------------------------------------ rows too wide to hold

// A block to a row, which it reads three times (forward) or twice (backward):
// the second time from L2.
constexpr int LN_LONG_THREADS = 512;

// Sum over the block, in every thread.
__device__ __forceinline__ float block_sum(float v, float (&part)[LN_LONG_THREADS / 32]) {
  v = warp_sum(v);
  __syncthreads();  // the previous sum's reads
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < LN_LONG_THREADS / 32; ++i) t += part[i];
  return t;
}

template <class T, bool DROP>
__global__ void __launch_bounds__(LN_LONG_THREADS) layer_norm_long_kernel(const __grid_constant__ NormParams p) {
  __shared__ float part[LN_LONG_THREADS / 32];
  DropKey key{};
  if constexpr (DROP) key = drop_key(p.drop);
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    auto load = [&](int g, float (&h)[8]) {
      load_group(static_cast<const T*>(p.x) + row * p.ld_x + g * 8, p.N - g * 8, p.wide_in, h);
      float r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = 0.0f;
      if (p.other != nullptr)
        load_group(static_cast<const T*>(p.other) + row * p.ld_other + g * 8, p.N - g * 8, p.wide_in, r);
      if constexpr (DROP) {
        uint32_t w[4];
        drop_words(key, static_cast<uint32_t>(row), static_cast<uint32_t>(g), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = drop_keeps(w, j, p.drop.above) ? fmaf(h[j], p.drop.scale, r[j]) : r[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] += r[j];
      }
    };
    float s = 0.0f;
    for (int g = threadIdx.x; g < p.groups; g += LN_LONG_THREADS) {
      float h[8];
      load(g, h);  // zeros behind the row's end
#pragma unroll
      for (int j = 0; j < 8; ++j) s += h[j];
    }
    const float mean = block_sum(s, part) * p.inv_n;
    s = 0.0f;
    for (int g = threadIdx.x; g < p.groups; g += LN_LONG_THREADS) {
      float h[1][8];
      load(g, h[0]);
      const int valid[1] = {p.N - g * 8};
      s += squares_from(h, valid, mean);
    }
    const float rstd = 1.0f / sqrtf(fmaf(block_sum(s, part), p.inv_n, p.eps));
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    for (int g = threadIdx.x; g < p.groups; g += LN_LONG_THREADS) {
      const int valid = p.N - g * 8;
      float h[8], w[8], b[8];
      load(g, h);
      if (p.sum != nullptr) store_group(static_cast<T*>(p.sum) + row * p.ld_sum + g * 8, valid, p.wide_out, h);
      load_weights(p.w, g * 8, valid, p.wide_w, 1.0f, w);
      load_weights(p.b, g * 8, valid, p.wide_w, 0.0f, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = fmaf((h[j] - mean) * rstd, w[j], b[j]);
      store_group(static_cast<T*>(p.y) + row * p.ld_y + g * 8, valid, p.wide_out, w);
    }
  }
}

// The sums over rows are kept in the block's partials themselves, each column
// by the thread that works on it in every row.
template <class T, bool DROP>
__global__ void __launch_bounds__(LN_LONG_THREADS) layer_norm_backward_long_kernel(const __grid_constant__ NormParams p) {
  __shared__ float part[LN_LONG_THREADS / 32];
  DropKey key{};
  if constexpr (DROP) key = drop_key(p.drop);
  float* sums = p.partials == nullptr ? nullptr : p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.N;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
    auto load = [&](int g, float (&dy)[8], float (&n)[8]) {
      load_group(static_cast<const T*>(p.other) + row * p.ld_other + g * 8, p.N - g * 8, p.wide_in, dy);
      load_group(static_cast<const T*>(p.x) + row * p.ld_x + g * 8, p.N - g * 8, p.wide_in, n);
#pragma unroll
      for (int j = 0; j < 8; ++j) n[j] = (n[j] - mean) * rstd;
    };
    float s1 = 0.0f, s2 = 0.0f;
    for (int g = threadIdx.x; g < p.groups; g += LN_LONG_THREADS) {
      const int valid = p.N - g * 8;
      float dy[8], n[8], w[8];
      load(g, dy, n);
      load_weights(p.w, g * 8, valid, p.wide_w, 1.0f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = dy[j] * w[j];
        s1 += a;
        s2 = fmaf(a, n[j], s2);
        if (sums != nullptr && j < valid) {
          const int c = g * 8 + j;
          const bool first = row == blockIdx.x;
          float& db = sums[static_cast<int64_t>(p.N) + c];
          sums[c] = first ? dy[j] * n[j] : fmaf(dy[j], n[j], sums[c]);
          db = first ? dy[j] : db + dy[j];
        }
      }
    }
    if (p.y == nullptr && p.sum == nullptr) continue;
    s1 = block_sum(s1, part) * p.inv_n;
    s2 = block_sum(s2, part) * p.inv_n;
    for (int g = threadIdx.x; g < p.groups; g += LN_LONG_THREADS) {
      const int valid = p.N - g * 8;
      float dy[8], n[8], w[8];
      load(g, dy, n);
      load_weights(p.w, g * 8, valid, p.wide_w, 1.0f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) dy[j] = rstd * (fmaf(dy[j], w[j], -s1) - n[j] * s2);
      if (p.add != nullptr) {
        load_group(static_cast<const T*>(p.add) + row * p.ld_add + g * 8, valid, p.wide_in, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) dy[j] += w[j];
      }
      if (p.sum != nullptr) store_group(static_cast<T*>(p.sum) + row * p.ld_sum + g * 8, valid, p.wide_out, dy);
      if (p.y != nullptr) {
        if constexpr (DROP) drop8(p.drop, key, static_cast<uint32_t>(row), static_cast<uint32_t>(g), dy);
        store_group(static_cast<T*>(p.y) + row * p.ld_y + g * 8, valid, p.wide_out, dy);
      }
    }
  }
}

}  // namespace ge
