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

#include <utility>

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
  __device__ __forceinline__ void clear() { q[0] = make_uint4(0, 0, 0, 0); }
  // The first `valid` (up to 8) values at p, zeros behind them.  `wide`: p is on 16 bytes.
  __device__ __forceinline__ void load(const uint16_t* p, int valid, bool wide) {
    if (wide && valid >= 8) {
      q[0] = *reinterpret_cast<const uint4*>(p);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int h = 0; h < 4; ++h)
        w[h] = (2 * h < valid ? static_cast<uint32_t>(p[2 * h]) : 0u) |
               (2 * h + 1 < valid ? static_cast<uint32_t>(p[2 * h + 1]) << 16 : 0u);
      q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
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
  __device__ __forceinline__ void clear() { q[0] = q[1] = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const float* p, int valid, bool wide) {
    if (wide && valid >= 8) {
      q[0] = reinterpret_cast<const uint4*>(p)[0];
      q[1] = reinterpret_cast<const uint4*>(p)[1];
    } else {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < valid ? p[j] : 0.0f;
      pack(v);
    }
  }
  static __device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
};

template <class T>
__device__ __forceinline__ void load_group(const T* p, int valid, bool wide, float (&v)[8]) {
  Group<T> g;
  g.load(p, valid, wide);
  g.unpack(v);
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

// Eight fp32 values of a thread, two to a register pair.
struct Eight {
  float2 v[4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(0.0f, 0.0f);
  }
  __device__ __forceinline__ void from(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ void to(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = v[i].x, f[2 * i + 1] = v[i].y;
  }
  template <class T>
  __device__ __forceinline__ void from(const Group<T>& g) {
    float f[8];
    g.unpack(f);
    from(f);
  }
  template <class T>
  __device__ __forceinline__ void load(const T* p, int valid, bool wide) {
    Group<T> g;
    g.load(p, valid, wide);
    from(g);
  }
  __device__ __forceinline__ void plus(const Eight& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __fadd2_rn(v[i], r.v[i]);
  }
  template <class T>
  __device__ __forceinline__ void store(T* p, int valid, bool wide) const {
    float f[8];
    to(f);
    store_group(p, valid, wide, f);
  }
  __device__ __forceinline__ void weights(const float* w, int col, int valid, bool wide, float none) {
    float f[8];
    load_weights(w, col, valid, wide, none, f);
    from(f);
  }
  // D(this) + r
  __device__ __forceinline__ void drop_onto(const Eight& r, const Dropout& d, const uint32_t (&w)[4]) {
    const float2 scale = make_float2(d.scale, d.scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 kept = __ffma2_rn(v[i], scale, r.v[i]);
      v[i].x = drop_keeps(w, 2 * i, d.above) ? kept.x : r.v[i].x;
      v[i].y = drop_keeps(w, 2 * i + 1, d.above) ? kept.y : r.v[i].y;
    }
  }
  __device__ __forceinline__ void drop(const Dropout& d, const uint32_t (&w)[4]) {
    const float2 scale = make_float2(d.scale, d.scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 kept = __fmul2_rn(v[i], scale);
      v[i].x = drop_keeps(w, 2 * i, d.above) ? kept.x : 0.0f;
      v[i].y = drop_keeps(w, 2 * i + 1, d.above) ? kept.y : 0.0f;
    }
  }
  __device__ __forceinline__ float2 sum() const {
    return __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3]));
  }
  // Sum of (v - m)^2 over the first `valid`.
  __device__ __forceinline__ float2 squares(float m) const {
    const float2 minus = make_float2(-m, -m);
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 c = __fadd2_rn(v[i], minus);
      s = __ffma2_rn(c, c, s);
    }
    return s;
  }
  __device__ __forceinline__ float squares(float m, int valid) const {
    float f[8], s = 0.0f;
    to(f);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) s = fmaf(f[j] - m, f[j] - m, s);
    return s;
  }
  // (this - mean) rstd
  __device__ __forceinline__ void normalise(float mean, float rstd) {
    const float2 minus = make_float2(-mean, -mean), r = make_float2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __fmul2_rn(__fadd2_rn(v[i], minus), r);
  }
};

__device__ __forceinline__ float2 fma2(const float2 a, float b, const float2 c) {
  return __ffma2_rn(a, make_float2(b, b), c);
}

// ------------------------------------------------------------------ dropout

constexpr int DO_THREADS = 256;
constexpr int DO_BLOCKS = 3;  // resident per SM
template <class T>
constexpr int DO_UNROLL = 8 / sizeof(T);  // groups of a thread in flight

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
  constexpr int U = DO_UNROLL<T>;
  int64_t i = static_cast<int64_t>(blockIdx.x) * DO_THREADS + threadIdx.x;
  if (i >= p.total) return;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * DO_THREADS;
  int64_t row = i / p.groups;
  int32_t group = static_cast<int32_t>(i - row * p.groups);
  const bool drops = p.drop.step != nullptr;
  const uint32_t step = drops ? drop_step(p.drop) : 0;
  while (i < p.total) {
    uint32_t rows[U], groups[U];
    Group<T> x[U], r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rows[u] = static_cast<uint32_t>(row), groups[u] = static_cast<uint32_t>(group);
      x[u].clear();
      r[u].clear();
      if (i + u * stride < p.total) {
        const int col = group * 8;
        x[u].load(static_cast<const T*>(p.x) + row * p.ld_x + col, p.N - col, p.wide_in);
        if (p.residual != nullptr)
          r[u].load(static_cast<const T*>(p.residual) + row * p.ld_residual + col, p.N - col, p.wide_in);
      }
      row += p.step_rows, group += p.step_groups;
      if (group >= p.groups) group -= p.groups, ++row;
    }
    uint32_t words[U][4];
    if (drops) drop_words(p.drop, step, rows, groups, words);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Eight v, add;
      v.from(x[u]);
      add.from(r[u]);
      if (drops)
        v.drop_onto(add, p.drop, words[u]);
      else
        v.plus(add);
      const int col = static_cast<int>(groups[u]) * 8;
      if (i + u * stride < p.total) v.store(static_cast<T*>(p.y) + rows[u] * p.ld_y + col, p.N - col, p.wide_out);
    }
    i += U * stride;
  }
}

// ------------------------------------------------------------------ teams

// A team of W warps holds a row: warp i the columns from i K 256 on, lane l in
// each of its K pieces of 256 columns the 8 from 8 l.  The offsets between
// pieces are constants, and what a row costs a thread beside its values (its
// sums' shuffles, the barrier, the addresses) is spread over 8 K of them.
constexpr int LN_PIECE = 256;
constexpr int LN_MAX_WARPS = 16;
constexpr int LN_BLOCK_WARPS = 8;  // of blocks that hold several teams
constexpr int LN_MAX_SHARED = 224 * 1024;  // of the 227 KB of a block, beside what is not dynamic

struct NormParams {
  int32_t M, N, groups;
  int32_t warps;      // of a team
  int32_t staged;     // the norm's weights go through shared memory
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
  Dropout drop;
};

// Sum over the 2^log_lanes lanes of a team within a warp.
__device__ __forceinline__ float team_sum(float v, int log_lanes) {
#pragma unroll
  for (int g = 4; g >= 0; --g)
    if (g < log_lanes) v += __shfl_xor_sync(0xffffffffu, v, 1 << g);
  return v;
}

__device__ __forceinline__ float warp_sum(float v) { return team_sum(v, 5); }

// Rows of a thread that the backward pass's ring holds.
template <class T>
constexpr int LN_BACKWARD_DEPTH = sizeof(T) == 2 ? 2 : 1;

// A barrier of one team of several.
__device__ __forceinline__ void team_sync(int team, int warps) {
  if (warps > 1) ptx::named_barrier_sync(team + 1, warps * 32);
}

// A thread's columns in its team's rows, and those it copies into the ring:
// with fp32 two pieces of 16 bytes 128 columns apart, so that a warp's copy
// takes whole sectors.
template <class T, int K>
struct RowPlace {
  static constexpr int EACH = 16 / sizeof(T);  // columns of 16 bytes
  int col;   // of piece 0; piece k: LN_PIECE k further on
  int left;  // columns from `col` to the row's end (<= 0: none)
  int copy_col, copy_left;
  bool full;  // all of the warp's columns are in the row

  __device__ __forceinline__ RowPlace(const NormParams& p, int warp_in_team) {
    const int begin = warp_in_team * K * LN_PIECE, lane = threadIdx.x & 31;
    col = begin + lane * 8;
    left = p.N - col;
    copy_col = begin + lane * EACH;
    copy_left = p.N - copy_col;
    full = begin + K * LN_PIECE <= p.N;
  }
  __device__ __forceinline__ int valid(int k) const { return min(left - k * LN_PIECE, 8); }
  // of the i-th 16 bytes that the thread copies of piece k
  __device__ __forceinline__ int copied(int k, int i) const {
    return min(copy_left - k * LN_PIECE - i * (LN_PIECE / 2), EACH);
  }
};

// Copies of a warp's values of the next rows on their way into its slots, 16
// bytes of each lane side by side.  bf16: each thread copies what it reads.
// fp32: 16 bytes j of a piece are part j % 2 of lane j / 2, so a __syncwarp()
// lies between the copies' end and the reads, and the reads and the next copies.
template <class T, int K, int TENSORS, int DEPTH>
struct RowRing {
  static constexpr int PARTS = Group<T>::PIECES;  // of 16 bytes
  static constexpr int WARP_BYTES = DEPTH * TENSORS * K * PARTS * 512;
  const uint4* slots;  // this thread's first to read
  uint4* to;           // and to fill
  uint32_t at;

  __device__ __forceinline__ RowRing(uint4* smem, int warp) {
    const int lane = threadIdx.x & 31;
    smem += warp * (WARP_BYTES / 16);
    slots = smem + lane;
    to = smem + (PARTS == 1 ? lane : (lane & 1) * 32 + (lane >> 1));
    at = ptx::smem_addr(to);
  }
  static __device__ __forceinline__ constexpr int read_index(int d, int t, int k, int part) {
    return (((d * TENSORS + t) * K + k) * PARTS + part) * 32;
  }
  static __device__ __forceinline__ constexpr int fill_index(int d, int t, int k, int i) {
    return ((d * TENSORS + t) * K + k) * PARTS * 32 + i * 16;
  }
  static __device__ __forceinline__ void sync() {
    if (PARTS > 1) __syncwarp();
  }
  // Zeros where no copy will land.
  __device__ __forceinline__ void clear(const RowPlace<T, K>& place, int first_unused_tensor) const {
#pragma unroll 1
    for (int d = 0; d < DEPTH; ++d)
      for (int t = 0; t < TENSORS; ++t)
        for (int k = 0; k < K; ++k)
          for (int i = 0; i < PARTS; ++i)
            if (t >= first_unused_tensor || place.copied(k, i) <= 0) to[fill_index(d, t, k, i)] = make_uint4(0, 0, 0, 0);
  }
  template <int... Is>
  static __device__ __forceinline__ void fetch_full(uint32_t to, const T* row, std::integer_sequence<int, Is...>) {
    (ptx::cp_async16<fill_index(0, 0, Is / PARTS, Is % PARTS) * 16,
                     (Is / PARTS * LN_PIECE + Is % PARTS * (LN_PIECE / 2)) * static_cast<int>(sizeof(T))>(to, row), ...);
  }
  // `row`: at the first column that the thread copies.
  __device__ __forceinline__ void fetch(int d, int t, const T* row, const RowPlace<T, K>& place) const {
    const uint32_t first = at + static_cast<uint32_t>(fill_index(d, t, 0, 0)) * 16u;
    if (place.full) {
      fetch_full(first, row, std::make_integer_sequence<int, K * PARTS>{});
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < PARTS; ++i)
          if (place.copied(k, i) > 0)
            ptx::cp_async16(first + static_cast<uint32_t>(fill_index(0, 0, k, i)) * 16u,
                            row + k * LN_PIECE + i * (LN_PIECE / 2), static_cast<uint32_t>(place.copied(k, i)) * sizeof(T));
    }
  }
  __device__ __forceinline__ void take(int d, int t, int k, Eight& v) const {
    Group<T> g;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) g.q[i] = slots[read_index(d, t, k, i)];
    v.from(g);
  }
};

// A block's teams, and where its shared memory's parts begin: the ring, then
// the norm's weights.
template <int K>
struct Teams {
  int warp, team, count;  // of the thread; of the block
  int width;              // columns of a team's warps
  int64_t first, stride;  // rows of the team

  __device__ __forceinline__ explicit Teams(const NormParams& p)
      : warp(threadIdx.x >> 5), team(warp / p.warps), count((blockDim.x >> 5) / p.warps), width(p.warps * K * LN_PIECE),
        first(static_cast<int64_t>(blockIdx.x) * count + team), stride(static_cast<int64_t>(gridDim.x) * count) {}
  __device__ __forceinline__ int warp_in_team(const NormParams& p) const { return warp - team * p.warps; }
};

// Weights in shared memory, by all threads of the block: a row's cost is then
// free of the L1 misses that its streams cause.  A piece's 256 lie as the first
// halves of its lanes' groups and then the second ones, so that 16-byte reads
// meet no bank twice.  A barrier has to follow.
__device__ __forceinline__ void stage_weights(float* to, const float* w, int n, int width, float none) {
  for (int i = threadIdx.x; i < width; i += blockDim.x) {
    const int col = (i & ~(LN_PIECE - 1)) + (i >> 2 & 31) * 8 + (i >> 7 & 1) * 4 + (i & 3);
    to[i] = w != nullptr && col < n ? __ldg(w + col) : none;
  }
}

// w: the thread's first half of piece 0, i.e. its warp's first column + 4 lane.
__device__ __forceinline__ void staged_weights(const float* w, int k, Eight& v) {
  const float4 a = *reinterpret_cast<const float4*>(w + k * LN_PIECE);
  const float4 b = *reinterpret_cast<const float4*>(w + k * LN_PIECE + LN_PIECE / 2);
  v.v[0] = make_float2(a.x, a.y), v.v[1] = make_float2(a.z, a.w);
  v.v[2] = make_float2(b.x, b.y), v.v[3] = make_float2(b.z, b.w);
}

// The words of B of a thread's groups of a row, the first one at column `col`.
template <int B>
__device__ __forceinline__ void row_words(const Dropout& d, uint32_t step, uint32_t row, int col, uint32_t (&words)[B][4]) {
  uint32_t rows[B], groups[B];
#pragma unroll
  for (int i = 0; i < B; ++i) rows[i] = row, groups[i] = static_cast<uint32_t>(col + i * LN_PIECE) >> 3;
  drop_words(d, step, rows, groups, words);
}

// ------------------------------------------------------------------ forward

// A team works on R neighbouring rows at once: they share the weights' reads,
// and their sums' shuffles and the barrier overlap.  WIDE: every tensor takes
// 16-byte accesses, and its rows come through the ring (with a depth of 1: rows
// are in registers while the next ones are on their way); else single elements,
// straight to registers.
template <class T, bool DROP, bool ADD, int K, int R, bool WIDE>
__global__ void __launch_bounds__(32 * LN_MAX_WARPS) layer_norm_kernel(const __grid_constant__ NormParams p) {
  using Ring = RowRing<T, K, ADD ? 2 : 1, R>;
  extern __shared__ uint4 ln_smem[];
  __shared__ float4 part[2][R][LN_MAX_WARPS];  // a warp's mean, sum of squares from it, count
  const Teams<K> teams(p);
  const int warp = teams.warp_in_team(p);
  const RowPlace<T, K> place(p, warp);
  const Ring ring(ln_smem, teams.warp);
  const uint32_t rows = static_cast<uint32_t>(p.M), stride = static_cast<uint32_t>(teams.stride) * R;
  // this thread's columns: of the rows to fetch next (WIDE) or to work on
  const T* x = static_cast<const T*>(p.x) + teams.first * R * p.ld_x + (WIDE ? place.copy_col : place.col);
  const T* residual = ADD && p.other != nullptr
                          ? static_cast<const T*>(p.other) + teams.first * R * p.ld_other + (WIDE ? place.copy_col : place.col)
                          : nullptr;
  const int64_t step_x = stride * p.ld_x, step_residual = stride * p.ld_other;
  auto fetch = [&](uint32_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (row + r < rows) {
        ring.fetch(r, 0, x + r * p.ld_x, place);
        if (ADD && residual != nullptr) ring.fetch(r, 1, residual + r * p.ld_other, place);
      }
    ptx::cp_async_commit();
  };
  const uint32_t first_row = static_cast<uint32_t>(teams.first) * R;
  if constexpr (WIDE) {
    if (!place.full || (ADD && residual == nullptr)) ring.clear(place, residual == nullptr ? 1 : 2);
    fetch(first_row);
  }
  uint32_t step = 0;
  if constexpr (DROP) step = drop_step(p.drop);
  const float* weights = nullptr;  // this thread's, staged: w, then b `width` further on
  if (p.staged) {
    float* to = reinterpret_cast<float*>(ln_smem + (blockDim.x >> 5) * (Ring::WARP_BYTES / 16));
    stage_weights(to, p.w, p.N, teams.width, 1.0f);
    stage_weights(to + teams.width, p.b, p.N, teams.width, 0.0f);
    weights = to + warp * K * LN_PIECE + (threadIdx.x & 31) * 4;
    __syncthreads();
  }
  T* y = static_cast<T*>(p.y) + teams.first * R * p.ld_y + place.col;
  T* sum = p.sum != nullptr ? static_cast<T*>(p.sum) + teams.first * R * p.ld_sum + place.col : nullptr;
  const int64_t step_y = stride * p.ld_y, step_sum = stride * p.ld_sum;

  const int count = min(max(p.N - warp * K * LN_PIECE, 0), K * LN_PIECE);  // of the warp's values
  const float inv_count = 1.0f / static_cast<float>(max(count, 1));
  int parity = 0;
  for (uint32_t row = first_row; row < rows; row += stride) {
    Eight h[R][K];
    float mean[R], square[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      uint32_t words[K][4];
      if constexpr (DROP) row_words(p.drop, step, row + r, place.col, words);
      if (WIDE && r == 0) {
        ptx::cp_async_wait<0>();
        Ring::sync();
      }
      float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Eight add;
        add.clear();
        if constexpr (WIDE) {
          ring.take(r, 0, k, h[r][k]);
          if constexpr (ADD) ring.take(r, 1, k, add);
        } else {
          const int valid = row + r < rows ? place.valid(k) : 0;
          h[r][k].load(x + r * p.ld_x + k * LN_PIECE, valid, false);
          if (ADD && residual != nullptr) add.load(residual + r * p.ld_other + k * LN_PIECE, valid, false);
        }
        if constexpr (DROP)
          h[r][k].drop_onto(add, p.drop, words[k]);
        else if constexpr (ADD)
          h[r][k].plus(add);
        s2 = __fadd2_rn(s2, h[r][k].sum());
      }
      mean[r] = s2.x + s2.y;
    }
    x += step_x;  // the slots' values are in registers
    if (ADD && residual != nullptr) residual += step_residual;
    if constexpr (WIDE) {
      Ring::sync();
      fetch(row + stride);
    }

#pragma unroll
    for (int r = 0; r < R; ++r) mean[r] = warp_sum(mean[r]) * inv_count;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (place.full) {
        float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k) s2 = __fadd2_rn(s2, h[r][k].squares(mean[r]));
        square[r] = s2.x + s2.y;
      } else {
        square[r] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) square[r] += h[r][k].squares(mean[r], place.valid(k));
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) square[r] = warp_sum(square[r]);
    if (p.warps > 1) {
      if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r)
          part[parity][r][teams.warp] = make_float4(mean[r], square[r], static_cast<float>(count), 0.0f);
      }
      team_sync(teams.team, p.warps);  // the other buffer is read before the next rows' barrier
#pragma unroll
      for (int r = 0; r < R; ++r) {
        // Sums of the warps' means and squares, both from the first warp's mean.
        const float4* theirs = part[parity][r] + teams.team * p.warps;
        const float4 first = theirs[0];
        float shift = 0.0f;
        square[r] = first.y;
        for (int i = 1; i < p.warps; ++i) {
          const float4 v = theirs[i];
          const float delta = v.x - first.x;
          shift = fmaf(v.z, delta, shift);
          square[r] += fmaf(v.z * delta, delta, v.y);
        }
        shift *= p.inv_n;
        mean[r] = first.x + shift;
        square[r] = fmaf(-shift * shift, static_cast<float>(p.N), square[r]);
        square[r] = square[r] < 0.0f ? 0.0f : square[r];  // a NaN stays
      }
      parity ^= 1;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rstd[r] = 1.0f / sqrtf(fmaf(square[r], p.inv_n, p.eps));
      if (place.col == 0 && row + r < rows) {
        if (p.mean != nullptr) p.mean[row + r] = mean[r];
        if (p.rstd != nullptr) p.rstd[row + r] = rstd[r];
      }
    }
    auto finish = [&](int k, int valid, const Eight& w, const Eight& b) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (row + r >= rows) break;
        Eight& v = h[r][k];
        if (sum != nullptr) v.store(sum + r * p.ld_sum + k * LN_PIECE, valid, WIDE);
        v.normalise(mean[r], rstd[r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.v[i] = __ffma2_rn(v.v[i], w.v[i], b.v[i]);
        v.store(y + r * p.ld_y + k * LN_PIECE, valid, WIDE);
      }
    };
    if (place.full && weights != nullptr) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Eight w, b;
        staged_weights(weights, k, w);
        staged_weights(weights + teams.width, k, b);
        finish(k, 8, w, b);
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int valid = place.valid(k);
        if (valid <= 0) continue;
        Eight w, b;
        w.weights(p.w, place.col + k * LN_PIECE, valid, WIDE, 1.0f);
        b.weights(p.b, place.col + k * LN_PIECE, valid, WIDE, 0.0f);
        finish(k, valid, w, b);
      }
    }
    y += step_y;
    if (sum != nullptr) sum += step_sum;
  }
}

// Rows of up to 256 columns: teams of part of a warp (or all of it), each R
// neighbouring rows at once, whose sums' shuffles then overlap, and the next
// ones on their way: two sets of R rows in the ring.
template <class T>
constexpr int LN_NARROW_ROWS = 8 / sizeof(T);
template <class T>
constexpr int LN_NARROW_BACKWARD_ROWS = 4 / sizeof(T);

// A thread's place and its warp's ring, laid out and filled as RowRing.
template <class T, int R, int TENSORS>
struct NarrowRows {
  static constexpr int PARTS = Group<T>::PIECES, DEPTH = 2;
  static constexpr int WARP_BYTES = DEPTH * TENSORS * R * PARTS * 512;
  int64_t row, stride;  // of R neighbouring ones
  int64_t leader;       // the warp's first: the same for all its lanes
  int col, valid;
  const uint4* slots;   // this thread's first to read

  __device__ __forceinline__ NarrowRows(const NormParams& p, uint4* smem) {
    const int teams = 32 >> p.log_lanes, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    leader = (static_cast<int64_t>(blockIdx.x) * LN_BLOCK_WARPS + warp) * teams * R;
    row = leader + (lane >> p.log_lanes) * R;
    stride = static_cast<int64_t>(gridDim.x) * LN_BLOCK_WARPS * teams * R;
    col = (lane & ((1 << p.log_lanes) - 1)) * 8;
    valid = min(p.N - col, 8);
    if (valid <= 0) col = valid = 0;
    slots = smem + warp * (WARP_BYTES / 16) + lane;
  }
  static __device__ __forceinline__ constexpr int index(int d, int t, int r, int part) {
    return (((d * TENSORS + t) * R + r) * PARTS + part) * 32;
  }
  // Rows `at` .. at + R - 1 of a tensor into set d, zeros behind its last row and
  // column.
  __device__ __forceinline__ void fetch(const NormParams& p, int d, int t, const void* data, int64_t ld, int64_t at) const {
    constexpr int EACH = 8 / PARTS;
    const int lane = threadIdx.x & 31, lanes = 1 << p.log_lanes, in_team = lane & (lanes - 1);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < PARTS; ++i) {
        const int j = i * lanes + in_team;  // which 16 bytes of the row
        const int n = at + r < p.M ? min(max(p.N - j * EACH, 0), EACH) : 0;
        const T* src = static_cast<const T*>(data) + (n > 0 ? (at + r) * ld + j * EACH : 0);
        const int to = PARTS == 1 ? index(d, t, r, 0) : index(d, t, r, j & 1) + (j >> 1) - in_team;
        ptx::cp_async16(ptx::smem_addr(slots + to), src, static_cast<uint32_t>(n) * sizeof(T));
      }
  }
  __device__ __forceinline__ void take(int d, int t, int r, Eight& v) const {
    Group<T> g;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) g.q[i] = slots[index(d, t, r, i)];
    v.from(g);
  }
  __device__ __forceinline__ void load(const NormParams& p, const void* data, int64_t ld, int64_t at, Eight& v) const {
    v.load(static_cast<const T*>(data) + at * ld + col, at < p.M ? valid : 0, false);
  }
  // The words of the thread's group in its R rows.
  __device__ __forceinline__ void words(const Dropout& d, uint32_t step, int64_t at, uint32_t (&w)[R][4]) const {
    uint32_t rows[R], groups[R];
#pragma unroll
    for (int r = 0; r < R; ++r) rows[r] = static_cast<uint32_t>(at + r), groups[r] = static_cast<uint32_t>(col) >> 3;
    drop_words(d, step, rows, groups, w);
  }
};

template <class T, bool DROP, bool WIDE>
__global__ void __launch_bounds__(32 * LN_BLOCK_WARPS, 2) layer_norm_narrow_kernel(const __grid_constant__ NormParams p) {
  constexpr int R = LN_NARROW_ROWS<T>;
  using Rows = NarrowRows<T, R, 2>;
  extern __shared__ uint4 ln_smem[];
  const Rows at(p, ln_smem);
  auto fetch = [&](int d, int64_t row) {
    if constexpr (WIDE) {
      at.fetch(p, d, 0, p.x, p.ld_x, row);
      if (p.other != nullptr) at.fetch(p, d, 1, p.other, p.ld_other, row);
      ptx::cp_async_commit();
    }
  };
  fetch(0, at.row);
  fetch(1, at.row + at.stride);
  uint32_t step = 0;
  if constexpr (DROP) step = drop_step(p.drop);
  Eight w, b;
  w.weights(p.w, at.col, at.valid, WIDE, 1.0f);
  b.weights(p.b, at.col, at.valid, WIDE, 0.0f);
  int64_t row = at.row;
  int d = 0;
  for (int64_t leader = at.leader; leader < p.M; leader += at.stride, row += at.stride) {
    Eight h[R];
    float mean[R], square[R];
    uint32_t words[R][4];
    if constexpr (DROP) at.words(p.drop, step, row, words);
    if constexpr (WIDE) {
      ptx::cp_async_wait<1>();
      __syncwarp();
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Eight add;
      add.clear();
      if constexpr (WIDE) {
        at.take(d, 0, r, h[r]);
        if (p.other != nullptr) at.take(d, 1, r, add);
      } else {
        at.load(p, p.x, p.ld_x, row + r, h[r]);
        if (p.other != nullptr) at.load(p, p.other, p.ld_other, row + r, add);
      }
      if constexpr (DROP)
        h[r].drop_onto(add, p.drop, words[r]);
      else
        h[r].plus(add);
      const float2 s = h[r].sum();
      mean[r] = s.x + s.y;
    }
    __syncwarp();  // all lanes have read
    fetch(d, row + 2 * at.stride);
    d ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) mean[r] = team_sum(mean[r], p.log_lanes) * p.inv_n;
#pragma unroll
    for (int r = 0; r < R; ++r) square[r] = h[r].squares(mean[r], at.valid);
#pragma unroll
    for (int r = 0; r < R; ++r) square[r] = team_sum(square[r], p.log_lanes);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float rstd = 1.0f / sqrtf(fmaf(square[r], p.inv_n, p.eps));
      if (row + r >= p.M || at.valid == 0) continue;
      if (at.col == 0) {
        if (p.mean != nullptr) p.mean[row + r] = mean[r];
        if (p.rstd != nullptr) p.rstd[row + r] = rstd;
      }
      if (p.sum != nullptr) h[r].store(static_cast<T*>(p.sum) + (row + r) * p.ld_sum + at.col, at.valid, WIDE);
      h[r].normalise(mean[r], rstd);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[r].v[j] = __ffma2_rn(h[r].v[j], w.v[j], b.v[j]);
      h[r].store(static_cast<T*>(p.y) + (row + r) * p.ld_y + at.col, at.valid, WIDE);
    }
  }
}

// ------------------------------------------------------------------ backward

// g of one group from dy, n = (x - mean) rstd and the row's two means.
__device__ __forceinline__ void norm_gradient(Eight& g, const Eight& n, const Eight& w, const Eight& add, float rstd, float m1,
                                              float m2) {
  const float2 r = make_float2(rstd, rstd), minus1 = make_float2(-m1, -m1), minus2 = make_float2(-m2, -m2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = __ffma2_rn(g.v[i], w.v[i], minus1);
    g.v[i] = __ffma2_rn(__ffma2_rn(n.v[i], minus2, a), r, add.v[i]);
  }
}

// Sums of a row's a and a n, and the weights' gradients, of one group.
__device__ __forceinline__ void add_group(const Eight& g, const Eight& n, const Eight& w, Eight& dw, Eight& db, float2& s1,
                                          float2& s2) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    dw.v[i] = __ffma2_rn(g.v[i], n.v[i], dw.v[i]);
    db.v[i] = __fadd2_rn(db.v[i], g.v[i]);
    const float2 a = __fmul2_rn(g.v[i], w.v[i]);
    s1 = __fadd2_rn(s1, a);
    s2 = __ffma2_rn(a, n.v[i], s2);
  }
}

// The sums of dw and db of a block's teams meet in shared memory at the end.  A
// row stays in its slots until it is finished, while the next is on its way.
template <class T, bool DROP, bool ADD, int K, bool WIDE>
__global__ void __launch_bounds__(32 * LN_MAX_WARPS) layer_norm_backward_kernel(const __grid_constant__ NormParams p) {
  constexpr int DEPTH = LN_BACKWARD_DEPTH<T>;
  using Ring = RowRing<T, K, ADD ? 3 : 2, DEPTH>;
  constexpr int BATCH = K % 2 == 0 ? 2 : K;
  extern __shared__ uint4 ln_smem[];
  __shared__ float2 part[2][LN_MAX_WARPS];  // a warp's sums of a and a n
  const Teams<K> teams(p);
  const int warp = teams.warp_in_team(p);
  const RowPlace<T, K> place(p, warp);
  const int col = WIDE ? place.copy_col : place.col;
  const Ring ring(ln_smem, teams.warp);
  const uint32_t rows = static_cast<uint32_t>(p.M), stride = static_cast<uint32_t>(teams.stride);
  // Addresses are worked out where they are needed: kept, they would cost 20 of
  // the 128 registers, of which the sums of dw and db take 64 at K = 4.
  auto at = [&](const void* data, int64_t ld, uint32_t row) { return static_cast<const T*>(data) + row * ld + col; };
  auto fetch = [&](int d, uint32_t row) {
    if (row < rows) {
      ring.fetch(d, 0, at(p.other, p.ld_other, row), place);
      ring.fetch(d, 1, at(p.x, p.ld_x, row), place);
      if constexpr (ADD) ring.fetch(d, 2, at(p.add, p.ld_add, row), place);
    }
    ptx::cp_async_commit();
  };
  if constexpr (WIDE) {
    if (!place.full) ring.clear(place, 3);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) fetch(d, static_cast<uint32_t>(teams.first) + d * stride);
  }
  uint32_t step = 0;
  if constexpr (DROP) step = drop_step(p.drop);
  const float* weights = nullptr;  // this thread's, staged
  if (p.staged) {
    float* to = reinterpret_cast<float*>(ln_smem + (blockDim.x >> 5) * (Ring::WARP_BYTES / 16));
    stage_weights(to, p.w, p.N, teams.width, 1.0f);
    weights = to + warp * K * LN_PIECE + (threadIdx.x & 31) * 4;
    __syncthreads();
  }

  Eight dw[K], db[K];
#pragma unroll
  for (int k = 0; k < K; ++k) dw[k].clear(), db[k].clear();

  int d = 0, parity = 0;
  float next_mean = teams.first < p.M ? __ldg(p.mean + teams.first) : 0.0f;
  float next_rstd = teams.first < p.M ? __ldg(p.rstd + teams.first) : 0.0f;
  for (uint32_t row = static_cast<uint32_t>(teams.first); row < rows; row += stride) {
    const float mean = next_mean, rstd = next_rstd;
    if (row + stride < rows) {
      next_mean = __ldg(p.mean + row + stride);
      next_rstd = __ldg(p.rstd + row + stride);
    }
    auto take = [&](int k, Eight& g, Eight& n) {
      if constexpr (WIDE) {
        ring.take(d, 0, k, g);
        ring.take(d, 1, k, n);
      } else {
        g.load(at(p.other, p.ld_other, row) + k * LN_PIECE, place.valid(k), false);
        n.load(at(p.x, p.ld_x, row) + k * LN_PIECE, place.valid(k), false);
      }
      n.normalise(mean, rstd);
    };
    // f(k, valid columns, weights) of the thread's pieces that have any
    auto pieces = [&](auto&& f) {
      if (place.full && weights != nullptr) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          Eight w;
          staged_weights(weights, k, w);
          f(k, 8, w);
        }
      } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int valid = place.valid(k);
          if (valid <= 0) continue;
          Eight w;
          w.weights(p.w, place.col + k * LN_PIECE, valid, WIDE, 1.0f);
          f(k, valid, w);
        }
      }
    };
    if constexpr (WIDE) {
      ptx::cp_async_wait<DEPTH - 1>();
      Ring::sync();
    }
    float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
    pieces([&](int k, int, const Eight& w) {
      Eight g, n;
      take(k, g, n);  // dy is zero behind the row's end
      add_group(g, n, w, dw[k], db[k], s1, s2);
    });
    if (p.y != nullptr || p.sum != nullptr) {
      float m1 = warp_sum(s1.x + s1.y), m2 = warp_sum(s2.x + s2.y);
      if (p.warps > 1) {
        const float2* theirs = part[parity] + teams.team * p.warps;
        if ((threadIdx.x & 31) == 0) part[parity][teams.warp] = make_float2(m1, m2);
        team_sync(teams.team, p.warps);  // the other buffer is read before the next row's barrier
        m1 = m2 = 0.0f;
        for (int i = 0; i < p.warps; ++i) {
          const float2 v = theirs[i];
          m1 += v.x;
          m2 += v.y;
        }
        parity ^= 1;
      }
      m1 *= p.inv_n;
      m2 *= p.inv_n;
      uint32_t words[BATCH][4];
      T* y = static_cast<T*>(p.y) + row * p.ld_y + place.col;
      T* sum = static_cast<T*>(p.sum) + row * p.ld_sum + place.col;
      pieces([&](int k, int valid, const Eight& w) {
        if constexpr (DROP) {
          if (k % BATCH == 0) row_words(p.drop, step, row, place.col + k * LN_PIECE, words);
        }
        Eight g, n, a;
        take(k, g, n);
        a.clear();
        if constexpr (ADD) {
          if constexpr (WIDE)
            ring.take(d, 2, k, a);
          else
            a.load(at(p.add, p.ld_add, row) + k * LN_PIECE, valid, false);
        }
        norm_gradient(g, n, w, a, rstd, m1, m2);
        if (p.sum != nullptr) g.store(sum + k * LN_PIECE, valid, WIDE);
        if constexpr (DROP) g.drop(p.drop, words[k % BATCH]);
        if (p.y != nullptr) g.store(y + k * LN_PIECE, valid, WIDE);
      });
    }
    if constexpr (WIDE) {
      Ring::sync();
      fetch(d, row + DEPTH * stride);
      d = d + 1 == DEPTH ? 0 : d + 1;
    }
  }
  if (p.partials == nullptr) return;
  if constexpr (WIDE) ptx::cp_async_wait<0>();
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.N;
  float* shared = reinterpret_cast<float*>(ln_smem);  // [team][2][N]
  if (teams.count > 1) {
    __syncthreads();  // the slots are read
    out = shared + teams.team * 2 * p.N;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float a[8], b[8];
    dw[k].to(a);
    db[k].to(b);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < place.valid(k)) {
        out[place.col + k * LN_PIECE + j] = a[j];
        out[p.N + place.col + k * LN_PIECE + j] = b[j];
      }
  }
  if (teams.count > 1) {
    __syncthreads();
    out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.N;
    for (int i = threadIdx.x; i < 2 * p.N; i += blockDim.x) {
      float t = 0.0f;
      for (int v = 0; v < teams.count; ++v) t += shared[v * 2 * p.N + i];
      out[i] = t;
    }
  }
}

template <class T, bool DROP, bool WIDE>
__global__ void __launch_bounds__(32 * LN_BLOCK_WARPS, 2)
    layer_norm_backward_narrow_kernel(const __grid_constant__ NormParams p) {
  constexpr int R = LN_NARROW_BACKWARD_ROWS<T>;
  using Rows = NarrowRows<T, R, 3>;
  extern __shared__ uint4 ln_smem[];
  __shared__ float shared[LN_BLOCK_WARPS][2][LN_PIECE];
  const Rows at(p, ln_smem);
  float next_mean[R], next_rstd[R];
  auto fetch = [&](int d, int64_t row) {
    if constexpr (WIDE) {
      at.fetch(p, d, 0, p.other, p.ld_other, row);
      at.fetch(p, d, 1, p.x, p.ld_x, row);
      if (p.add != nullptr) at.fetch(p, d, 2, p.add, p.ld_add, row);
      ptx::cp_async_commit();
    }
  };
  auto statistics = [&](int64_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      next_mean[r] = row + r < p.M ? __ldg(p.mean + row + r) : 0.0f;
      next_rstd[r] = row + r < p.M ? __ldg(p.rstd + row + r) : 0.0f;
    }
  };
  fetch(0, at.row);
  fetch(1, at.row + at.stride);
  statistics(at.row);
  uint32_t step = 0;
  if constexpr (DROP) step = drop_step(p.drop);
  Eight w, dw, db;
  w.weights(p.w, at.col, at.valid, WIDE, 1.0f);
  dw.clear(), db.clear();
  int64_t row = at.row;
  int d = 0;
  for (int64_t leader = at.leader; leader < p.M; leader += at.stride, row += at.stride) {
    Eight g[R], n[R];
    float m1[R], m2[R], rstd[R];
    uint32_t words[R][4];
    if constexpr (DROP) at.words(p.drop, step, row, words);
    if constexpr (WIDE) {
      ptx::cp_async_wait<1>();
      __syncwarp();
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if constexpr (WIDE) {
        at.take(d, 0, r, g[r]);
        at.take(d, 1, r, n[r]);
      } else {
        at.load(p, p.other, p.ld_other, row + r, g[r]);
        at.load(p, p.x, p.ld_x, row + r, n[r]);
      }
      rstd[r] = next_rstd[r];
      n[r].normalise(next_mean[r], rstd[r]);
      float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
      add_group(g[r], n[r], w, dw, db, s1, s2);  // dy is zero behind the last row and column
      m1[r] = s1.x + s1.y;
      m2[r] = s2.x + s2.y;
    }
    statistics(row + at.stride);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m1[r] = team_sum(m1[r], p.log_lanes) * p.inv_n;
      m2[r] = team_sum(m2[r], p.log_lanes) * p.inv_n;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Eight add;
      add.clear();
      if (p.add != nullptr) {
        if constexpr (WIDE)
          at.take(d, 2, r, add);
        else
          at.load(p, p.add, p.ld_add, row + r, add);
      }
      if (row + r >= p.M || at.valid == 0) continue;
      norm_gradient(g[r], n[r], w, add, rstd[r], m1[r], m2[r]);
      if (p.sum != nullptr) g[r].store(static_cast<T*>(p.sum) + (row + r) * p.ld_sum + at.col, at.valid, WIDE);
      if constexpr (DROP) g[r].drop(p.drop, words[r]);
      if (p.y != nullptr) g[r].store(static_cast<T*>(p.y) + (row + r) * p.ld_y + at.col, at.valid, WIDE);
    }
    __syncwarp();  // all lanes have read
    fetch(d, row + 2 * at.stride);
    d ^= 1;
  }
  if (p.partials == nullptr) return;
  // A warp's teams by shuffles, then the warps in shared memory.
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float a[8], b[8];
  dw.to(a);
  db.to(b);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    for (int s = 1 << p.log_lanes; s < 32; s <<= 1) {
      a[j] += __shfl_xor_sync(0xffffffffu, a[j], s);
      b[j] += __shfl_xor_sync(0xffffffffu, b[j], s);
    }
    if (lane >> p.log_lanes == 0 && j < at.valid) {
      shared[warp][0][at.col + j] = a[j];
      shared[warp][1][at.col + j] = b[j];
    }
  }
  __syncthreads();
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.N;
  for (int i = threadIdx.x; i < 2 * p.N; i += blockDim.x) {
    const int which = i >= p.N, col = i - which * p.N;
    float t = 0.0f;
#pragma unroll
    for (int v = 0; v < LN_BLOCK_WARPS; ++v) t += shared[v][which][col];
    out[i] = t;
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

template <class T, bool DROP, bool WIDE>
__global__ void __launch_bounds__(LN_LONG_THREADS) layer_norm_long_kernel(const __grid_constant__ NormParams p) {
  __shared__ float part[LN_LONG_THREADS / 32];
  uint32_t step = 0;
  if constexpr (DROP) step = drop_step(p.drop);
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    auto load = [&](int g, float (&h)[8]) {
      load_group(static_cast<const T*>(p.x) + row * p.ld_x + g * 8, p.N - g * 8, WIDE, h);
      float r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = 0.0f;
      if (p.other != nullptr)
        load_group(static_cast<const T*>(p.other) + row * p.ld_other + g * 8, p.N - g * 8, WIDE, r);
      if constexpr (DROP) {
        uint32_t w[1][4];
        row_words(p.drop, step, static_cast<uint32_t>(row), g * 8, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = drop_keeps(w[0], j, p.drop.above) ? fmaf(h[j], p.drop.scale, r[j]) : r[j];
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
      float f[8];
      load(g, f);
      Eight h;
      h.from(f);
      s += h.squares(mean, p.N - g * 8);
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
      if (p.sum != nullptr) store_group(static_cast<T*>(p.sum) + row * p.ld_sum + g * 8, valid, WIDE, h);
      load_weights(p.w, g * 8, valid, WIDE, 1.0f, w);
      load_weights(p.b, g * 8, valid, WIDE, 0.0f, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = fmaf((h[j] - mean) * rstd, w[j], b[j]);
      store_group(static_cast<T*>(p.y) + row * p.ld_y + g * 8, valid, WIDE, w);
    }
  }
}

// The sums over rows are kept in the block's partials themselves, each column
// by the thread that works on it in every row.
template <class T, bool DROP, bool WIDE>
__global__ void __launch_bounds__(LN_LONG_THREADS) layer_norm_backward_long_kernel(const __grid_constant__ NormParams p) {
  __shared__ float part[LN_LONG_THREADS / 32];
  uint32_t step = 0;
  if constexpr (DROP) step = drop_step(p.drop);
  float* sums = p.partials == nullptr ? nullptr : p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.N;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
    auto load = [&](int g, float (&dy)[8], float (&n)[8]) {
      load_group(static_cast<const T*>(p.other) + row * p.ld_other + g * 8, p.N - g * 8, WIDE, dy);
      load_group(static_cast<const T*>(p.x) + row * p.ld_x + g * 8, p.N - g * 8, WIDE, n);
#pragma unroll
      for (int j = 0; j < 8; ++j) n[j] = (n[j] - mean) * rstd;
    };
    float s1 = 0.0f, s2 = 0.0f;
    for (int g = threadIdx.x; g < p.groups; g += LN_LONG_THREADS) {
      const int valid = p.N - g * 8;
      float dy[8], n[8], w[8];
      load(g, dy, n);
      load_weights(p.w, g * 8, valid, WIDE, 1.0f, w);
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
      load_weights(p.w, g * 8, valid, WIDE, 1.0f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) dy[j] = rstd * (fmaf(dy[j], w[j], -s1) - n[j] * s2);
      if (p.add != nullptr) {
        load_group(static_cast<const T*>(p.add) + row * p.ld_add + g * 8, valid, WIDE, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) dy[j] += w[j];
      }
      if (p.sum != nullptr) store_group(static_cast<T*>(p.sum) + row * p.ld_sum + g * 8, valid, WIDE, dy);
      if (p.y != nullptr) {
        if constexpr (DROP) {
          uint32_t words[1][4];
          row_words(p.drop, step, static_cast<uint32_t>(row), g * 8, words);
#pragma unroll
          for (int j = 0; j < 8; ++j) dy[j] = drop_keeps(words[0], j, p.drop.above) ? dy[j] * p.drop.scale : 0.0f;
        }
        store_group(static_cast<T*>(p.y) + row * p.ld_y + g * 8, valid, WIDE, dy);
      }
    }
  }
}

}  // namespace ge
