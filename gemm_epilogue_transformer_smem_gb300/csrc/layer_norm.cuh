// layer_norm.cuh -- dropout, and layer norm with the dropout and the residual
// add in front of it in the same pass (its backward: layer_norm_backward.cuh).
//
// For a row x of N values (D: dropout, w and b the norm's weight and bias):
//   dropout    y  = D(x) + residual
//   norm       h  = D(x) + residual,  mean and variance of h,
//              r  = 1 / sqrt(variance + eps),  y = (h - mean) r w + b
//   backward   n  = (h - mean) r,  a = dy w
//              g  = r (a - mean(a) - n mean(a n)) + add     (the gradient of h)
//              d_residual = g,  dx = D(g),  dw = sum of dy n,  db = sum of dy
// Everything is fp32 between one load and one store of each value, the sums of
// dw and db too: each thread's over its rows, then the blocks' in a fixed order.
// The variance is that of the differences from a mean taken first, never of the
// squares and the mean; several warps take theirs from means of their own, which
// are joined by the means' differences.
//
// All of it is memory-bound, so a row is read once: a team of threads -- part of
// a warp, a warp, or up to 16 of them, as the width asks for -- holds a row in
// registers while its sums are taken.  The teams stay for all rows, so that the
// next rows are on their way while one is worked on: per-thread asynchronous
// copies bring them into shared-memory slots that only that thread reads,
// without a barrier and without registers.
//
// One GB300, of the measured copy bandwidth (6792 GB/s), what is left beside the
// copies: the chain from a row's sums to its stores, which 16 warps of an SM
// hide, and with dropout 8 integer instructions an element for the mask.
//   norm, dropout and residual, 16384 x 4096 bf16 (537 MB)   92.4 us  0.86
//   the same without dropout                                 88.6 us  0.89
//   norm alone, 16384 x 4096 (268 MB)                        47.5 us  0.83
//   backward with dropout and `add`, 16384 x 4096 (671 MB)  112.7 us  0.88
//   the same of 65536 x 1024                                112.4 us  0.88
//   backward with `add`, 2048 x 14336 (235 MB)               53.6 us  0.65 (16384
//     rows 290 us, 0.95): 13.5 rows to an SM, so that the way in of the first, the
//     14th round and the sum of the partial sums (5.5 us) weigh.  A row shared by a
//     cluster of two blocks, with two rows on an SM: 61
//   dropout, 8192 x 14336 (470 MB)                           78.5 us  0.88
//   rows that start anywhere, 16384 x 4095 (537 MB)         151   us  0.52: words
//     of 4 bytes in place of 16; backward (671 MB) 265 us, 0.37; up to 256 columns
//     by single elements, 65536 x 253 (133 MB) 73 us, 0.27, backward 96, 0.25; more
//     than 16384 likewise, 4096 x 16389 443 us, 0.18, backward 416, 0.24
//   weights off 16 bytes take aligned rows with them: 16384 x 4096 129 us, backward 210
#pragma once

#include <stdint.h>

#include <type_traits>
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
};

// The first `valid` values of 16 bytes' worth at p into q, which is zeros.
// `wide`: p is on 16 bytes.
template <class T>
__device__ __forceinline__ void load_part(const T* p, int valid, bool wide, uint4& q) {
  constexpr int EACH = 16 / sizeof(T);
  if (wide && valid >= EACH) {
    q = *reinterpret_cast<const uint4*>(p);
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < EACH; ++j)
      if (j < valid) {
        if (sizeof(T) == 4)
          w[j % 4] = *reinterpret_cast<const uint32_t*>(p + j);
        else
          w[j / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p + j)) << (j % 2 * 16);
      }
    q = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <class T>
__device__ __forceinline__ void store_part(T* p, int valid, bool wide, const uint4& q) {
  constexpr int EACH = 16 / sizeof(T);
  if (wide && valid >= EACH) {
    *reinterpret_cast<uint4*>(p) = q;
  } else {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < EACH; ++j)
      if (j < valid) {
        if (sizeof(T) == 4)
          *reinterpret_cast<uint32_t*>(p + j) = w[j % 4];
        else
          *reinterpret_cast<uint16_t*>(p + j) = static_cast<uint16_t>(w[j / 2] >> (j % 2 * 16));
      }
  }
}

// Eight neighbouring values likewise.
template <class T>
__device__ __forceinline__ void load_group(const T* p, int valid, bool wide, Group<T>& g) {
  constexpr int EACH = 16 / sizeof(T);
  g.clear();
#pragma unroll
  for (int i = 0; i < Group<T>::PIECES; ++i) load_part(p + i * EACH, valid - i * EACH, wide, g.q[i]);
}

template <class T>
__device__ __forceinline__ void load_group(const T* p, int valid, bool wide, float (&v)[8]) {
  Group<T> g;
  load_group(p, valid, wide, g);
  g.unpack(v);
}

template <class T>
__device__ __forceinline__ void store_group(T* p, int valid, bool wide, const float (&v)[8]) {
  constexpr int EACH = 16 / sizeof(T);
  Group<T> g;
  g.pack(v);
#pragma unroll
  for (int i = 0; i < Group<T>::PIECES; ++i) store_part(p + i * EACH, valid - i * EACH, wide, g.q[i]);
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
  __device__ __forceinline__ void plus(const Eight& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __fadd2_rn(v[i], r.v[i]);
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
  // Sum of (v - m)^2, m0 of the first four and m1 of the others.
  __device__ __forceinline__ float2 squares(float m0, float m1) const {
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float minus = -(i < 2 ? m0 : m1);
      const float2 c = __fadd2_rn(v[i], make_float2(minus, minus));
      s = __ffma2_rn(c, c, s);
    }
    return s;
  }
  // (this - mean) rstd
  __device__ __forceinline__ void normalise(float mean, float rstd) {
    const float2 minus = make_float2(-mean, -mean), r = make_float2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __fmul2_rn(__fadd2_rn(v[i], minus), r);
  }
};

// ------------------------------------------------------------------ rows

// A team of W warps holds a row: warp i the columns from i K 256 on, lane l in
// each of its K pieces of 256 columns the 8 from 8 l.  The offsets between
// pieces are constants, and what a row costs a thread beside its values (its
// sums' shuffles, the barrier, the addresses) is spread over 8 K of them.
constexpr int LN_PIECE = 256;
// Which columns of a piece are in the row: any, each 16 bytes' worth whole or not
// at all, all.
enum { LN_ANY, LN_WHOLE, LN_ALL };
constexpr int LN_MAX_WARPS = 16;
constexpr int LN_BLOCK_WARPS = 8;  // of blocks that hold several teams
constexpr int LN_MAX_SHARED = 224 * 1024;  // of the 227 KB of a block, beside what is not dynamic

// Columns of a partial sum: whole pieces.
__host__ __device__ constexpr int64_t partial_width(int64_t N) { return (N + LN_PIECE - 1) / LN_PIECE * LN_PIECE; }

struct NormParams {
  int32_t M, N, groups;
  int32_t warps;      // of a team
  int32_t staged;     // the norm's weights go through shared memory
  int32_t rows;       // rows too wide to hold, backward: at a time
  int32_t wide_w;     // else: 16-byte accesses serve them
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

// Where a thread's 8 K values of a row lie: in each of K pieces of 256 columns,
// PARTS times 16 bytes, neighbouring threads' side by side, so that an access of
// a warp takes whole sectors -- 8 neighbouring columns of bf16, twice 4 of fp32,
// 128 columns apart.
template <class T, int K>
struct RowPlace {
  static constexpr int PARTS = Group<T>::PIECES;
  static constexpr int EACH = 8 / PARTS, APART = LN_PIECE / PARTS;
  int col;    // of piece 0, part 0
  int left;   // columns from `col` to the row's end (<= 0: none)
  bool full;   // all of the warp's columns are in the row
  bool whole;  // each of a thread's 16 bytes is in the row or is not

  __device__ __forceinline__ RowPlace(int N, int begin) {
    col = begin + (threadIdx.x & 31) * EACH;
    left = N - col;
    full = begin + K * LN_PIECE <= N;
    whole = N % EACH == 0;
  }
  // Columns of a part that are in the row (<= 0: none).
  __device__ __forceinline__ int valid(int k, int i) const { return min(left - k * LN_PIECE - i * APART, EACH); }
  // Piece k from a row at `col`, zeros behind its end; all: none is there.
  __device__ __forceinline__ void load(const T* row, int k, bool all, Group<T>& g) const {
    g.clear();
#pragma unroll
    for (int i = 0; i < PARTS; ++i) load_part(row + k * LN_PIECE + i * APART, all ? EACH : valid(k, i), true, g.q[i]);
  }
  __device__ __forceinline__ void store(T* row, int k, bool all, const Eight& v) const {
    Group<T> g;
    float f[8];
    v.to(f);
    g.pack(f);
#pragma unroll
    for (int i = 0; i < PARTS; ++i) store_part(row + k * LN_PIECE + i * APART, all ? EACH : valid(k, i), true, g.q[i]);
  }
  // The same of a row whose 16 bytes are there whole or not at all, without a branch.
  __device__ __forceinline__ void store_whole(T* row, int k, const Eight& v) const {
    Group<T> g;
    float f[8];
    v.to(f);
    g.pack(f);
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
      if (valid(k, i) > 0) *reinterpret_cast<uint4*>(row + k * LN_PIECE + i * APART) = g.q[i];
  }
  // fp32 vectors, `none` behind the row's end and without one.
  __device__ __forceinline__ void weights(const float* w, int k, bool wide, float none, Eight& v) const {
    float f[8];
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const int at = col + k * LN_PIECE + i * APART, n = valid(k, i);
      if (w != nullptr && wide && n >= EACH) {
#pragma unroll
        for (int j = 0; j < EACH; j += 4) {
          const float4 q = __ldg(reinterpret_cast<const float4*>(w + at + j));
          f[i * EACH + j] = q.x, f[i * EACH + j + 1] = q.y, f[i * EACH + j + 2] = q.z, f[i * EACH + j + 3] = q.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < EACH; ++j) f[i * EACH + j] = w != nullptr && j < n ? __ldg(w + at + j) : none;
      }
    }
    v.from(f);
  }
  // f(value's place among the 8, its column) of piece k's columns in the row.
  template <class F>
  __device__ __forceinline__ void columns(int k, F&& f) const {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j % EACH < valid(k, j / EACH)) f(j, col + k * LN_PIECE + j / EACH * APART + j % EACH);
  }
  // Sum of (v - m)^2 over piece k's columns in the row, behind whose end v is 0.
  __device__ __forceinline__ float2 squares_whole(const Eight& v, float m, int k) const {
    return v.squares(valid(k, 0) > 0 ? m : 0.0f, valid(k, PARTS - 1) > 0 ? m : 0.0f);
  }
  __device__ __forceinline__ float squares(const Eight& v, float m, int k) const {
    float f[8], s = 0.0f;
    v.to(f);
    columns(k, [&](int j, int) { s = fmaf(f[j] - m, f[j] - m, s); });
    return s;
  }
  // The masks' words of B pieces from piece k0 on: words 0 and 1 of the first
  // four values, 2 and 3 of the others.  fp32's two parts are of two groups,
  // half of each: twice the work for an element, of twice the bytes.
  template <int B>
  __device__ __forceinline__ void words(const Dropout& d, uint32_t step, uint32_t row, int k0, uint32_t (&w)[B][4]) const {
    uint32_t rows[B * PARTS], groups[B * PARTS], all[B * PARTS][4];
#pragma unroll
    for (int i = 0; i < B * PARTS; ++i) {
      rows[i] = row;
      groups[i] = static_cast<uint32_t>(col + k0 * LN_PIECE + i * APART) >> 3;
    }
    drop_words(d, step, rows, groups, all);
    const bool second = PARTS == 2 && (col & 4);
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (PARTS == 1)
          w[i][j] = all[i][j];
        else
          w[i][j] = second ? all[2 * i + j / 2][2 + j % 2] : all[2 * i + j / 2][j % 2];
      }
  }
};

// Copies of a thread's values of the next rows on their way into slots that
// only it reads.  The ring starts on 128 bytes: a warp's 512 are then 4
// wavefronts and not 5 (16384 x 4096 backward: 134 us on 16 bytes, 126 so).
template <class T, int K, int TENSORS, int DEPTH>
struct RowRing {
  using Place = RowPlace<T, K>;
  static constexpr int PARTS = Place::PARTS;
  static constexpr int WARP_BYTES = DEPTH * TENSORS * K * PARTS * 512;
  uint4* slots;  // this thread's first
  uint32_t at;

  __device__ __forceinline__ RowRing(uint4* smem, int warp)
      : slots(smem + warp * (WARP_BYTES / 16) + (threadIdx.x & 31)), at(ptx::smem_addr(slots)) {}
  static __device__ __forceinline__ constexpr int index(int d, int t, int k, int part) {
    return (((d * TENSORS + t) * K + k) * PARTS + part) * 32;
  }
  // Zeros where no copy will land.
  __device__ __forceinline__ void clear(const Place& place, int first_unused_tensor) const {
#pragma unroll 1
    for (int d = 0; d < DEPTH; ++d)
      for (int t = 0; t < TENSORS; ++t)
        for (int k = 0; k < K; ++k)
          for (int i = 0; i < PARTS; ++i)
            if (t >= first_unused_tensor || place.valid(k, i) <= 0) slots[index(d, t, k, i)] = make_uint4(0, 0, 0, 0);
  }
  template <int... Is>
  static __device__ __forceinline__ void fetch_full(uint32_t to, const T* row, std::integer_sequence<int, Is...>) {
    (ptx::cp_async16<Is * 512, (Is / PARTS * LN_PIECE + Is % PARTS * Place::APART) * static_cast<int>(sizeof(T))>(to, row), ...);
  }
  // `row`: at the thread's first column.
  __device__ __forceinline__ void fetch(int d, int t, const T* row, const Place& place) const {
    const uint32_t to = at + static_cast<uint32_t>(index(d, t, 0, 0)) * 16u;
    if (place.full) {
      fetch_full(to, row, std::make_integer_sequence<int, K * PARTS>{});
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < PARTS; ++i)
          if (place.valid(k, i) > 0)
            ptx::cp_async16(to + static_cast<uint32_t>(index(0, 0, k, i)) * 16u, row + k * LN_PIECE + i * Place::APART,
                            static_cast<uint32_t>(place.valid(k, i)) * sizeof(T));
    }
  }
  __device__ __forceinline__ void take(int d, int t, int k, Eight& v) const {
    Group<T> g;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) g.q[i] = slots[index(d, t, k, i)];
    v.from(g);
  }
};

// The same for rows that start anywhere: a warp copies its columns word by word
// as they lie in memory, so a lane reads what others copied, and with bf16 rows
// that start between two words every lane's values lie half a word off.  A
// __syncwarp() lies between the copies' end and the reads, and the reads and the
// next copies.  (By single elements straight to registers, 16384 x 4095 bf16 with
// dropout and residual took 435 us.)
template <class T, int K, int TENSORS, int DEPTH>
struct WordRing {
  using Place = RowPlace<T, K>;
  static constexpr int SEGMENT = K * Place::PARTS * 512 + 128;  // of a row's columns, half a word off or not
  static constexpr int WARP_BYTES = DEPTH * TENSORS * SEGMENT;
  uint8_t* slots;  // the warp's
  uint32_t at;

  __device__ __forceinline__ WordRing(uint4* smem, int warp)
      : slots(reinterpret_cast<uint8_t*>(smem) + warp * WARP_BYTES), at(ptx::smem_addr(slots)) {}
  // Bytes that `row` lies behind a word's start: 2 or 0.
  static __device__ __forceinline__ uint32_t shift(const T* row) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) & 3u;
  }
  // A warp's words but the first of each lane.
  template <int... Is>
  static __device__ __forceinline__ void fetch_full(uint32_t to, const uint8_t* from, std::integer_sequence<int, Is...>) {
    (ptx::cp_async4<(Is + 1) * 128, (Is + 1) * 128>(to, from), ...);
  }
  // `row`: at the warp's first column, `count` of which are in the row.
  __device__ __forceinline__ void fetch(int d, int t, const T* row, int count) const {
    if (count <= 0) return;
    const uint32_t off = shift(row), bytes = static_cast<uint32_t>(count) * sizeof(T) + off;
    const uint8_t* src = reinterpret_cast<const uint8_t*>(row) - off;
    const int segment = (d * TENSORS + t) * SEGMENT;
    if (count == K * LN_PIECE) {  // an instruction to a word: 16384 x 4095 plain 94.5 us, 115 with the loop alone
      constexpr int FULL = K * LN_PIECE * static_cast<int>(sizeof(T)) / 128;
      const uint32_t lane = threadIdx.x & 31;
      if (off != 0 && lane == 0) {  // the first and the last half words
        uint16_t* to = reinterpret_cast<uint16_t*>(slots + segment);
        const uint16_t* from = reinterpret_cast<const uint16_t*>(row);
        to[1] = from[0];
        to[K * LN_PIECE] = from[K * LN_PIECE - 1];
      } else {
        ptx::cp_async4<0, 0>(at + segment + lane * 4, src + lane * 4);
      }
      fetch_full(at + segment + lane * 4, src + lane * 4, std::make_integer_sequence<int, FULL - 1>{});
      return;
    }
    uint32_t i = (threadIdx.x & 31) * 4;
    if (i == 0 && off != 0) {  // nothing in front of the row is read
      *reinterpret_cast<uint16_t*>(slots + segment + 2) = *reinterpret_cast<const uint16_t*>(row);
      i += 128;
    }
#pragma unroll 4
    for (; i + 4 <= bytes; i += 128) ptx::cp_async4<0, 0>(at + segment + i, src + i);
    if (i < bytes) ptx::cp_async4(at + segment + i, src + i, bytes - i);
  }
  // Zeros behind the row's end.
  __device__ __forceinline__ void take(int d, int t, int k, const T* row, const Place& place, Eight& v) const {
    Group<T> g;
    const uint8_t* from = slots + (d * TENSORS + t) * SEGMENT + (k * LN_PIECE + (threadIdx.x & 31) * Place::EACH) * sizeof(T);
#pragma unroll
    for (int i = 0; i < Place::PARTS; ++i)
      g.q[i] = *reinterpret_cast<const uint4*>(from + i * Place::APART * sizeof(T));
    if (shift(row) != 0) {
      const uint32_t next = *reinterpret_cast<const uint32_t*>(from + 16);
      uint4& q = g.q[0];
      q = make_uint4(__funnelshift_r(q.x, q.y, 16), __funnelshift_r(q.y, q.z, 16), __funnelshift_r(q.z, q.w, 16),
                     __funnelshift_r(q.w, next, 16));
    }
    float f[8];
    g.unpack(f);
    if (!place.full) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = j % Place::EACH < place.valid(k, j / Place::EACH) ? f[j] : 0.0f;
    }
    v.from(f);
  }
};

// Piece k of a warp's columns to a row that starts anywhere, through 1 KB of
// shared memory of the warp's own: words, side by side.  `row`: at the warp's
// first column, `count` of which are in the row.
template <class T>
__device__ __forceinline__ void store_words(uint4* smem, T* row, int count, int k, const Eight& v) {
  Group<T> g;
  float f[8];
  v.to(f);
  g.pack(f);
  const int lane = threadIdx.x & 31, left = min(count - k * LN_PIECE, LN_PIECE);
#pragma unroll
  for (int i = 0; i < Group<T>::PIECES; ++i) smem[i * 32 + lane] = g.q[i];
  __syncwarp();
  T* to = row + k * LN_PIECE;
  const T* from = reinterpret_cast<const T*>(smem);
  if (left == LN_PIECE) {
    const uint32_t* words = reinterpret_cast<const uint32_t*>(smem) + lane;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < 8; ++j) reinterpret_cast<uint32_t*>(to)[lane + 32 * j] = words[32 * j];
    } else if ((reinterpret_cast<uintptr_t>(to) & 2) == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) reinterpret_cast<uint32_t*>(to)[lane + 32 * j] = words[32 * j];
    } else {  // an element in front of the first word, one behind the last
      if (lane == 0) to[0] = from[0];
      uint32_t* at = reinterpret_cast<uint32_t*>(to + 1) + lane;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = __funnelshift_r(words[32 * j], words[32 * j + 1], 16);
        if (j == 3 && lane == 31)
          *reinterpret_cast<uint16_t*>(at + 32 * j) = static_cast<uint16_t>(w);
        else
          at[32 * j] = w;
      }
    }
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (lane + 32 * j < left) to[lane + 32 * j] = from[lane + 32 * j];
  } else {
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(to) >> 1) & 1;  // an element in front of the first word
    if (odd && lane == 0 && left > 0) to[0] = from[0];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = odd + 2 * (lane + 32 * j);
      if (e + 1 < left)
        *reinterpret_cast<uint32_t*>(to + e) = static_cast<uint32_t>(from[e]) | static_cast<uint32_t>(from[e + 1]) << 16;
      else if (e < left)
        to[e] = from[e];
    }
  }
  __syncwarp();
}

// ------------------------------------------------------------------ dropout

constexpr int DO_THREADS = 256;
constexpr int DO_BLOCKS = 3;  // resident per SM

struct DropoutParams {
  int32_t M, N;
  int32_t spans;      // of a warp's columns in a row; narrow rows: groups of 8 columns
  int64_t total;      // rows * spans
  int64_t step_rows;  // from one span of a warp (or group of a thread) to its next: rows and spans
  int32_t step_spans;
  const void* x;
  int64_t ld_x;
  const void* residual;  // or NULL
  int64_t ld_residual;
  void* y;
  int64_t ld_y;
  int32_t wide_in, wide_out;
  Dropout drop;
};

// A warp to K pieces of a row.  WIDE as in the norm's kernels.
template <class T, int K, bool WIDE>
__global__ void __launch_bounds__(DO_THREADS, DO_BLOCKS) dropout_kernel(const __grid_constant__ DropoutParams p) {
  using Words = WordRing<T, K, 2, 1>;
  extern __shared__ __align__(128) uint4 ln_smem[];  // by words: rings, then what is stored through
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (DO_THREADS / 32);
  int64_t i = static_cast<int64_t>(blockIdx.x) * (DO_THREADS / 32) + (threadIdx.x >> 5);
  int64_t row = i / p.spans;
  int32_t span = static_cast<int32_t>(i - row * p.spans);
  const uint32_t step = p.drop.step != nullptr ? drop_step(p.drop) : 0;
  for (; i < p.total; i += warps) {
    const int begin = span * K * LN_PIECE;
    const RowPlace<T, K> place(p.N, begin);
    uint32_t words[K][4];
    auto finish = [&](int k, Eight& v, const Eight& add) {
      if (p.drop.step != nullptr)
        v.drop_onto(add, p.drop, words[k]);
      else
        v.plus(add);
    };
    if constexpr (WIDE) {
      const T* x = static_cast<const T*>(p.x) + row * p.ld_x + place.col;
      const T* residual = p.residual != nullptr ? static_cast<const T*>(p.residual) + row * p.ld_residual + place.col : nullptr;
      T* y = static_cast<T*>(p.y) + row * p.ld_y + place.col;
      Group<T> g[K], r[K];
      auto load = [&](bool all) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          place.load(x, k, all, g[k]);
          r[k].clear();
          if (residual != nullptr) place.load(residual, k, all, r[k]);
        }
      };
      auto store = [&](bool all) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          Eight v, add;
          v.from(g[k]);
          add.from(r[k]);
          finish(k, v, add);
          place.store(y, k, all, v);
        }
      };
      place.full ? load(true) : load(false);
      if (p.drop.step != nullptr) place.words(p.drop, step, static_cast<uint32_t>(row), 0, words);
      place.full ? store(true) : store(false);
    } else {
      const int warp = threadIdx.x >> 5, count = min(p.N - begin, K * LN_PIECE);
      const Words ring(ln_smem, warp);
      uint4* staging = ln_smem + DO_THREADS / 32 * (Words::WARP_BYTES / 16) + warp * 64;
      const T* x = static_cast<const T*>(p.x) + row * p.ld_x + begin;
      const T* residual = p.residual != nullptr ? static_cast<const T*>(p.residual) + row * p.ld_residual + begin : nullptr;
      __syncwarp();  // the previous share's reads
      ring.fetch(0, 0, x, count);
      if (residual != nullptr) ring.fetch(0, 1, residual, count);
      ptx::cp_async_commit();
      if (p.drop.step != nullptr) place.words(p.drop, step, static_cast<uint32_t>(row), 0, words);
      ptx::cp_async_wait<0>();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Eight v, add;
        add.clear();
        ring.take(0, 0, k, x, place, v);
        if (residual != nullptr) ring.take(0, 1, k, residual, place, add);
        finish(k, v, add);
        store_words<T>(staging, static_cast<T*>(p.y) + row * p.ld_y + begin, count, k, v);
      }
    }
    row += p.step_rows, span += p.step_spans;
    if (span >= p.spans) span -= p.spans, ++row;
  }
}

// Rows of up to 256 columns: a thread to 8 neighbouring columns, whatever row
// they are in.
template <class T>
__global__ void __launch_bounds__(DO_THREADS, DO_BLOCKS) dropout_narrow_kernel(const __grid_constant__ DropoutParams p) {
  const int64_t threads = static_cast<int64_t>(gridDim.x) * DO_THREADS;
  int64_t i = static_cast<int64_t>(blockIdx.x) * DO_THREADS + threadIdx.x;
  int64_t row = i / p.spans;
  int32_t group = static_cast<int32_t>(i - row * p.spans);
  const uint32_t step = p.drop.step != nullptr ? drop_step(p.drop) : 0;
  constexpr int U = 4 / Group<T>::PIECES;  // of a thread in flight
  while (i < p.total) {
    uint32_t rows[U], groups[U], words[U][4];
    Group<T> x[U], r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rows[u] = static_cast<uint32_t>(row), groups[u] = static_cast<uint32_t>(group);
      x[u].clear();
      r[u].clear();
      if (i + u * threads < p.total) {
        const int col = group * 8;
        load_group(static_cast<const T*>(p.x) + row * p.ld_x + col, p.N - col, p.wide_in, x[u]);
        if (p.residual != nullptr)
          load_group(static_cast<const T*>(p.residual) + row * p.ld_residual + col, p.N - col, p.wide_in, r[u]);
      }
      row += p.step_rows, group += p.step_spans;
      if (group >= p.spans) group -= p.spans, ++row;
    }
    if (p.drop.step != nullptr) drop_words(p.drop, step, rows, groups, words);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Eight v, add;
      v.from(x[u]);
      add.from(r[u]);
      if (p.drop.step != nullptr)
        v.drop_onto(add, p.drop, words[u]);
      else
        v.plus(add);
      float f[8];
      v.to(f);
      const int col = static_cast<int>(groups[u]) * 8;
      if (i + u * threads < p.total)
        store_group(static_cast<T*>(p.y) + rows[u] * p.ld_y + col, p.N - col, p.wide_out, f);
    }
    i += U * threads;
  }
}

// ------------------------------------------------------------------ teams

// Shared memory of a warp: its ring, and what it stores words through.
template <class Ring, bool WIDE>
constexpr int HELD_WARP_BYTES = Ring::WARP_BYTES + (WIDE ? 0 : 1024);

// A block's teams.  Its shared memory: the warps' rings, by words what they store
// through, the norm's weights.
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
// four of its lanes' eight and then the others, so that 16-byte reads meet no
// bank twice.  A barrier has to follow.
template <class T>
__device__ __forceinline__ void stage_weights(float* to, const float* w, int n, int width, float none) {
  for (int i = threadIdx.x; i < width; i += blockDim.x) {
    const int col = sizeof(T) == 4 ? i : (i & ~(LN_PIECE - 1)) + (i >> 2 & 31) * 8 + (i >> 7 & 1) * 4 + (i & 3);
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

// ------------------------------------------------------------------ forward

// A team works on R neighbouring rows at once: they share the weights' reads,
// and their sums' shuffles and the barrier overlap.  WIDE: every tensor takes
// 16-byte accesses, and its rows come through the ring (with a depth of 1: rows
// are in registers while the next ones are on their way); else they come and go
// by words.
template <class T, bool DROP, bool ADD, int K, int R, bool WIDE>
__global__ void __launch_bounds__(32 * LN_MAX_WARPS) layer_norm_kernel(const __grid_constant__ NormParams p) {
  using Ring = std::conditional_t<WIDE, RowRing<T, K, ADD ? 2 : 1, R>, WordRing<T, K, ADD ? 2 : 1, R>>;
  extern __shared__ __align__(128) uint4 ln_smem[];
  __shared__ float4 part[2][R][LN_MAX_WARPS + 3];  // a warp's mean, sum of squares from it, count
  const Teams<K> teams(p);
  const int warp = teams.warp_in_team(p);
  const RowPlace<T, K> place(p.N, warp * K * LN_PIECE);
  const Ring ring(ln_smem, teams.warp);
  uint4* staging = ln_smem + (blockDim.x >> 5) * (Ring::WARP_BYTES / 16) + teams.warp * 64;  // by words: the warp's 1 KB
  const uint32_t rows = static_cast<uint32_t>(p.M), stride = static_cast<uint32_t>(teams.stride) * R;
  const bool residual = ADD && p.other != nullptr;
  // A row that ends inside the warp's columns, on 16 bytes, costs next to nothing more
  // (4000 columns plain 43 us, 58 else); the small kernels have no registers for it:
  // 64 are two blocks to an SM.
  constexpr bool BY_16 = K * R > 2;
  // worked out where they are needed: kept, they would cost registers
  const int begin = WIDE ? place.col : warp * K * LN_PIECE;
  const int count = min(max(p.N - warp * K * LN_PIECE, 0), K * LN_PIECE);  // of the warp's values
  auto at = [&](const void* data, int64_t ld, uint32_t row) { return static_cast<const T*>(data) + row * ld + begin; };
  auto fetch = [&](uint32_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (row + r < rows) {
        if constexpr (WIDE) {
          ring.fetch(r, 0, at(p.x, p.ld_x, row + r), place);
          if (residual) ring.fetch(r, 1, at(p.other, p.ld_other, row + r), place);
        } else {
          ring.fetch(r, 0, at(p.x, p.ld_x, row + r), count);
          if (residual) ring.fetch(r, 1, at(p.other, p.ld_other, row + r), count);
        }
      }
    ptx::cp_async_commit();
  };
  const uint32_t first_row = static_cast<uint32_t>(teams.first) * R;
  if constexpr (WIDE) {
    if (!place.full || (ADD && !residual)) ring.clear(place, residual ? 2 : 1);
  }
  fetch(first_row);
  uint32_t step = 0;
  if constexpr (DROP) step = drop_step(p.drop);
  const float* weights = nullptr;  // this thread's, staged: w, then b `width` further on
  if (p.staged) {
    float* to = reinterpret_cast<float*>(ln_smem + (blockDim.x >> 5) * (HELD_WARP_BYTES<Ring, WIDE> / 16));
    stage_weights<T>(to, p.w, p.N, teams.width, 1.0f);
    stage_weights<T>(to + teams.width, p.b, p.N, teams.width, 0.0f);
    weights = to + warp * K * LN_PIECE + (threadIdx.x & 31) * 4;
    __syncthreads();
  }

  const float inv_count = 1.0f / static_cast<float>(max(count, 1));
  int parity = 0;
  for (uint32_t row = first_row; row < rows; row += stride) {
    Eight h[R][K];
    float mean[R], square[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      uint32_t words[K][4];
      if constexpr (DROP) place.words(p.drop, step, row + r, 0, words);
      if (r == 0) {
        ptx::cp_async_wait<0>();
        if constexpr (!WIDE) __syncwarp();
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
          ring.take(r, 0, k, at(p.x, p.ld_x, row + r), place, h[r][k]);
          if (residual) ring.take(r, 1, k, at(p.other, p.ld_other, row + r), place, add);
        }
        if constexpr (DROP)
          h[r][k].drop_onto(add, p.drop, words[k]);
        else if constexpr (ADD)
          h[r][k].plus(add);
        s2 = __fadd2_rn(s2, h[r][k].sum());
      }
      mean[r] = s2.x + s2.y;
    }
    if constexpr (!WIDE) __syncwarp();
    fetch(row + stride);  // the slots' values are in registers

#pragma unroll
    for (int r = 0; r < R; ++r) mean[r] = warp_sum(mean[r]) * inv_count;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (place.full || (WIDE && BY_16 && place.whole)) {
        float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k)
          s2 = __fadd2_rn(s2, WIDE && BY_16 ? place.squares_whole(h[r][k], mean[r], k) : h[r][k].squares(mean[r], mean[r]));
        square[r] = s2.x + s2.y;
      } else {
        square[r] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) square[r] += place.squares(h[r][k], mean[r], k);
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
        for (int i0 = 1; i0 < p.warps; i0 += 4) {
#pragma unroll
          for (int i = i0; i < i0 + 4; ++i) {  // reads side by side; the last ones may be another team's
            const float4 v = theirs[i];
            const float delta = v.x - first.x;
            shift = i < p.warps ? fmaf(v.z, delta, shift) : shift;
            square[r] += i < p.warps ? fmaf(v.z * delta, delta, v.y) : 0.0f;
          }
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
    T* y = static_cast<T*>(p.y) + row * p.ld_y + begin;
    T* sum = static_cast<T*>(p.sum) + row * p.ld_sum + begin;
    auto store = [&](T* to, int k, auto part, const Eight& v) {
      if constexpr (!WIDE)
        store_words<T>(staging, to, count, k, v);
      else if constexpr (part == LN_WHOLE)
        place.store_whole(to, k, v);
      else
        place.store(to, k, part == LN_ALL, v);
    };
    auto finish = [&](int k, auto part, const Eight& w, const Eight& b) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (row + r >= rows) break;
        Eight& v = h[r][k];
        if (p.sum != nullptr) store(sum + r * p.ld_sum, k, part, v);
        v.normalise(mean[r], rstd[r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.v[i] = __ffma2_rn(v.v[i], w.v[i], b.v[i]);
        store(y + r * p.ld_y, k, part, v);
      }
    };
    auto staged = [&](auto part) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Eight w, b;
        staged_weights(weights, k, w);
        staged_weights(weights + teams.width, k, b);
        finish(k, part, w, b);
      }
    };
    if (WIDE && (place.full || (BY_16 && place.whole)) && weights != nullptr) {
      staged(std::integral_constant<int, BY_16 ? LN_WHOLE : LN_ALL>{});
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (WIDE ? place.valid(k, 0) <= 0 : count <= k * LN_PIECE) continue;  // by words: the warp as one
        Eight w, b;
        if (!WIDE && weights != nullptr) {
          staged_weights(weights, k, w);
          staged_weights(weights + teams.width, k, b);
        } else {
          place.weights(p.w, k, WIDE || p.wide_w, 1.0f, w);
          place.weights(p.b, k, WIDE || p.wide_w, 0.0f, b);
        }
        finish(k, std::integral_constant<int, LN_ANY>{}, w, b);
      }
    }
  }
}

// Rows of up to 256 columns: teams of part of a warp (or all of it), each R
// neighbouring rows at once, whose sums' shuffles then overlap, and the next
// ones on their way: two sets of R rows in the ring.
template <class T>
constexpr int LN_NARROW_ROWS = 8 / sizeof(T);
template <class T>
constexpr int LN_NARROW_BACKWARD_ROWS = 4 / sizeof(T);

// A thread's place and its slots in the ring.  As RowPlace, with the team's
// lanes in place of a warp's.
template <class T, int R, int TENSORS>
struct NarrowRows {
  static constexpr int PARTS = Group<T>::PIECES, EACH = 8 / PARTS, DEPTH = 2;
  static constexpr int WARP_BYTES = DEPTH * TENSORS * R * PARTS * 512;
  int64_t row, stride;  // of R neighbouring ones
  int64_t leader;       // the warp's first: the same for all its lanes
  int col, apart, N;    // part i at col + i apart
  uint4* slots;

  __device__ __forceinline__ NarrowRows(const NormParams& p, uint4* smem) {
    const int teams = 32 >> p.log_lanes, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    leader = (static_cast<int64_t>(blockIdx.x) * LN_BLOCK_WARPS + warp) * teams * R;
    row = leader + (lane >> p.log_lanes) * R;
    stride = static_cast<int64_t>(gridDim.x) * LN_BLOCK_WARPS * teams * R;
    col = (lane & ((1 << p.log_lanes) - 1)) * EACH;
    apart = EACH << p.log_lanes;
    N = p.N;
    slots = smem + warp * (WARP_BYTES / 16) + lane;
  }
  __device__ __forceinline__ int valid(int i) const { return max(min(N - col - i * apart, EACH), 0); }
  static __device__ __forceinline__ constexpr int index(int d, int t, int r, int part) {
    return (((d * TENSORS + t) * R + r) * PARTS + part) * 32;
  }
  // Rows `at` .. at + R - 1 of a tensor into set d, zeros behind its last row and
  // column.
  __device__ __forceinline__ void fetch(int M, int d, int t, const void* data, int64_t ld, int64_t at) const {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < PARTS; ++i) {
        const int n = at + r < M ? valid(i) : 0;
        const T* src = static_cast<const T*>(data) + (n > 0 ? (at + r) * ld + col + i * apart : 0);
        ptx::cp_async16(ptx::smem_addr(slots + index(d, t, r, i)), src, static_cast<uint32_t>(n) * sizeof(T));
      }
  }
  __device__ __forceinline__ void take(int d, int t, int r, Eight& v) const {
    Group<T> g;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) g.q[i] = slots[index(d, t, r, i)];
    v.from(g);
  }
  // The same of one row by single elements.
  __device__ __forceinline__ void load(int M, const void* data, int64_t ld, int64_t at, Eight& v) const {
    Group<T> g;
    g.clear();
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
      if (at < M) load_part(static_cast<const T*>(data) + at * ld + col + i * apart, valid(i), false, g.q[i]);
    v.from(g);
  }
  __device__ __forceinline__ void store(void* data, int64_t ld, int64_t at, bool wide, const Eight& v) const {
    Group<T> g;
    float f[8];
    v.to(f);
    g.pack(f);
#pragma unroll
    for (int i = 0; i < PARTS; ++i) store_part(static_cast<T*>(data) + at * ld + col + i * apart, valid(i), wide, g.q[i]);
  }
  // f(value's place among the 8, its column) of the columns in the row.
  template <class F>
  __device__ __forceinline__ void columns(F&& f) const {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j % EACH < valid(j / EACH)) f(j, col + j / EACH * apart + j % EACH);
  }
  __device__ __forceinline__ float squares(const Eight& v, float m) const {
    float f[8], s = 0.0f;
    v.to(f);
    columns([&](int j, int) { s = fmaf(f[j] - m, f[j] - m, s); });
    return s;
  }
  __device__ __forceinline__ void weights(const float* w, float none, Eight& v) const {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = none;
    if (w != nullptr) columns([&](int j, int c) { f[j] = __ldg(w + c); });
    v.from(f);
  }
  // The words of the thread's values in its R rows, as RowPlace::words.
  __device__ __forceinline__ void words(const Dropout& d, uint32_t step, int64_t at, uint32_t (&w)[R][4]) const {
    uint32_t rows[R * PARTS], groups[R * PARTS], all[R * PARTS][4];
#pragma unroll
    for (int i = 0; i < R * PARTS; ++i) {
      rows[i] = static_cast<uint32_t>(at + i / PARTS);
      groups[i] = static_cast<uint32_t>(col + i % PARTS * apart) >> 3;
    }
    drop_words(d, step, rows, groups, all);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (PARTS == 1)
          w[r][j] = all[r][j];
        else
          w[r][j] = ((col + j / 2 * apart) & 4) ? all[2 * r + j / 2][2 + j % 2] : all[2 * r + j / 2][j % 2];
      }
  }
};

template <class T, bool DROP, bool WIDE>
__global__ void __launch_bounds__(32 * LN_BLOCK_WARPS, 2) layer_norm_narrow_kernel(const __grid_constant__ NormParams p) {
  constexpr int R = LN_NARROW_ROWS<T>;
  using Rows = NarrowRows<T, R, 2>;
  extern __shared__ __align__(128) uint4 ln_smem[];
  const Rows at(p, ln_smem);
  auto fetch = [&](int d, int64_t row) {
    if constexpr (WIDE) {
      at.fetch(p.M, d, 0, p.x, p.ld_x, row);
      if (p.other != nullptr) at.fetch(p.M, d, 1, p.other, p.ld_other, row);
      ptx::cp_async_commit();
    }
  };
  fetch(0, at.row);
  fetch(1, at.row + at.stride);
  uint32_t step = 0;
  if constexpr (DROP) step = drop_step(p.drop);
  Eight w, b;
  at.weights(p.w, 1.0f, w);
  at.weights(p.b, 0.0f, b);
  int64_t row = at.row;
  int d = 0;
  for (int64_t leader = at.leader; leader < p.M; leader += at.stride, row += at.stride) {
    Eight h[R];
    float mean[R], square[R];
    uint32_t words[R][4];
    if constexpr (DROP) at.words(p.drop, step, row, words);
    if constexpr (WIDE) ptx::cp_async_wait<1>();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Eight add;
      add.clear();
      if constexpr (WIDE) {
        at.take(d, 0, r, h[r]);
        if (p.other != nullptr) at.take(d, 1, r, add);
      } else {
        at.load(p.M, p.x, p.ld_x, row + r, h[r]);
        if (p.other != nullptr) at.load(p.M, p.other, p.ld_other, row + r, add);
      }
      if constexpr (DROP)
        h[r].drop_onto(add, p.drop, words[r]);
      else
        h[r].plus(add);
      const float2 s = h[r].sum();
      mean[r] = s.x + s.y;
    }
    fetch(d, row + 2 * at.stride);
    d ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) mean[r] = team_sum(mean[r], p.log_lanes) * p.inv_n;
#pragma unroll
    for (int r = 0; r < R; ++r) square[r] = at.squares(h[r], mean[r]);
#pragma unroll
    for (int r = 0; r < R; ++r) square[r] = team_sum(square[r], p.log_lanes);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float rstd = 1.0f / sqrtf(fmaf(square[r], p.inv_n, p.eps));
      if (row + r >= p.M) continue;
      if (at.col == 0) {
        if (p.mean != nullptr) p.mean[row + r] = mean[r];
        if (p.rstd != nullptr) p.rstd[row + r] = rstd;
      }
      if (p.sum != nullptr) at.store(p.sum, p.ld_sum, row + r, WIDE, h[r]);
      h[r].normalise(mean[r], rstd);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[r].v[j] = __ffma2_rn(h[r].v[j], w.v[j], b.v[j]);
      at.store(p.y, p.ld_y, row + r, WIDE, h[r]);
    }
  }
}

// ------------------------------------------------------------------ rows too wide to hold

// A block to a row, which it reads three times forward and twice backward, from
// L2 after the first.  (Forward, h kept in shared memory for the second and third
// time leaves one block to two to an SM: 4096 x 16392 bf16 212 us, 195 read again.)
constexpr int LN_LONG_THREADS = 512;
constexpr int LN_LONG_ROWS = 4;  // of a block at a time, backward

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
    auto read = [&](int g, float (&h)[8]) {
      load_group(static_cast<const T*>(p.x) + row * p.ld_x + g * 8, p.N - g * 8, WIDE, h);
      float r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = 0.0f;
      if (p.other != nullptr)
        load_group(static_cast<const T*>(p.other) + row * p.ld_other + g * 8, p.N - g * 8, WIDE, r);
      if constexpr (DROP) {
        uint32_t w[1][4];
        drop_words(p.drop, step, {static_cast<uint32_t>(row)}, {static_cast<uint32_t>(g)}, w);
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
      read(g, h);  // zeros behind the row's end
#pragma unroll
      for (int j = 0; j < 8; ++j) s += h[j];
    }
    const float mean = block_sum(s, part) * p.inv_n;
    s = 0.0f;
    for (int g = threadIdx.x; g < p.groups; g += LN_LONG_THREADS) {
      const int valid = p.N - g * 8;
      float h[8];
      read(g, h);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < valid) s = fmaf(h[j] - mean, h[j] - mean, s);
    }
    const float rstd = 1.0f / sqrtf(fmaf(block_sum(s, part), p.inv_n, p.eps));
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[row] = mean;
      if (p.rstd != nullptr) p.rstd[row] = rstd;
    }
    for (int g = threadIdx.x; g < p.groups; g += LN_LONG_THREADS) {
      const int valid = p.N - g * 8;
      float h[8], w[8], b[8];
      read(g, h);
      if (p.sum != nullptr) store_group(static_cast<T*>(p.sum) + row * p.ld_sum + g * 8, valid, WIDE, h);
      load_weights(p.w, g * 8, valid, p.wide_w, 1.0f, w);
      load_weights(p.b, g * 8, valid, p.wide_w, 0.0f, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = fmaf((h[j] - mean) * rstd, w[j], b[j]);
      store_group(static_cast<T*>(p.y) + row * p.ld_y + g * 8, valid, WIDE, w);
    }
  }
}

}  // namespace ge
