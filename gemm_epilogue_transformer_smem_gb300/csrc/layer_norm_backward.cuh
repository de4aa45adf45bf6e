// layer_norm_backward.cuh -- the backward pass of layer_norm.cuh.
#pragma once

#include "layer_norm.cuh"

namespace ge {

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
  ptx::launch_dependents();  // the sum of the partial sums, once there is room for it
  constexpr int DEPTH = LN_BACKWARD_DEPTH<T>;
  using Ring = std::conditional_t<WIDE, RowRing<T, K, ADD ? 3 : 2, DEPTH>, WordRing<T, K, ADD ? 3 : 2, DEPTH>>;
  constexpr int BATCH = K % 2 == 0 ? 2 : K;
  extern __shared__ __align__(128) uint4 ln_smem[];
  __shared__ __align__(16) float2 part[2][LN_MAX_WARPS + 3];  // a warp's sums of a and a n
  const Teams<K> teams(p);
  const int warp = teams.warp_in_team(p);
  const RowPlace<T, K> place(p.N, warp * K * LN_PIECE);
  const Ring ring(ln_smem, teams.warp);
  uint4* staging = ln_smem + (blockDim.x >> 5) * (Ring::WARP_BYTES / 16) + teams.warp * 64;  // by words: the warp's 1 KB
  const int begin = WIDE ? place.col : warp * K * LN_PIECE;
  const int count = min(max(p.N - warp * K * LN_PIECE, 0), K * LN_PIECE);  // of the warp's columns in the row
  const uint32_t rows = static_cast<uint32_t>(p.M), stride = static_cast<uint32_t>(teams.stride);
  // Addresses are worked out where they are needed: kept, they would cost 20 of
  // the 128 registers, of which the sums of dw and db take 64 at K = 4.
  auto at = [&](const void* data, int64_t ld, uint32_t row) { return static_cast<const T*>(data) + row * ld + begin; };
  auto fetch = [&](int d, uint32_t row) {
    if (row < rows) {
      if constexpr (WIDE) {
        ring.fetch(d, 0, at(p.other, p.ld_other, row), place);
        ring.fetch(d, 1, at(p.x, p.ld_x, row), place);
        if constexpr (ADD) ring.fetch(d, 2, at(p.add, p.ld_add, row), place);
      } else {
        ring.fetch(d, 0, at(p.other, p.ld_other, row), count);
        ring.fetch(d, 1, at(p.x, p.ld_x, row), count);
        if constexpr (ADD) ring.fetch(d, 2, at(p.add, p.ld_add, row), count);
      }
    }
    ptx::cp_async_commit();
  };
  if constexpr (WIDE) {
    if (!place.full) ring.clear(place, 3);
  }
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) fetch(d, static_cast<uint32_t>(teams.first) + d * stride);
  uint32_t step = 0;
  if constexpr (DROP) step = drop_step(p.drop);
  const float* weights = nullptr;  // this thread's, staged
  if (p.staged) {
    float* to = reinterpret_cast<float*>(ln_smem + (blockDim.x >> 5) * (HELD_WARP_BYTES<Ring, WIDE> / 16));
    stage_weights<T>(to, p.w, p.N, teams.width, 1.0f);
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
        ring.take(d, 0, k, at(p.other, p.ld_other, row), place, g);
        ring.take(d, 1, k, at(p.x, p.ld_x, row), place, n);
      }
      n.normalise(mean, rstd);
    };
    // f(k, which of its columns are in the row, weights) of the pieces
    auto pieces = [&](auto&& f) {
      auto staged = [&](auto part) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          Eight w;
          staged_weights(weights, k, w);
          f(k, part, w);
        }
      };
      if (WIDE && (place.full || place.whole) && weights != nullptr) {
        staged(std::integral_constant<int, LN_WHOLE>{});
      } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (WIDE ? place.valid(k, 0) <= 0 : count <= k * LN_PIECE) continue;  // by words: the warp as one
          Eight w;
          if (weights != nullptr)
            staged_weights(weights, k, w);
          else
            place.weights(p.w, k, WIDE || p.wide_w, 1.0f, w);
          f(k, std::integral_constant<int, LN_ANY>{}, w);
        }
      }
    };
    ptx::cp_async_wait<DEPTH - 1>();
    if constexpr (!WIDE) __syncwarp();
    float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
    pieces([&](int k, auto, const Eight& w) {
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
        for (int i0 = 0; i0 < p.warps; i0 += 4) {
#pragma unroll
          for (int i = i0; i < i0 + 4; ++i) {  // reads side by side; the last ones may be another team's
            const float2 v = theirs[i];
            m1 += i < p.warps ? v.x : 0.0f;
            m2 += i < p.warps ? v.y : 0.0f;
          }
        }
        parity ^= 1;
      }
      m1 *= p.inv_n;
      m2 *= p.inv_n;
      uint32_t words[BATCH][4];
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
      pieces([&](int k, auto part, const Eight& w) {
        if constexpr (DROP) {
          if (k % BATCH == 0) place.words(p.drop, step, row, k, words);
        }
        Eight g, n, a;
        take(k, g, n);
        a.clear();
        if constexpr (ADD) {
          if constexpr (WIDE)
            ring.take(d, 2, k, a);
          else
            ring.take(d, 2, k, at(p.add, p.ld_add, row), place, a);
        }
        norm_gradient(g, n, w, a, rstd, m1, m2);
        if (p.sum != nullptr) store(sum, k, part, g);
        if constexpr (DROP) g.drop(p.drop, words[k % BATCH]);
        if (p.y != nullptr) store(y, k, part, g);
      });
    }
    if constexpr (!WIDE) __syncwarp();
    fetch(d, row + DEPTH * stride);
    d = d + 1 == DEPTH ? 0 : d + 1;
  }
  if (p.partials == nullptr) return;
  ptx::cp_async_wait<0>();
  // In the order of the staged weights, [2][width] of each block: 16 bytes of
  // each lane side by side.
  const int mine = warp * K * LN_PIECE + (threadIdx.x & 31) * 4;
  auto put = [&](float* to) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float4* at_w = reinterpret_cast<float4*>(to + mine + k * LN_PIECE + i * (LN_PIECE / 2));
        float4* at_b = reinterpret_cast<float4*>(to + teams.width + mine + k * LN_PIECE + i * (LN_PIECE / 2));
        *at_w = make_float4(dw[k].v[2 * i].x, dw[k].v[2 * i].y, dw[k].v[2 * i + 1].x, dw[k].v[2 * i + 1].y);
        *at_b = make_float4(db[k].v[2 * i].x, db[k].v[2 * i].y, db[k].v[2 * i + 1].x, db[k].v[2 * i + 1].y);
      }
  };
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * teams.width;
  if (teams.count == 1) {
    put(out);
    return;
  }
  float* shared = reinterpret_cast<float*>(ln_smem);  // [team][2][width]: no more than the ring
  __syncthreads();                                    // whose slots are read
  put(shared + teams.team * 2 * teams.width);
  __syncthreads();
  for (int i = threadIdx.x; i < teams.width / 2; i += blockDim.x) {
    float4 t = reinterpret_cast<const float4*>(shared)[i];
    for (int v = 1; v < teams.count; ++v) {
      const float4 q = reinterpret_cast<const float4*>(shared)[v * (teams.width / 2) + i];
      t.x += q.x, t.y += q.y, t.z += q.z, t.w += q.w;
    }
    reinterpret_cast<float4*>(out)[i] = t;
  }
}

template <class T, bool DROP, bool WIDE>
__global__ void __launch_bounds__(32 * LN_BLOCK_WARPS, 2)
    layer_norm_backward_narrow_kernel(const __grid_constant__ NormParams p) {
  ptx::launch_dependents();
  constexpr int R = LN_NARROW_BACKWARD_ROWS<T>;
  using Rows = NarrowRows<T, R, 3>;
  extern __shared__ __align__(128) uint4 ln_smem[];
  __shared__ float shared[LN_BLOCK_WARPS][2][LN_PIECE];
  const Rows at(p, ln_smem);
  float next_mean[R], next_rstd[R];
  auto fetch = [&](int d, int64_t row) {
    if constexpr (WIDE) {
      at.fetch(p.M, d, 0, p.other, p.ld_other, row);
      at.fetch(p.M, d, 1, p.x, p.ld_x, row);
      if (p.add != nullptr) at.fetch(p.M, d, 2, p.add, p.ld_add, row);
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
  at.weights(p.w, 1.0f, w);
  dw.clear(), db.clear();
  int64_t row = at.row;
  int d = 0;
  for (int64_t leader = at.leader; leader < p.M; leader += at.stride, row += at.stride) {
    Eight g[R], n[R];
    float m1[R], m2[R], rstd[R];
    uint32_t words[R][4];
    if constexpr (DROP) at.words(p.drop, step, row, words);
    if constexpr (WIDE) ptx::cp_async_wait<1>();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if constexpr (WIDE) {
        at.take(d, 0, r, g[r]);
        at.take(d, 1, r, n[r]);
      } else {
        at.load(p.M, p.other, p.ld_other, row + r, g[r]);
        at.load(p.M, p.x, p.ld_x, row + r, n[r]);
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
          at.load(p.M, p.add, p.ld_add, row + r, add);
      }
      if (row + r >= p.M) continue;
      norm_gradient(g[r], n[r], w, add, rstd[r], m1[r], m2[r]);
      if (p.sum != nullptr) at.store(p.sum, p.ld_sum, row + r, WIDE, g[r]);
      if constexpr (DROP) g[r].drop(p.drop, words[r]);
      if (p.y != nullptr) at.store(p.y, p.ld_y, row + r, WIDE, g[r]);
    }
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
  for (int j = 0; j < 8; ++j)
    for (int s = 1 << p.log_lanes; s < 32; s <<= 1) {
      a[j] += __shfl_xor_sync(0xffffffffu, a[j], s);
      b[j] += __shfl_xor_sync(0xffffffffu, b[j], s);
    }
  if (lane >> p.log_lanes == 0)
    at.columns([&](int j, int col) {
      shared[warp][0][col] = a[j];
      shared[warp][1][col] = b[j];
    });
  __syncthreads();
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * LN_PIECE;
  for (int i = threadIdx.x; i < 2 * LN_PIECE; i += blockDim.x) {
    const int which = i / LN_PIECE, col = i % LN_PIECE;
    float t = 0.0f;
#pragma unroll
    for (int v = 0; v < LN_BLOCK_WARPS; ++v) t += col < p.N ? shared[v][which][col] : 0.0f;
    out[i] = t;
  }
}

// dw (blockIdx.y 0) and db (1): the sum of the blocks' partial sums, [2][width]
// each, in a fixed order.  A block to 128 columns, 32 of its threads' rows side
// by side.  staged: the columns lie as stage_weights<uint16_t> puts them.
__global__ void __launch_bounds__(1024) layer_norm_weight_grad_kernel(const float* partials, int blocks, int width,
                                                                      int staged, int N, float* dw, float* db) {
  __shared__ float4 part[32][32];
  ptx::wait_dependencies();  // launched beside the backward kernel's end
  float* dst = blockIdx.y == 0 ? dw : db;
  if (dst == nullptr) return;
  const int at = (blockIdx.x * 32 + threadIdx.x) * 4;
  const float* src = partials + static_cast<int64_t>(blockIdx.y) * width + at;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int r = threadIdx.y; r < blocks; r += 32) {
    const float4 q = __ldcg(reinterpret_cast<const float4*>(src + static_cast<int64_t>(r) * 2 * width));
    sum.x += q.x, sum.y += q.y, sum.z += q.z, sum.w += q.w;
  }
  part[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0) {
#pragma unroll
    for (int r = 1; r < 32; ++r) {
      const float4 q = part[r][threadIdx.x];
      sum.x += q.x, sum.y += q.y, sum.z += q.z, sum.w += q.w;
    }
    const int col = staged ? (at & ~(LN_PIECE - 1)) + (at >> 2 & 31) * 8 + (at >> 7 & 1) * 4 : at;
    if (col < N) dst[col] = sum.x;
    if (col + 1 < N) dst[col + 1] = sum.y;
    if (col + 2 < N) dst[col + 2] = sum.z;
    if (col + 3 < N) dst[col + 3] = sum.w;
  }
}

// ------------------------------------------------------------------ rows too wide to hold

// A block takes up to four rows at a time: first the two sums of each, then,
// column by column, the gradients of all four, read again from L2 (304 blocks'
// four rows of 16392 bf16 columns are 80 of its 126 MB).  The sums over rows are
// kept in the block's partials themselves, each column by the thread that works
// on it every time.
template <class T, bool DROP, bool WIDE>
__global__ void __launch_bounds__(LN_LONG_THREADS) layer_norm_backward_long_kernel(const __grid_constant__ NormParams p) {
  ptx::launch_dependents();
  constexpr int R = LN_LONG_ROWS;
  __shared__ float part[LN_LONG_THREADS / 32];
  __shared__ float stats[R][4];  // mean, rstd and the two means
  uint32_t step = 0;
  if constexpr (DROP) step = drop_step(p.drop);
  const int64_t width = partial_width(p.N);
  float* sums = p.partials == nullptr ? nullptr : p.partials + static_cast<int64_t>(blockIdx.x) * 2 * width;
  const bool wants_g = p.y != nullptr || p.sum != nullptr;
  auto load = [&](int64_t row, int g, float mean, float rstd, float (&dy)[8], float (&n)[8]) {
    load_group(static_cast<const T*>(p.other) + row * p.ld_other + g * 8, p.N - g * 8, WIDE, dy);
    load_group(static_cast<const T*>(p.x) + row * p.ld_x + g * 8, p.N - g * 8, WIDE, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) n[j] = (n[j] - mean) * rstd;
  };
  bool first = true;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.rows; row0 < p.M; row0 += static_cast<int64_t>(gridDim.x) * p.rows) {
    const int rows = static_cast<int>(min(static_cast<int64_t>(p.rows), p.M - row0));
    for (int r = 0; r < rows; ++r) {
      const float mean = __ldg(p.mean + row0 + r), rstd = __ldg(p.rstd + row0 + r);
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll 2
      for (int g = threadIdx.x; wants_g && g < p.groups; g += LN_LONG_THREADS) {
        float dy[8], n[8], w[8];
        load(row0 + r, g, mean, rstd, dy, n);  // dy is zero behind the row's end
        load_weights(p.w, g * 8, p.N - g * 8, p.wide_w, 1.0f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float a = dy[j] * w[j];
          s1 += a;
          s2 = fmaf(a, n[j], s2);
        }
      }
      s1 = block_sum(s1, part) * p.inv_n;
      s2 = block_sum(s2, part) * p.inv_n;
      if (threadIdx.x == 0) stats[r][0] = mean, stats[r][1] = rstd, stats[r][2] = s1, stats[r][3] = s2;
    }
    __syncthreads();
    for (int g = threadIdx.x; g < p.groups; g += LN_LONG_THREADS) {
      const int valid = p.N - g * 8;
      float w[8], dw[8], db[8];
      load_weights(p.w, g * 8, valid, p.wide_w, 1.0f, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[j] = db[j] = 0.0f;
      for (int r = 0; r < rows; ++r) {
        const int64_t row = row0 + r;
        const float rstd = stats[r][1], m1 = stats[r][2], m2 = stats[r][3];
        float dy[8], n[8];
        load(row, g, stats[r][0], rstd, dy, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw[j] = fmaf(dy[j], n[j], dw[j]);
          db[j] += dy[j];
          dy[j] = rstd * (fmaf(dy[j], w[j], -m1) - n[j] * m2);
        }
        if (p.add != nullptr && wants_g) {
          load_group(static_cast<const T*>(p.add) + row * p.ld_add + g * 8, valid, WIDE, n);
#pragma unroll
          for (int j = 0; j < 8; ++j) dy[j] += n[j];
        }
        if (p.sum != nullptr) store_group(static_cast<T*>(p.sum) + row * p.ld_sum + g * 8, valid, WIDE, dy);
        if (p.y != nullptr) {
          if constexpr (DROP) {
            uint32_t words[1][4];
            drop_words(p.drop, step, {static_cast<uint32_t>(row)}, {static_cast<uint32_t>(g)}, words);
#pragma unroll
            for (int j = 0; j < 8; ++j) dy[j] = drop_keeps(words[0], j, p.drop.above) ? dy[j] * p.drop.scale : 0.0f;
          }
          store_group(static_cast<T*>(p.y) + row * p.ld_y + g * 8, valid, WIDE, dy);
        }
      }
      if (sums != nullptr) {
        float* at[2] = {sums + g * 8, sums + width + g * 8};  // whole groups: the width is in pieces
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float4* q = reinterpret_cast<float4*>(at[i / 2]) + i % 2;
          const float* v = (i < 2 ? dw : db) + i % 2 * 4;
          float4 t = first ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : *q;
          t.x += v[0], t.y += v[1], t.z += v[2], t.w += v[3];
          *q = t;
        }
      }
    }
    first = false;
    __syncthreads();  // the statistics are read
  }
}

}  // namespace ge
