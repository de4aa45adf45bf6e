// layer_norm.cu -- host side of dropout, layer norm and its backward pass, and
// their kernels.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "host.h"
#include "layer_norm.cuh"
#include "layer_norm_kernels.h"

namespace {

using ge_host::cuda_fail;
using ge_host::fail;
using ge_norm::Choice;
using ge_norm::HELD;
using ge_norm::Kernel;
using ge_norm::LONG;
using ge_norm::NARROW;
using ge_norm::Shape;

// ---------------------------------------------------------------- kernels

// How many pieces of 256 columns a warp holds, how many rows a team works on at
// once, how many teams share a block and whether they share the weights: from
// timing them all at 512 to 14336 columns (one GB300, 537 MB forward, 671 MB
// backward with dropout, unless others are named; the times beside the rules are
// of those).  Few rows: not more than two to an SM, whose latency counts, so many
// warps to a row and nothing staged.
Shape forward_shape(int64_t rows, int64_t cols, int64_t pieces, const Choice& c, int sms) {
  const bool few = rows <= 2 * sms;
  bool staged = c.drop;
  Shape s{HELD, 4, 1, 1, 0, 1, false};
  auto take = [&](int k, int r) {
    s.k = k, s.rows = r;
    s.warps = static_cast<int>((pieces + k - 1) / k);
  };
  auto warps = [&](int n) { s.teams = std::max(1, n / s.warps); };
  // bf16 with a second stream: two pieces and one row make for more teams, but the
  // last warp of a row that ends inside its columns has no staged weights there.
  // With dropout they are taken where every warp is full, or where of four to a warp
  // two or more would be empty, at up to ten pieces (537 MB, two against four): 3 of
  // them 113 us and 91.4, 4 (800 columns) 116 and 95.0, 1024 columns 90.0 and 99.1,
  // 5 (1280) 105.5 and 116, 6 (1400) 103 and 117, 7 (1792) 99.5 and 94.3, 8 (1904)
  // 102 and 95.4, 9 (2304) 99.0 and 107, 10 (2560) 89.6 and 101, 11 (2816) 103 and
  // 94.3, 12 (3000) 104 and 96.2, 13 (3328) 103 and 98.4, 14 (3400) 104 and 108, 15
  // (3840) 103 and 93.3, 16 (4096) 95.0 and 90.7.  Without it: 3 (640) 105 and 98.3,
  // one warp in place of two, 4 (896) 90.0 and 101, 6 (1480) 92.2 and 103, 8 (1992)
  // 93.5 and 97.9, 9 (2304) 93.6 and 90.3, 11 (2816) 92.4 and 89.5, 16 (4000) 91.0 and
  // 88.0, 4096 columns 87.3 and 93.4.
  const bool even = cols % (2 * ge::LN_PIECE) == 0;
  const bool two = c.drop ? pieces <= 10 && (even || pieces % 4 == 1 || pieces % 4 == 2)
                          : pieces <= 16 && (even || (pieces <= 8 && pieces != 3));
  if (!c.wide && (!few || pieces > 2 * ge::LN_MAX_WARPS)) {
    // by words 8 warps to a block: 16384 x 4095 149 us with dropout (fp32 240), 16 151
    // (261); 1777 x 1003 fp32 4 warps 5.6, 16 8.6
    take(4, 1);
    warps(rows > 16 * sms ? 8 : 4);
  } else if (few && pieces <= 2 * ge::LN_MAX_WARPS) {
    take(2, 1);
  } else if (c.f32) {
    // 8192 x 4096: 2 pieces, 2 rows 90.8 us with dropout, 4 and 1 94.9; 13421 x 5000
    // 98.9 and 87.9
    pieces <= 16 ? take(2, 2) : take(4, 1);
    if (pieces <= 16 && (c.drop || !c.add)) warps(16);
  } else if (!c.drop && !c.add) {
    // one stream in: 4096 columns with 2 pieces, 1 row over 75 us, 4 and 2 47.8 (57.1
    // not staged); 512: 46.0 with 2 and 1, over 53 with 4 and 2
    pieces <= 2 ? take(2, 1) : take(4, 2);
    warps(16);
    staged = true;
  } else if (two) {
    take(2, 1);
    warps(c.drop || s.warps <= 4 ? 16 : 8);
  } else {
    // 8192: one team to a block 89.4 us (95.6 with dropout), two that share the
    // weights 100 (94.2)
    take(4, 2);
    if (c.drop) warps(16);
    else if (s.warps <= 2) warps(8);
  }
  // For few rounds staging the weights costs more than their misses in L1 (1777 x
  // 1024 5.9 us staged, 4.9 not).
  s.staged = rows > 16 * sms && (!c.wide || (!c.f32 && staged));
  return s;
}

Shape backward_shape(int64_t rows, int64_t cols, int64_t pieces, const Choice& c, int sms) {
  const bool few = rows <= 2 * sms;
  Shape s{HELD, 4, 1, 1, 0, 1, false};
  auto take = [&](int k) {
    s.k = k;
    s.warps = static_cast<int>((pieces + k - 1) / k);
  };
  if (!c.wide) {
    // by words, with dropout, 4 pieces spill 60 to 148 bytes of registers: 12000 x 4095
    // 203 us with 2, 259 with 4; without 141 and 117
    take(pieces > 2 * ge::LN_MAX_WARPS || (!c.drop && pieces > 2 && rows > 16 * sms) ? 4 : 2);
    if (few) return s;
  } else if (few) {
    take(pieces <= ge::LN_MAX_WARPS ? 1 : pieces <= 2 * ge::LN_MAX_WARPS ? 2 : 4);
    return s;
  } else if (c.f32) {
    // of 235 MB: 1280 columns 1 piece 46.0 us (55.1 with dropout), 2 52.3 (62.9);
    // 4096: 2 pieces 51.0 (61.2), 4 53.1 (63.6); 6000: 65.9 (82.0) and 53.6 (76.0)
    take(pieces <= 5 ? 1 : pieces <= 16 ? 2 : 4);
  } else {
    // 768 columns of 268 MB: 2 pieces 57.2 us (63.9 with dropout), all 3 in a warp 47.2
    // (59.2); 1024: 2 pieces 90.3 (110.4), 4 93.4 (127.8); 4096: 99.5 (120.6) and 89.3
    // (113.5)
    take(pieces == 3 || pieces > 8 ? 4 : 2);
  }
  // 3000 columns: one team of 3 warps to a block 126 us (158 with dropout, and only two
  // blocks to an SM have room for their sums), five 103 (123)
  s.teams = ge::LN_MAX_WARPS / s.warps;
  // A team fewer where `add` is the third stream, more than 176 KB would be on their
  // way to a block (two rows of each team) and 12 warps stay: over many rows of whole
  // 64 bytes the copies then get in each other's way.  Three teams of 4 warps against
  // four, with dropout and without, at 4096 columns 112.2 and 123.8 us, 87.3 and 91.0
  // (67 M elements); 3968 112.8 and 122.7, 87.7 and 90.4; 3776 116.6 and 119.9, 88.8
  // and 89.2.  With less on the way they lose: 3712 118.8 and 117.7, 3456 125.3 and
  // 110.9, 4096 without `add` 100.5 and 92.5.  So do they in rows off 64 bytes (4088
  // 128.4 and 122.3) and in few of them (2929 of 4096 30.2 and 29.0, 7500 of 4000 59.1
  // and 57.2).  Four teams of 3 against five: 3040 111.4 and 122.5, 87.5 and 93.4.
  const int64_t on_the_way = int64_t{2 * 3} * s.teams * cols * static_cast<int64_t>(sizeof(uint16_t));
  if (c.wide && !c.f32 && c.add && on_the_way > 176 * 1024 && cols % 32 == 0 && rows > 64 * sms &&
      (s.teams - 1) * s.warps >= 12)
    --s.teams;
  s.staged = true;  // 4096: 91.5 us, 113.3 from L1
  return s;
}

Shape shape_of(bool backward, int64_t rows, int64_t cols, const Choice& c, int sms) {
  const int64_t groups = (cols + 7) / 8, pieces = (cols + ge::LN_PIECE - 1) / ge::LN_PIECE;
  if (groups <= 32) {
    Shape s{NARROW, 0, 1, 1, 0, 1, false};
    while ((1 << s.log_lanes) < groups) ++s.log_lanes;
    s.rows = backward ? (c.f32 ? ge::LN_NARROW_BACKWARD_ROWS<float> : ge::LN_NARROW_BACKWARD_ROWS<uint16_t>)
                      : (c.f32 ? ge::LN_NARROW_ROWS<float> : ge::LN_NARROW_ROWS<uint16_t>);
    s.teams = ge::LN_BLOCK_WARPS << (5 - s.log_lanes);
    return s;
  }
  if (pieces > 4 * ge::LN_MAX_WARPS) {
    Shape s{LONG, 0, ge::LN_LONG_THREADS / 32, 1, 0, 1, false};
    if (backward) s.rows = static_cast<int>(std::min<int64_t>(ge::LN_LONG_ROWS, std::max<int64_t>(1, rows / (2 * sms))));
    return s;
  }
  Shape s = backward ? backward_shape(rows, cols, pieces, c, sms) : forward_shape(rows, cols, pieces, c, sms);
  // a block to every SM before a second team to a block
  s.teams = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(s.teams, rows / (s.rows * sms))));
  return s;
}

int block_warps(const Shape& s) { return s.form == NARROW ? ge::LN_BLOCK_WARPS : s.warps * s.teams; }

// The ring, and behind it the weights.
size_t shared_bytes(bool backward, const Shape& s, const Kernel& k) {
  return static_cast<size_t>(k.warp_bytes) * block_warps(s) +
         (s.staged ? static_cast<size_t>(backward ? 1 : 2) * s.warps * s.k * ge::LN_PIECE * sizeof(float) : 0);
}

// Fewer teams where a block's rings need that; the weights only where there is
// room beside them.
void fit_shared(bool backward, Shape& s, const Kernel& k) {
  if (shared_bytes(backward, s, k) > ge::LN_MAX_SHARED) s.staged = false;
  while (s.teams > 1 && shared_bytes(backward, s, k) > ge::LN_MAX_SHARED) --s.teams;
}

// Blocks of a kernel resident on an SM of the current device: asked for once and
// kept by what the answer depends on, one word to an entry, so that an entry is
// read and written whole.
gemm_epi_status resident_blocks(int dev, bool backward, const Shape& s, const Choice& c, const Kernel& k, size_t bytes,
                                int* blocks) {
  constexpr size_t ENTRIES = 1024;
  static std::atomic<uint64_t> known[ENTRIES];
  uint64_t key = static_cast<uint64_t>(dev) << 1 | static_cast<uint64_t>(backward);
  for (const int part : {c.index(), s.index(), s.warps, block_warps(s), s.rows, static_cast<int>(bytes / 1024)})
    key = key << 8 | static_cast<uint64_t>(part);
  key = key << 1 | 1;  // an empty entry is zero
  std::atomic<uint64_t>& at = known[(key * 0x9E3779B97F4A7C15u >> 32) % ENTRIES];
  const uint64_t entry = at.load(std::memory_order_acquire);
  if (entry >> 7 == key) {
    *blocks = static_cast<int>(entry & 127);
    return GEMM_EPI_OK;
  }
  const void* fn = reinterpret_cast<const void*>(k.fn);
  // the most that a block may take, so that no other thread's call lowers it
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       s.form == HELD ? ge::LN_MAX_SHARED : static_cast<int>(bytes));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  int n = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, 32 * block_warps(s), bytes);
  if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor");
  if (n < 1) return fail(GEMM_EPI_ERR_CUDA, "a layer norm kernel does not fit an SM");
  at.store(key << 7 | static_cast<uint64_t>(n), std::memory_order_release);
  *blocks = n;
  return GEMM_EPI_OK;
}

struct DropoutKernel {
  void (*fn)(ge::DropoutParams);
  int span;  // columns of a warp's share of a row, or of a thread's
  bool narrow;
  int bytes;  // dynamic shared memory
};

template <class T, int K>
DropoutKernel dropout_kernel_of(bool wide) {
  if (wide) return {ge::dropout_kernel<T, K, true>, K * ge::LN_PIECE, false, 0};
  return {ge::dropout_kernel<T, K, false>, K * ge::LN_PIECE, false,
          ge::DO_THREADS / 32 * (ge::WordRing<T, K, 2, 1>::WARP_BYTES + 1024)};
}

template <class T>
DropoutKernel dropout_kernel_of(int64_t cols, bool wide) {
  if (cols <= ge::LN_PIECE) return {ge::dropout_narrow_kernel<T>, 8, true, 0};
  // as many pieces to a warp as leave few of a row's last share's empty
  const int64_t pieces = (cols + ge::LN_PIECE - 1) / ge::LN_PIECE;
  auto few_empty = [&](int64_t k) { return ((pieces + k - 1) / k * k - pieces) * 8 <= pieces; };
  if constexpr (sizeof(T) == 2)
    if (few_empty(4)) return dropout_kernel_of<T, 4>(wide);
  return few_empty(2) ? dropout_kernel_of<T, 2>(wide) : dropout_kernel_of<T, 1>(wide);
}

// Partial sums of dw and db: the most blocks a backward pass has, two to an SM.
constexpr int MOST_PARTIALS = 304;

// ---------------------------------------------------------------- checks

constexpr int64_t LIM = 0x7FFFFFFF;
constexpr int64_t MOST_COLUMNS = LIM - 4095;  // a column past the end of the last pieces is still an int

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

struct Rows {
  const void* data;
  int64_t ld;
  const char* name;
};

// The sizes, tensors and dropout of a call, with what 16-byte accesses serve.
struct Checked {
  int64_t M, N;
  size_t size;
  bool wide_in = true, wide_out = true;

  gemm_epi_status sizes(int64_t rows, int64_t cols, int32_t type) {
    if (rows < 0 || rows > LIM) return fail(GEMM_EPI_ERR_INVALID_VALUE, "M must be in [0, 2^31)");
    if (cols < 1 || cols > MOST_COLUMNS) return fail(GEMM_EPI_ERR_INVALID_VALUE, "N must be in [1, 2^31 - 4096]");
    if (type != GEMM_EPI_TYPE_BF16 && type != GEMM_EPI_TYPE_F32)
      return fail(GEMM_EPI_ERR_UNSUPPORTED, "the tensors must be BF16 or F32 (type %d)", type);
    M = rows, N = cols;
    size = type == GEMM_EPI_TYPE_F32 ? 4 : 2;
    return GEMM_EPI_OK;
  }
  gemm_epi_status tensor(const Rows& t, bool output) {
    if (!t.data) return fail(GEMM_EPI_ERR_INVALID_VALUE, "%s is NULL", t.name);
    if (!aligned(t.data, size)) return fail(GEMM_EPI_ERR_MISALIGNED, "%s is not aligned to its element size", t.name);
    // the rows of an input may be the same memory (stride 0), those of an output not
    if (M > 1 && (t.ld < 0 || t.ld > (int64_t(1) << 40)))
      return fail(GEMM_EPI_ERR_INVALID_VALUE, "the row stride of %s is out of range", t.name);
    if (M > 1 && output && t.ld < N) return fail(GEMM_EPI_ERR_INVALID_VALUE, "row stride of %s < N", t.name);
    if (!aligned(t.data, 16) || (M > 1 && t.ld * static_cast<int64_t>(size) % 16 != 0))
      (output ? wide_out : wide_in) = false;
    return GEMM_EPI_OK;
  }
  // An output is written over an input element by element or not at all.
  gemm_epi_status in_place(const Rows& out, const Rows& in) const {
    if (out.data && out.data == in.data && M > 1 && out.ld != in.ld)
      return fail(GEMM_EPI_ERR_INVALID_VALUE, "%s starts where %s does but has another row stride", out.name, in.name);
    return GEMM_EPI_OK;
  }
};

gemm_epi_status check_vector(const void* v, const char* name) {
  return aligned(v, 4) ? GEMM_EPI_OK : fail(GEMM_EPI_ERR_MISALIGNED, "%s must be 4-byte aligned", name);
}

gemm_epi_status check_mask(const gemm_epi_mask& d, ge::Dropout* out) {
  std::memset(out, 0, sizeof *out);
  if (d.threshold < 0 || d.threshold > 65536)
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "the dropout threshold must be in [0, 65536] (got %d)", d.threshold);
  if (d.threshold == 0) return GEMM_EPI_OK;
  if (!d.step) return fail(GEMM_EPI_ERR_INVALID_VALUE, "the dropout step is NULL");
  if (!aligned(d.step, 8)) return fail(GEMM_EPI_ERR_MISALIGNED, "the dropout step must be 8-byte aligned");
  *out = ge::dropout_of(d);
  return GEMM_EPI_OK;
}

// ---------------------------------------------------------------- launches

// What the sum of the blocks' partial sums has to know.
struct Launched {
  int blocks, width;
  bool staged;
};

gemm_epi_status launch_norm(bool backward, ge::NormParams& p, Choice c, int64_t most_blocks, cudaStream_t st, Launched* launched) {
  int dev = 0, sms = 0, resident = 0;
  gemm_epi_status s = ge_host::device_sms(&dev, &sms);
  if (s) return s;
  c.drop = p.drop.step != nullptr;
  c.add = backward ? p.add != nullptr : p.other != nullptr;
  Shape shape = shape_of(backward, p.M, p.N, c, sms);
  const Kernel k = backward ? ge_norm::backward_kernel(shape, c) : ge_norm::forward_kernel(shape, c);
  if (shape.form == HELD) fit_shared(backward, shape, k);
  const size_t bytes = (shared_bytes(backward, shape, k) + 1023) / 1024 * 1024;
  if ((s = resident_blocks(dev, backward, shape, c, k, bytes, &resident))) return s;
  const int64_t rows = static_cast<int64_t>(shape.teams) * shape.rows;  // a block works on at once
  int64_t blocks = std::min<int64_t>((p.M + rows - 1) / rows, static_cast<int64_t>(sms) * resident);
  blocks = std::min(blocks, most_blocks);
  p.warps = shape.warps;
  p.log_lanes = shape.log_lanes;
  p.staged = shape.staged;
  p.rows = shape.rows;
  k.fn<<<static_cast<unsigned>(blocks), static_cast<unsigned>(32 * block_warps(shape)), bytes, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  *launched = {static_cast<int>(blocks), shape.form == HELD ? shape.warps * shape.k * ge::LN_PIECE : static_cast<int>(ge::partial_width(p.N)),
               shape.form == HELD && !c.f32};
  return e == cudaSuccess ? GEMM_EPI_OK : cuda_fail(e, "launch of the layer norm kernel");
}

void set_sizes(ge::NormParams& p, const Checked& c) {
  std::memset(&p, 0, sizeof p);
  p.M = static_cast<int32_t>(c.M);
  p.N = static_cast<int32_t>(c.N);
  p.groups = static_cast<int32_t>((c.N + 7) / 8);
  p.inv_n = 1.0f / static_cast<float>(c.N);
}

}  // namespace

extern "C" {

gemm_epi_status gemm_epi_dropout(const gemm_epi_dropout_args* a, void* stream) {
  ge_host::clear_error();
  if (!a) return fail(GEMM_EPI_ERR_INVALID_VALUE, "args must not be NULL");
  Checked c;
  gemm_epi_status s = c.sizes(a->M, a->N, a->type);
  if (s) return s;
  ge::DropoutParams p;
  std::memset(&p, 0, sizeof p);
  if ((s = check_mask(a->mask, &p.drop))) return s;
  const Rows x{a->x, a->ld_x, "x"}, residual{a->residual, a->ld_residual, "residual"}, y{a->y, a->ld_y, "y"};
  if (c.M > 0) {
    if ((s = c.tensor(x, false)) || (s = c.tensor(y, true)) || (s = c.in_place(y, x))) return s;
    if (a->residual && ((s = c.tensor(residual, false)) || (s = c.in_place(y, residual)))) return s;
  }
  int dev = 0, sms = 0;
  if ((s = ge_host::device_sms(&dev, &sms))) return s;
  if (c.M == 0) return GEMM_EPI_OK;
  p.M = static_cast<int32_t>(c.M);
  p.N = static_cast<int32_t>(c.N);
  p.x = a->x, p.ld_x = a->ld_x;
  p.residual = a->residual, p.ld_residual = a->ld_residual;
  p.y = a->y, p.ld_y = a->ld_y;
  p.wide_in = c.wide_in, p.wide_out = c.wide_out;
  const bool wide = c.wide_in && c.wide_out;
  const DropoutKernel k = c.size == 4 ? dropout_kernel_of<float>(c.N, wide) : dropout_kernel_of<uint16_t>(c.N, wide);
  p.spans = static_cast<int32_t>((c.N + k.span - 1) / k.span);
  p.total = c.M * p.spans;
  const int64_t each = k.narrow ? ge::DO_THREADS : ge::DO_THREADS / 32;  // spans of a block
  const int64_t blocks = std::min<int64_t>((p.total + each - 1) / each, static_cast<int64_t>(sms) * ge::DO_BLOCKS);
  p.step_rows = blocks * each / p.spans;
  p.step_spans = static_cast<int32_t>(blocks * each % p.spans);
  k.fn<<<static_cast<unsigned>(blocks), ge::DO_THREADS, static_cast<size_t>(k.bytes), static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? GEMM_EPI_OK : cuda_fail(e, "launch of the dropout kernel");
}

gemm_epi_status gemm_epi_layer_norm(const gemm_epi_layer_norm_args* a, void* stream) {
  ge_host::clear_error();
  if (!a) return fail(GEMM_EPI_ERR_INVALID_VALUE, "args must not be NULL");
  Checked c;
  gemm_epi_status s = c.sizes(a->M, a->N, a->type);
  if (s) return s;
  if (!(a->eps >= 0.0f) || !std::isfinite(a->eps))
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "eps must be finite and >= 0");
  ge::NormParams p;
  set_sizes(p, c);
  if ((s = check_mask(a->mask, &p.drop))) return s;
  const Rows x{a->x, a->ld_x, "x"}, residual{a->residual, a->ld_residual, "residual"}, y{a->y, a->ld_y, "y"},
      sum{a->sum, a->ld_sum, "sum"};
  if (c.M > 0) {
    if ((s = c.tensor(x, false)) || (s = c.tensor(y, true)) || (s = c.in_place(y, x))) return s;
    if (a->residual && ((s = c.tensor(residual, false)) || (s = c.in_place(y, residual)))) return s;
    if (a->sum && ((s = c.tensor(sum, true)) || (s = c.in_place(sum, x)) || (s = c.in_place(sum, residual)))) return s;
    if (a->sum && a->sum == a->y) return fail(GEMM_EPI_ERR_INVALID_VALUE, "sum and y are the same buffer");
  }
  if ((s = check_vector(a->w, "w")) || (s = check_vector(a->b, "b")) || (s = check_vector(a->mean, "mean")) ||
      (s = check_vector(a->rstd, "rstd")))
    return s;
  if (a->mean && a->mean == a->rstd) return fail(GEMM_EPI_ERR_INVALID_VALUE, "mean and rstd are the same buffer");
  int dev = 0, sms = 0;
  if ((s = ge_host::device_sms(&dev, &sms))) return s;
  if (c.M == 0) return GEMM_EPI_OK;
  p.x = a->x, p.ld_x = a->ld_x;
  p.other = a->residual, p.ld_other = a->ld_residual;
  p.y = a->y, p.ld_y = a->ld_y;
  p.sum = a->sum, p.ld_sum = a->ld_sum;
  p.w = a->w, p.b = a->b;
  p.mean = a->mean, p.rstd = a->rstd;
  p.eps = a->eps;
  p.wide_w = aligned(a->w, 16) && aligned(a->b, 16);
  const Choice choice{c.size == 4, false, false, c.wide_in && c.wide_out && p.wide_w};
  Launched launched;
  return launch_norm(false, p, choice, LIM, static_cast<cudaStream_t>(stream), &launched);
}

gemm_epi_status gemm_epi_layer_norm_backward(const gemm_epi_layer_norm_bwd_args* a, void* stream) {
  ge_host::clear_error();
  if (!a) return fail(GEMM_EPI_ERR_INVALID_VALUE, "args must not be NULL");
  Checked c;
  gemm_epi_status s = c.sizes(a->M, a->N, a->type);
  if (s) return s;
  ge::NormParams p;
  set_sizes(p, c);
  if ((s = check_mask(a->mask, &p.drop))) return s;
  const Rows dy{a->dy, a->ld_dy, "dy"}, x{a->x, a->ld_x, "x"}, add{a->add, a->ld_add, "add"}, dx{a->dx, a->ld_dx, "dx"},
      dr{a->d_residual, a->ld_d_residual, "d_residual"};
  const bool wants_dw = a->dw || a->db;
  const bool work = c.M > 0 && (a->dx || a->d_residual || wants_dw);
  if (work) {
    if ((s = c.tensor(dy, false)) || (s = c.tensor(x, false))) return s;
    if (a->add && (s = c.tensor(add, false))) return s;
    for (const Rows& out : {dx, dr})
      if (out.data && ((s = c.tensor(out, true)) || (s = c.in_place(out, dy)) || (s = c.in_place(out, x)) ||
                       (s = c.in_place(out, add))))
        return s;
    if (a->dx && a->dx == a->d_residual)
      return fail(GEMM_EPI_ERR_INVALID_VALUE, "dx and d_residual are the same buffer");
    if (!a->mean || !a->rstd) return fail(GEMM_EPI_ERR_INVALID_VALUE, "mean and rstd must not be NULL");
  }
  for (const auto& v : {Rows{a->w, 0, "w"}, Rows{a->mean, 0, "mean"}, Rows{a->rstd, 0, "rstd"}, Rows{a->dw, 0, "dw"},
                        Rows{a->db, 0, "db"}})
    if ((s = check_vector(v.data, v.name))) return s;
  if (a->dw && a->dw == a->db) return fail(GEMM_EPI_ERR_INVALID_VALUE, "dw and db are the same buffer");
  const size_t ws = gemm_epi_layer_norm_backward_workspace_size(a->N);
  if (wants_dw && work && (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < ws))
    return fail(GEMM_EPI_ERR_WORKSPACE, "workspace must be 16-byte aligned and hold %zu bytes (got %zu)", ws,
                a->workspace ? a->workspace_bytes : static_cast<size_t>(0));
  int dev = 0, sms = 0;
  if ((s = ge_host::device_sms(&dev, &sms))) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (!work) {
    // nothing to sum: the weight's and the bias's gradients are zero
    for (float* d : {a->dw, a->db})
      if (d && (e = cudaMemsetAsync(d, 0, sizeof(float) * static_cast<size_t>(c.N), st)) != cudaSuccess)
        return cuda_fail(e, "cudaMemsetAsync of dw and db");
    return GEMM_EPI_OK;
  }
  p.x = a->x, p.ld_x = a->ld_x;
  p.other = a->dy, p.ld_other = a->ld_dy;
  p.add = a->dx || a->d_residual ? a->add : nullptr, p.ld_add = a->ld_add;
  p.y = a->dx, p.ld_y = a->ld_dx;
  p.sum = a->d_residual, p.ld_sum = a->ld_d_residual;
  p.w = a->w;
  p.mean = const_cast<float*>(a->mean), p.rstd = const_cast<float*>(a->rstd);
  p.partials = wants_dw ? static_cast<float*>(a->workspace) : nullptr;
  p.wide_w = aligned(a->w, 16);
  const Choice choice{c.size == 4, false, false, c.wide_in && c.wide_out && p.wide_w};
  Launched launched;
  if ((s = launch_norm(true, p, choice, MOST_PARTIALS, st, &launched))) return s;
  if (!wants_dw) return GEMM_EPI_OK;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>((launched.width + 127) / 128), 2);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  std::memset(&attr, 0, sizeof attr);
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, ge_norm::weight_grad_kernel, static_cast<const float*>(p.partials), launched.blocks,
                         launched.width, static_cast<int>(launched.staged), p.N, a->dw, a->db);
  return e == cudaSuccess ? GEMM_EPI_OK : cuda_fail(e, "launch of the weight gradient kernel");
}

size_t gemm_epi_layer_norm_backward_workspace_size(int64_t N) {
  if (N < 1 || N > MOST_COLUMNS) return 0;
  // rows held by warps: up to three pieces more than the row has
  const int64_t width = ge::partial_width(N) + (N <= ge::LN_PIECE ? 0 : 3 * ge::LN_PIECE);
  return static_cast<size_t>(MOST_PARTIALS) * 2 * static_cast<size_t>(width) * sizeof(float);
}

}  // extern "C"
