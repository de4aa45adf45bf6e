// layer_norm.cu -- host side of dropout, layer norm and its backward pass, and
// their kernels.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "host.h"
#include "layer_norm.cuh"

namespace {

using ge_host::cuda_fail;
using ge_host::fail;

enum Pass { FORWARD = 0, BACKWARD = 1 };

// ---------------------------------------------------------------- kernels

// How a row's groups of 8 columns are dealt out.
struct Shape {
  int k;          // groups per thread
  int log_lanes;  // teams within a warp: threads of a team
  int threads;    // of a block
  bool block;     // the team is the block
  bool wide_row;  // too wide to hold: the re-reading kernels
};

Shape shape_of(int pass, int groups) {
  Shape s{1, 5, 32 * ge::LN_WARP_TEAMS, false, false};
  if (groups <= 32) {
    s.log_lanes = 0;
    while ((1 << s.log_lanes) < groups) ++s.log_lanes;
    return s;
  }
  if (pass == FORWARD && groups <= 128) {
    s.k = groups <= 64 ? 2 : 4;
    return s;
  }
  s.block = true;
  if (groups > ge::LN_MAX_GROUPS) {
    s.wide_row = true;
    s.threads = ge::LN_LONG_THREADS;
    return s;
  }
  s.k = pass == BACKWARD && groups <= 256 ? 1 : groups <= 1024 ? 2 : 4;
  s.threads = 32 * ((groups + 32 * s.k - 1) / (32 * s.k));
  return s;
}

struct Kernel {
  void (*fn)(ge::NormParams);
  int ring_bytes;
};

template <class T, bool DROP, int K, bool BLOCK>
Kernel kernel_of(int pass, int threads) {
  if (pass == FORWARD) return {ge::layer_norm_kernel<T, DROP, K, BLOCK>, ge::RowRing<T, K, 2>::bytes(threads)};
  if constexpr (BLOCK || K == 1)
    return {ge::layer_norm_backward_kernel<T, DROP, K, BLOCK>, ge::RowRing<T, K, 3>::bytes(threads)};
  else
    return {nullptr, 0};
}

template <class T, bool DROP>
Kernel kernel_of(int pass, const Shape& s) {
  if (s.wide_row)
    return {pass == FORWARD ? ge::layer_norm_long_kernel<T, DROP> : ge::layer_norm_backward_long_kernel<T, DROP>, 0};
  if (s.block) {
    if (s.k == 1 && pass == BACKWARD)
      return {ge::layer_norm_backward_kernel<T, DROP, 1, true>, ge::RowRing<T, 1, 3>::bytes(s.threads)};
    return s.k == 2 ? kernel_of<T, DROP, 2, true>(pass, s.threads) : kernel_of<T, DROP, 4, true>(pass, s.threads);
  }
  return s.k == 1   ? kernel_of<T, DROP, 1, false>(pass, s.threads)
         : s.k == 2 ? kernel_of<T, DROP, 2, false>(pass, s.threads)
                    : kernel_of<T, DROP, 4, false>(pass, s.threads);
}

Kernel kernel_of(int pass, const Shape& s, bool f32, bool drop) {
  if (f32) return drop ? kernel_of<float, true>(pass, s) : kernel_of<float, false>(pass, s);
  return drop ? kernel_of<uint16_t, true>(pass, s) : kernel_of<uint16_t, false>(pass, s);
}

// Blocks of a kernel resident on an SM of the current device, asked for once
// for each kernel and block size (the shared memory goes with the size).
gemm_epi_status resident_blocks(int dev, int pass, const Shape& s, bool f32, bool drop, const Kernel& k, int* blocks) {
  static std::atomic<int> known[128][2][2][2][8][ge::LN_MAX_WARPS + 1];
  const int form = s.wide_row ? 7 : (s.block ? 4 : 0) + (s.k == 4 ? 2 : s.k - 1);
  std::atomic<int>& at = known[dev][pass][f32][drop][form][s.threads / 32];
  int n = at.load(std::memory_order_acquire);
  if (n == 0) {
    const void* fn = reinterpret_cast<const void*>(k.fn);
    // the most that any block size needs, so that no other thread's call lowers it
    const int most = k.ring_bytes / s.threads * (s.block ? 32 * ge::LN_MAX_WARPS : s.threads);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, s.threads, static_cast<size_t>(k.ring_bytes));
    if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor");
    if (n < 1) return fail(GEMM_EPI_ERR_CUDA, "a layer norm kernel does not fit an SM");
    at.store(n, std::memory_order_release);
  }
  *blocks = n;
  return GEMM_EPI_OK;
}

// Rows of partial sums of dw and db: the most blocks a backward pass has.
int most_partials(int64_t cols) { return cols <= 2048 ? 912 : 304; }

// ---------------------------------------------------------------- checks

constexpr int64_t LIM = 0x7FFFFFFF;

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
    if (cols < 1 || cols > LIM - 7) return fail(GEMM_EPI_ERR_INVALID_VALUE, "N must be in [1, 2^31 - 8]");
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
  if (!d.state) return fail(GEMM_EPI_ERR_INVALID_VALUE, "the dropout state is NULL");
  if (!aligned(d.state, 8)) return fail(GEMM_EPI_ERR_MISALIGNED, "the dropout state must be 8-byte aligned");
  *out = ge::dropout_of(d);
  return GEMM_EPI_OK;
}

// ---------------------------------------------------------------- launches

gemm_epi_status launch_norm(int pass, const ge::NormParams& p, bool f32, int64_t most_blocks, cudaStream_t st, int* grid) {
  int dev = 0, sms = 0, resident = 0;
  gemm_epi_status s = ge_host::device_sms(&dev, &sms);
  if (s) return s;
  const Shape shape = shape_of(pass, p.groups);
  const bool drop = p.drop.state != nullptr;
  const Kernel k = kernel_of(pass, shape, f32, drop);
  if ((s = resident_blocks(dev, pass, shape, f32, drop, k, &resident))) return s;
  const int64_t rows = shape.block ? 1 : static_cast<int64_t>(ge::LN_WARP_TEAMS) << (5 - shape.log_lanes);  // of a block
  int64_t blocks = std::min<int64_t>((p.M + rows - 1) / rows, static_cast<int64_t>(sms) * resident);
  blocks = std::min(blocks, most_blocks);
  ge::NormParams q = p;
  q.log_lanes = shape.log_lanes;
  k.fn<<<static_cast<unsigned>(blocks), static_cast<unsigned>(shape.threads), static_cast<size_t>(k.ring_bytes), st>>>(q);
  const cudaError_t e = cudaGetLastError();
  *grid = static_cast<int>(blocks);
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
  p.N = static_cast<int32_t>(c.N);
  p.groups = static_cast<int32_t>((c.N + 7) / 8);
  p.total = c.M * p.groups;
  p.x = a->x, p.ld_x = a->ld_x;
  p.residual = a->residual, p.ld_residual = a->ld_residual;
  p.y = a->y, p.ld_y = a->ld_y;
  p.wide_in = c.wide_in, p.wide_out = c.wide_out;
  const int64_t blocks = std::min<int64_t>((p.total + ge::DO_THREADS - 1) / ge::DO_THREADS,
                                           static_cast<int64_t>(sms) * ge::DO_BLOCKS);
  p.step_rows = blocks * ge::DO_THREADS / p.groups;
  p.step_groups = static_cast<int32_t>(blocks * ge::DO_THREADS % p.groups);
  const auto fn = c.size == 4 ? ge::dropout_kernel<float> : ge::dropout_kernel<uint16_t>;
  fn<<<static_cast<unsigned>(blocks), ge::DO_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(p);
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
  p.wide_in = c.wide_in, p.wide_out = c.wide_out;
  p.wide_w = aligned(a->w, 16) && aligned(a->b, 16);
  int grid = 0;
  return launch_norm(FORWARD, p, c.size == 4, LIM, static_cast<cudaStream_t>(stream), &grid);
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
  p.wide_in = c.wide_in, p.wide_out = c.wide_out;
  p.wide_w = aligned(a->w, 16);
  int grid = 0;
  if ((s = launch_norm(BACKWARD, p, c.size == 4, most_partials(c.N), st, &grid))) return s;
  if (!wants_dw) return GEMM_EPI_OK;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>((c.N + 31) / 32), 2);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  std::memset(&attr, 0, sizeof attr);
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, ge::layer_norm_weight_grad_kernel, static_cast<const float*>(p.partials), grid, p.N, a->dw,
                         a->db);
  return e == cudaSuccess ? GEMM_EPI_OK : cuda_fail(e, "launch of the weight gradient kernel");
}

size_t gemm_epi_layer_norm_backward_workspace_size(int64_t N) {
  if (N < 1 || N > LIM - 7) return 0;
  return static_cast<size_t>(most_partials(N)) * 2 * static_cast<size_t>(N) * sizeof(float);
}

}  // extern "C"
