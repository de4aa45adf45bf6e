// heads.cu -- host side of the entry points that act on the heads of q and k
// (rotary positions, the head norm with the rotation, its backward), and
// their kernels.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>
#include <cstring>

#include "heads.cuh"
#include "host.h"

namespace {

using ge_host::cuda_fail;
using ge_host::fail;

// ---------------------------------------------------------------- frequencies

constexpr double TWO_PI = 6.283185307179586476925286766559;

// ---------------------------------------------------------------- kernels

// A kernel, its resident blocks per SM and its dynamic shared memory.
struct HeadKernel {
  void (*fn)(ge::HeadParams);
  int blocks, smem;
};

template <class T, bool HALF, bool PART>
HeadKernel kernel_of(int mode, bool wide) {
  using Forward = ge::HeadRing<T, HALF, 1>;
  using Backward = ge::HeadRing<T, HALF, 2>;
  switch (mode) {
    case ge::HEAD_ROTARY:
      return wide ? HeadKernel{ge::heads_kernel<T, HALF, false, PART>, ge::HD_ROTARY_BLOCKS, Forward::BYTES}
                  : HeadKernel{ge::heads_any_kernel<T, HALF, false, PART>, 2, 0};
    case ge::HEAD_NORM:
      return wide ? HeadKernel{ge::heads_kernel<T, HALF, true, PART>, ge::HD_NORM_BLOCKS, Forward::BYTES}
                  : HeadKernel{ge::heads_any_kernel<T, HALF, true, PART>, 2, 0};
    default:
      return wide ? HeadKernel{ge::heads_backward_kernel<T, HALF, PART>, ge::HD_BWD_BLOCKS, Backward::BYTES}
                  : HeadKernel{ge::heads_backward_any_kernel<T, HALF, PART>, ge::HD_BWD_BLOCKS, 0};
  }
}

template <class T>
HeadKernel kernel_of(int mode, bool wide, bool half, bool part) {
  if (half) return part ? kernel_of<T, true, true>(mode, wide) : kernel_of<T, true, false>(mode, wide);
  return part ? kernel_of<T, false, true>(mode, wide) : kernel_of<T, false, false>(mode, wide);
}

// part: some of the values worked on do not rotate.
HeadKernel kernel_of(int mode, bool wide, bool half, bool part, bool f32) {
  return f32 ? kernel_of<float>(mode, wide, half, part) : kernel_of<uint16_t>(mode, wide, half, part);
}

// The current device's SM count.  The first call on a device gives every
// kernel its shared-memory limit.
gemm_epi_status device_setup(int* sms) {
  static std::atomic<bool> ready[128];
  int dev = 0;
  const gemm_epi_status s = ge_host::device_sms(&dev, sms);
  if (s != GEMM_EPI_OK || ready[dev].load(std::memory_order_acquire)) return s;
  for (int i = 0; i < 3 * 2 * 2 * 2; ++i) {
    const HeadKernel k = kernel_of(i / 8, true, (i & 1) != 0, (i & 2) != 0, (i & 4) != 0);
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k.fn),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  }
  ready[dev].store(true, std::memory_order_release);
  return GEMM_EPI_OK;
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

struct Checked {
  bool wide = true;  // 16-byte accesses serve every tensor
  size_t size = 2;
};

gemm_epi_status check_tensor(const gemm_epi_qk_args& a, const gemm_epi_heads& h, int32_t heads, const char* name,
                             Checked& c) {
  if (!h.data) return fail(GEMM_EPI_ERR_INVALID_VALUE, "%s is NULL", name);
  if (!aligned(h.data, c.size))
    return fail(GEMM_EPI_ERR_MISALIGNED, "%s is not aligned to its element size", name);
  const int64_t lim = int64_t(1) << 40;
  const int64_t extent[3] = {a.batch, a.tokens, heads};
  const int64_t stride[3] = {h.stride_batch, h.stride_token, h.stride_head};
  for (int i = 0; i < 3; ++i) {
    if (stride[i] <= -lim || stride[i] >= lim)
      return fail(GEMM_EPI_ERR_INVALID_VALUE, "a stride of %s is out of range", name);
    if (extent[i] > 1 && stride[i] * static_cast<int64_t>(c.size) % 16 != 0) c.wide = false;
  }
  if (!aligned(h.data, 16)) c.wide = false;
  return GEMM_EPI_OK;
}

// Different elements of an output must not share memory: taken by stride, each
// dimension of more than one step advances by at least what the smaller ones
// span (strides and extents are below 2^40 and 2^31: saturating, a span past
// 2^62 is followed by no larger stride).
gemm_epi_status check_output(const gemm_epi_qk_args& a, const gemm_epi_heads& h, int32_t heads, const char* name) {
  struct Dim {
    int64_t stride, extent;
  } dims[3] = {{std::abs(h.stride_batch), a.batch}, {std::abs(h.stride_token), a.tokens}, {std::abs(h.stride_head), heads}};
  std::sort(dims, dims + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
  const int64_t MOST = int64_t(1) << 62;
  int64_t span = a.head_dim;
  for (const Dim& d : dims) {
    if (d.extent <= 1) continue;
    if (d.stride < span)
      return fail(GEMM_EPI_ERR_INVALID_VALUE, "%s: a stride of %lld where the dimensions inside it span %lld makes heads "
                  "overlap", name, static_cast<long long>(d.stride), static_cast<long long>(span));
    span = d.stride > (MOST - span) / (d.extent - 1) ? MOST : span + d.stride * (d.extent - 1);
  }
  return GEMM_EPI_OK;
}

// The same elements: strides of dimensions of one step do not matter.
bool same_place(const gemm_epi_qk_args& args, int32_t heads, const gemm_epi_heads& a, const gemm_epi_heads& b) {
  return a.data == b.data && (args.batch <= 1 || a.stride_batch == b.stride_batch) &&
         (args.tokens <= 1 || a.stride_token == b.stride_token) && (heads <= 1 || a.stride_head == b.stride_head);
}

// An output is written over an input element by element or not at all.
gemm_epi_status check_in_place(const gemm_epi_qk_args& args, int32_t heads, const gemm_epi_heads& out,
                               const gemm_epi_heads& in, const char* o, const char* i) {
  if (out.data && out.data == in.data && !same_place(args, heads, out, in))
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "%s starts where %s does but has other strides", o, i);
  return GEMM_EPI_OK;
}

gemm_epi_status run_heads(const gemm_epi_qk_args* a, int mode, cudaStream_t st) {
  ge_host::clear_error();
  if (!a) return fail(GEMM_EPI_ERR_INVALID_VALUE, "args must not be NULL");
  const int64_t LIM = 0x7FFFFFFF;
  if (a->batch < 0 || a->tokens < 0 || a->batch > LIM || a->tokens > LIM || a->batch * a->tokens > LIM)
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "batch, tokens and their product must be in [0, 2^31)");
  if (a->q_heads < 0 || a->k_heads < 0 || a->q_heads > 65535 || a->k_heads > 65535)
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "q_heads and k_heads must be in [0, 65535]");
  if (a->head_dim < 2 || a->head_dim > ge::HD_MAX_DIM || a->head_dim % 2)
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "head_dim must be even, in [2, %d] (got %d)", ge::HD_MAX_DIM, a->head_dim);
  if (a->rotary_dim < 2 || a->rotary_dim > a->head_dim || a->rotary_dim % 2)
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "rotary_dim must be even, in [2, head_dim] (got %d)", a->rotary_dim);
  if (a->layout != GEMM_EPI_ROTARY_HALF && a->layout != GEMM_EPI_ROTARY_INTERLEAVED)
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "unknown rotary layout %d", a->layout);
  if (a->layout == GEMM_EPI_ROTARY_HALF && a->rotary_dim % 4)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "the half layout needs rotary_dim %% 4 == 0 (got %d)", a->rotary_dim);
  if (a->type != GEMM_EPI_TYPE_BF16 && a->type != GEMM_EPI_TYPE_F32)
    return fail(GEMM_EPI_ERR_UNSUPPORTED, "q and k must be BF16 or F32 (type %d)", a->type);
  if (!std::isfinite(a->amplitude)) return fail(GEMM_EPI_ERR_INVALID_VALUE, "amplitude must be finite");
  if (mode != ge::HEAD_ROTARY && (!(a->eps >= 0.0f) || !std::isfinite(a->eps)))
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "eps must be finite and >= 0");
  const bool rows = a->batch > 0 && a->tokens > 0;
  const bool bwd = mode == ge::HEAD_NORM_BWD;
  const bool wants_dw = bwd && (a->dw_q || a->dw_k);

  Checked c;
  c.size = a->type == GEMM_EPI_TYPE_F32 ? 4 : 2;
  gemm_epi_status s;
  const gemm_epi_heads* in[2] = {&a->q, &a->k};
  const gemm_epi_heads* dy[2] = {&a->dy_q, &a->dy_k};
  const gemm_epi_heads* out[2] = {&a->q_out, &a->k_out};
  const int32_t heads[2] = {a->q_heads, a->k_heads};
  static const char* const names[2][3] = {{"q", "dy_q", "q_out"}, {"k", "dy_k", "k_out"}};
  const float* w[2] = {a->q_weight, a->k_weight};
  for (int i = 0; i < 2; ++i) {
    if (w[i] && !aligned(w[i], 4)) return fail(GEMM_EPI_ERR_MISALIGNED, "%s_weight must be 4-byte aligned", names[i][0]);
    if (!rows || heads[i] == 0) continue;
    if ((s = check_tensor(*a, *in[i], heads[i], names[i][0], c))) return s;
    if (bwd && (s = check_tensor(*a, *dy[i], heads[i], names[i][1], c))) return s;
    // the backward pass may leave a gradient of q or k out
    if ((!bwd || out[i]->data) &&
        ((s = check_tensor(*a, *out[i], heads[i], names[i][2], c)) || (s = check_output(*a, *out[i], heads[i], names[i][2]))))
      return s;
    if ((s = check_in_place(*a, heads[i], *out[i], *in[i], names[i][2], names[i][0]))) return s;
    if (bwd && (s = check_in_place(*a, heads[i], *out[i], *dy[i], names[i][2], names[i][1]))) return s;
    for (int j = 0; j < 2; ++j)  // one tensor's rows must not be another's results
      if (j != i && heads[j] > 0 && out[i]->data &&
          (out[i]->data == in[j]->data || (bwd && out[i]->data == dy[j]->data) || out[i]->data == out[j]->data))
        return fail(GEMM_EPI_ERR_INVALID_VALUE, "%s shares its memory with a tensor of %s", names[i][2], names[j][0]);
  }
  for (const float* d : {a->dw_q, a->dw_k})
    if (bwd && d && !aligned(d, 4)) return fail(GEMM_EPI_ERR_MISALIGNED, "dw_q and dw_k must be 4-byte aligned");
  if (wants_dw && a->dw_q == a->dw_k) return fail(GEMM_EPI_ERR_INVALID_VALUE, "dw_q and dw_k are the same buffer");
  // The heads that a pass over the rows is for: backward, those a wanted result comes from.
  const int64_t q_work = !bwd || a->q_out.data || a->dw_q ? heads[0] : 0;
  const int64_t k_work = !bwd || a->k_out.data || a->dw_k ? heads[1] : 0;
  const bool work = rows && q_work + k_work > 0;
  if (work) {
    if (!a->steps) return fail(GEMM_EPI_ERR_INVALID_VALUE, "steps is NULL");
    if (!aligned(a->steps, 8)) return fail(GEMM_EPI_ERR_MISALIGNED, "steps must be 8-byte aligned");
    if (a->positions && !aligned(a->positions, a->positions_64 ? 8 : 4))
      return fail(GEMM_EPI_ERR_MISALIGNED, "positions is not aligned to its element size");
    if (a->positions && a->position_stride != 0 && a->position_stride < a->tokens)
      return fail(GEMM_EPI_ERR_INVALID_VALUE, "position_stride must be 0 (shared by the batch) or at least tokens");
  }
  const size_t ws = gemm_epi_qk_norm_rotary_workspace_size(a->head_dim);
  if (wants_dw && work && (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < ws))
    return fail(GEMM_EPI_ERR_WORKSPACE, "workspace must be 16-byte aligned and hold %zu bytes (got %zu)", ws,
                a->workspace ? a->workspace_bytes : static_cast<size_t>(0));
  int sms = 0;
  if ((s = device_setup(&sms))) return s;
  cudaError_t e;
  if (!work) {
    // nothing to sum: the weights' gradients are zero
    for (float* d : {a->dw_q, a->dw_k})
      if (bwd && d && (e = cudaMemsetAsync(d, 0, sizeof(float) * a->head_dim, st)) != cudaSuccess)
        return cuda_fail(e, "cudaMemsetAsync of dw");
    return GEMM_EPI_OK;
  }

  const bool half = a->layout == GEMM_EPI_ROTARY_HALF;
  const int pairs = a->rotary_dim / 2;
  // 16-byte accesses need whole chunks of them: in the head, and in each half
  // of the rotated part.
  const int chunk = static_cast<int>(16 / c.size);
  const bool wide = c.wide && a->head_dim % chunk == 0 && (!half || pairs % chunk == 0);
  const int V = wide ? chunk : 2, slots = 8 / V;

  ge::HeadParams p;
  std::memset(&p, 0, sizeof p);
  p.tokens = static_cast<int32_t>(a->tokens);
  p.rows = static_cast<int32_t>(a->batch * a->tokens);
  p.dim = a->head_dim;
  p.rot_pairs = pairs;
  // In place and without a norm, what does not rotate is already there.
  bool in_place = mode == ge::HEAD_ROTARY;
  for (int i = 0; i < 2; ++i) in_place = in_place && (heads[i] == 0 || same_place(*a, heads[i], *in[i], *out[i]));
  p.reach = in_place ? (a->rotary_dim + V - 1) / V * V : a->head_dim;
  const int chunks = p.reach / V;  // reach is whole chunks: V divides head_dim
  p.first_plain = half ? pairs / V : 0;
  p.num_pc = p.first_plain + (chunks - 2 * p.first_plain + 1) / 2;
  p.log_g = 0;
  while ((slots << p.log_g) < p.num_pc) ++p.log_g;
  for (int i = 0; i < 2; ++i) {
    ge::HeadPart& h = p.part[i];
    h.heads = heads[i];
    h.x = in[i]->data, h.x_b = in[i]->stride_batch, h.x_t = in[i]->stride_token, h.x_h = in[i]->stride_head;
    h.dy = dy[i]->data, h.dy_b = dy[i]->stride_batch, h.dy_t = dy[i]->stride_token, h.dy_h = dy[i]->stride_head;
    h.y = out[i]->data, h.y_b = out[i]->stride_batch, h.y_t = out[i]->stride_token, h.y_h = out[i]->stride_head;
    h.w = w[i];
  }
  p.steps = a->steps;
  p.positions = a->positions;
  p.positions_64 = a->positions_64 ? 1 : 0;
  p.pos_b = a->position_stride;
  p.amplitude = a->amplitude;
  p.sin_sign = (bwd || (mode == ge::HEAD_ROTARY && a->inverse)) ? -1.0f : 1.0f;
  p.eps = a->eps;
  p.inv_dim = 1.0f / static_cast<float>(a->head_dim);
  p.partials = wants_dw ? static_cast<float*>(a->workspace) : nullptr;

  const HeadKernel kernel = kernel_of(mode, wide, half, a->rotary_dim < p.reach, a->type == GEMM_EPI_TYPE_F32);
  const int64_t resident = static_cast<int64_t>(sms) * kernel.blocks;
  // One wave of blocks, and no more warps than iterations.
  const int64_t groups = 32 >> p.log_g;                   // lane groups of a warp, a token to each
  const int64_t sets = (p.rows + groups - 1) / groups;    // of tokens (64-bit: rows may be 2^31 - 1)
  auto share_out = [&](ge::HeadShare& h, int64_t per_row, int64_t most) {
    const int64_t total = sets * per_row;
    const int64_t blocks = std::min(most, (total + ge::HD_WARPS - 1) / ge::HD_WARPS);
    const int64_t warps = std::max<int64_t>(1, blocks * ge::HD_WARPS);
    const int64_t left = sets % warps * per_row;  // iterations past the whole rounds
    h.warps = static_cast<int32_t>(warps);
    h.per_row = static_cast<int32_t>(std::max<int64_t>(1, per_row));
    h.rounds = blocks ? static_cast<int32_t>(sets / warps) : 0;
    h.base = static_cast<int32_t>(left / warps);
    h.rest = static_cast<int32_t>(left % warps);
    return blocks;
  };
  int64_t blocks;
  if (bwd) {
    // shared between q and k by their work; a part none of whose results is
    // wanted gets no block
    const int64_t most = std::min<int64_t>(ge::HD_MAX_PARTIALS, resident);
    int64_t q_most = q_work ? most : 0;
    if (q_work && k_work)
      q_most = std::min(most - 1, std::max<int64_t>(1, (most * q_work + (q_work + k_work) / 2) / (q_work + k_work)));
    const int64_t q = share_out(p.share[0], q_work, q_most), k = share_out(p.share[1], k_work, most - q_most);
    p.q_blocks = static_cast<int32_t>(q);
    blocks = q + k;
  } else {
    blocks = share_out(p.share[0], q_work + k_work, resident);
  }
  kernel.fn<<<static_cast<unsigned>(blocks), ge::HD_THREADS, static_cast<size_t>(kernel.smem), st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch of the head kernel");
  if (wants_dw) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>((a->head_dim + 31) / 32), 2);
    cfg.blockDim = dim3(32, 32);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    std::memset(&attr, 0, sizeof attr);
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, ge::head_weight_grad_kernel, static_cast<const float*>(p.partials),
                           static_cast<int>(p.q_blocks), static_cast<int>(blocks), static_cast<int>(a->head_dim),
                           a->dw_q, a->dw_k);
    if (e != cudaSuccess) return cuda_fail(e, "launch of the weight gradient kernel");
  }
  return GEMM_EPI_OK;
}

}  // namespace

extern "C" {

gemm_epi_status gemm_epi_rotary_steps(const gemm_epi_rotary_freq* f, uint64_t* steps) {
  ge_host::clear_error();
  if (!f || !steps) return fail(GEMM_EPI_ERR_INVALID_VALUE, "freq and steps must not be NULL");
  if (f->rotary_dim < 2 || f->rotary_dim % 2 || f->rotary_dim > ge::HD_MAX_DIM)
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "rotary_dim must be even, in [2, %d] (got %d)", ge::HD_MAX_DIM,
                f->rotary_dim);
  if (!f->freq && (!(f->base > 0.0) || !std::isfinite(f->base)))
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "base must be finite and > 0");
  if (f->scaling < GEMM_EPI_ROTARY_UNSCALED || f->scaling > GEMM_EPI_ROTARY_BY_PARTS)
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "unknown scaling %d", f->scaling);
  if (f->scaling != GEMM_EPI_ROTARY_UNSCALED && (!(f->factor > 0.0) || !std::isfinite(f->factor)))
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "factor must be finite and > 0");
  if (f->scaling == GEMM_EPI_ROTARY_NTK && (f->rotary_dim < 4 || f->freq))
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "NTK scaling changes the base: it needs rotary_dim >= 4 and no freq");
  if (f->scaling == GEMM_EPI_ROTARY_BY_PARTS &&
      (!(f->original_length > 0.0) || !std::isfinite(f->original_length) || !std::isfinite(f->low) ||
       !std::isfinite(f->high) || !(f->low < f->high)))
    return fail(GEMM_EPI_ERR_INVALID_VALUE, "BY_PARTS scaling needs original_length > 0 and low < high");
  double base = f->base;
  if (f->scaling == GEMM_EPI_ROTARY_NTK)
    base *= std::pow(f->factor, f->rotary_dim / (f->rotary_dim - 2.0));
  if (!f->freq && !std::isfinite(base)) return fail(GEMM_EPI_ERR_INVALID_VALUE, "the scaled base is not finite");
  for (int i = 0; i < f->rotary_dim / 2; ++i) {
    double w = f->freq ? f->freq[i] : std::pow(base, -2.0 * i / f->rotary_dim);
    if (f->scaling == GEMM_EPI_ROTARY_LINEAR) w /= f->factor;
    if (f->scaling == GEMM_EPI_ROTARY_BY_PARTS) {
      const double turns = f->original_length * w / TWO_PI;
      const double keep = std::min(1.0, std::max(0.0, (turns - f->low) / (f->high - f->low)));
      w = w * keep + w / f->factor * (1.0 - keep);
    }
    if (!std::isfinite(w)) return fail(GEMM_EPI_ERR_INVALID_VALUE, "frequency %d is not finite", i);
    double frac = w / TWO_PI;
    frac -= std::floor(frac);  // [0, 1]
    const double scaled = std::nearbyint(frac * 18446744073709551616.0);
    steps[i] = scaled >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(scaled);
  }
  return GEMM_EPI_OK;
}

gemm_epi_status gemm_epi_rotary(const gemm_epi_qk_args* args, void* stream) {
  return run_heads(args, ge::HEAD_ROTARY, static_cast<cudaStream_t>(stream));
}

gemm_epi_status gemm_epi_qk_norm_rotary(const gemm_epi_qk_args* args, void* stream) {
  return run_heads(args, ge::HEAD_NORM, static_cast<cudaStream_t>(stream));
}

gemm_epi_status gemm_epi_qk_norm_rotary_backward(const gemm_epi_qk_args* args, void* stream) {
  return run_heads(args, ge::HEAD_NORM_BWD, static_cast<cudaStream_t>(stream));
}

size_t gemm_epi_qk_norm_rotary_workspace_size(int32_t head_dim) {
  if (head_dim < 2 || head_dim > ge::HD_MAX_DIM) return 0;
  return static_cast<size_t>(ge::HD_MAX_PARTIALS) * static_cast<size_t>(head_dim) * sizeof(float);
}

}  // extern "C"
