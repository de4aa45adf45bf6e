"""Torch-facing wrapper over the C ABI: builds the descriptor from an op list,
passes tensor data pointers and the current CUDA stream.  No arithmetic of the
method happens here; every step runs in the CUDA library.

Programs are written as op names (one optional numeric argument after a
colon):

  alpha, bias, row_scale, residual, gelu_tanh, relu, silu, pair_swiglu[:g], pair_mul[:g],
  gelu_tanh_grad, amax, store_bf16, store_e4m3, row_rms[:eps],
  row_rms_unrounded[:eps], col_sum, dswiglu[:g], col_scale, row_dot,
  head_rms[:eps], rotary, dropout
"""
from __future__ import annotations

import ctypes
import struct
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import native as N

PROGRAM_OPS = {
    "alpha": N.GEMM_EPI_OP_SCALE_ALPHA,
    "bias": N.GEMM_EPI_OP_ADD_BIAS_COL,
    "row_scale": N.GEMM_EPI_OP_MUL_ROW_SCALE,
    "residual": N.GEMM_EPI_OP_ADD_RESIDUAL,
    "gelu_tanh": N.GEMM_EPI_OP_ACT_GELU_TANH,
    "relu": N.GEMM_EPI_OP_ACT_RELU,
    "silu": N.GEMM_EPI_OP_ACT_SILU,
    "pair_swiglu": N.GEMM_EPI_OP_PAIR_SWIGLU,
    "pair_mul": N.GEMM_EPI_OP_PAIR_MUL,
    "dswiglu": N.GEMM_EPI_OP_DSWIGLU,
    "col_scale": N.GEMM_EPI_OP_MUL_COL_SCALE,
    "row_dot": N.GEMM_EPI_OP_ROW_DOT,
    "gelu_tanh_grad": N.GEMM_EPI_OP_MUL_GELU_TANH_GRAD,
    "amax": N.GEMM_EPI_OP_AMAX,
    "store_bf16": N.GEMM_EPI_OP_STORE_BF16,
    "store_e4m3": N.GEMM_EPI_OP_STORE_E4M3,
    "row_rms": N.GEMM_EPI_OP_ROW_RMS_RSQRT,
    "row_rms_unrounded": N.GEMM_EPI_OP_ROW_RMS_RSQRT,
    "col_sum": N.GEMM_EPI_OP_COL_SUM,
    "head_rms": N.GEMM_EPI_OP_HEAD_RMS,
    "rotary": N.GEMM_EPI_OP_ROTARY,
    "dropout": N.GEMM_EPI_OP_DROPOUT,
}


def encode_program(program: Sequence[str], drop_threshold: int = 0):
    ops = (N.gemm_epi_op * max(1, len(program)))()
    for i, spec in enumerate(program):
        name, _, arg = spec.partition(":")
        if name not in PROGRAM_OPS:
            raise ValueError("unknown epilogue op %r" % name)
        code = PROGRAM_OPS[name]
        i0, f0 = 0, 0.0
        if name in ("pair_swiglu", "pair_mul", "dswiglu"):
            i0 = int(arg) if arg else 1
        elif name.startswith("row_rms") or name == "head_rms":
            f0 = float(arg) if arg else 1e-6
            i0 = 1 if name == "row_rms_unrounded" else 0
        elif name == "dropout":
            if arg:
                raise ValueError("the dropout op takes its probability from dropout=, not %r" % spec)
            i0 = drop_threshold
        ops[i] = N.gemm_epi_op(code, i0, f0)
    return ops


# The current stream of a device as an integer, without the stream object that
# torch.cuda.current_stream() builds (2.9 us of a small call's 7).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
# The current device, where a CUDA tensor is at hand: CUDA is initialised.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call_on(t: Optional[torch.Tensor], stream: Optional[torch.cuda.Stream], call):
    """call(stream) with the given stream, or the current one of t's device, as
    an integer, and that device current: the library launches on the current
    device, which cannot read another one's memory."""
    index = -1 if t is None else t.get_device()
    if index < 0:  # host memory: the library says what is wrong
        return call(_raw_stream(torch.cuda.current_device()) if stream is None else stream.cuda_stream)
    if index == _current_device():
        return call(_raw_stream(index) if stream is None else stream.cuda_stream)
    with torch.cuda.device(index):
        return call(_raw_stream(index) if stream is None else stream.cuda_stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


_KIND_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _bytes_after(t: torch.Tensor) -> int:
    """Bytes of the tensor's storage from its first element to the end."""
    return t.untyped_storage().nbytes() - t.storage_offset() * t.element_size()


def _expect(name: str, t: Optional[torch.Tensor], kind: str, rows: int, cols: int = 1, ld: int = 1,
            batch: int = 1, batch_stride: int = 0) -> None:
    """Checks one buffer before its pointer crosses the C ABI, which sees
    neither dtype nor size: ``kind`` is "bf16", "f32" or "byte" (any 8-bit
    type), and the storage must hold ``batch`` matrices of ``rows`` x ``cols``
    elements at row stride ``ld`` and batch stride ``batch_stride``."""
    if t is None:
        return
    ok = {"bf16": t.dtype == torch.bfloat16, "f32": t.dtype == torch.float32,
          "byte": t.element_size() == 1}[kind]
    if not ok:
        raise TypeError("%s: expected a %s tensor, got %s" % (name, kind, t.dtype))
    if batch <= 0 or rows <= 0 or cols <= 0:
        return
    need = ((batch - 1) * batch_stride + (rows - 1) * ld + cols) * t.element_size()
    if need > _bytes_after(t):
        raise ValueError("%s: %d bytes needed from its first element, the storage holds %d"
                         % (name, need, _bytes_after(t)))


def _width_at(program: Sequence[str], N_: int):
    """Accumulator width each op sees: N before a pair op, N/2 after it, 2N
    after dswiglu."""
    w, out = N_, []
    for spec in program:
        name = spec.partition(":")[0]
        out.append((name, w))
        if name.startswith("pair_"):
            w = N_ // 2
        elif name == "dswiglu":
            w = 2 * N_
    return out


# Operand element types (desc.a_type / b_type); 8-bit operands are passed as
# uint8 (or torch float8) tensors of codes.
OPERAND_TYPES = {"bf16": N.GEMM_EPI_TYPE_BF16, "e4m3": N.GEMM_EPI_TYPE_E4M3, "e5m2": N.GEMM_EPI_TYPE_E5M2}


# Ops that read the auxiliary M x N_out tensor, by the argument it travels in.
RESIDUAL_OPS = frozenset({"residual", "row_dot"})
PREACT_OPS = frozenset({"gelu_tanh_grad", "dswiglu"})


def out_cols(program: Sequence[str], N_: int) -> int:
    """Output columns of a program over N accumulator columns."""
    names = [op.partition(":")[0] for op in program]
    if "dswiglu" in names:
        return 2 * N_
    return N_ // 2 if any(n.startswith("pair_") for n in names) else N_


class Plan:
    """One validated GEMM + epilogue plan (gemm_epi_create).  Strides default
    to tight row-major packing.

    Programs with head_rms or rotary (a q|k|v projection): columns
    [0, head_cols) are the heads of q and k, `rotary` holds the frequencies,
    head size and layout (head_dim alone is enough without the rotary op), and
    run() takes the rows' positions.

    Programs with dropout: `dropout` holds the probability, seed and step, run()
    takes the call's site; rows are counted through the batch."""

    def __init__(self, M: int, N_: int, K: int, program: Sequence[str], b_layout: str = "kn",
                 lda: Optional[int] = None, ldb: Optional[int] = None, ldc: Optional[int] = None,
                 ldc8: Optional[int] = None, ld_aux: Optional[int] = None, dual: bool = False,
                 batch: int = 1, batch_stride_a: Optional[int] = None,
                 batch_stride_b: Optional[int] = None, batch_stride_c: Optional[int] = None,
                 batch_stride_c8: Optional[int] = None, batch_stride_aux: Optional[int] = None,
                 a_type: str = "bf16", b_type: str = "bf16", rotary: Optional["Rotary"] = None,
                 head_dim: Optional[int] = None, head_cols: int = 0, dropout: Optional["Dropout"] = None):
        self.lib = N.load()
        self.program = list(program)
        self.M, self.N, self.K = M, N_, K
        self.b_layout = b_layout
        n_out = out_cols(program, N_)
        if dropout is None and "dropout" in self.program:
            raise ValueError("a program with the dropout op needs dropout=")
        self.dropout = dropout if "dropout" in self.program else None
        self._ops = encode_program(program, 0 if dropout is None else dropout.threshold)
        d = N.gemm_epi_desc()
        d.M, d.N, d.K = M, N_, K
        d.lda = K if lda is None else lda
        b_cols = N_ // 2 if dual else N_
        d.ldb = (b_cols if b_layout == "kn" else K) if ldb is None else ldb
        d.ldc = n_out if ldc is None else ldc
        d.ldc8 = n_out if ldc8 is None else ldc8
        d.ld_aux = n_out if ld_aux is None else ld_aux
        d.b_layout = (N.GEMM_EPI_B_KN if b_layout == "kn" else N.GEMM_EPI_B_NK) | (N.GEMM_EPI_B_DUAL if dual else 0)
        self.dual = dual
        d.n_ops = len(program)
        d.ops = ctypes.cast(self._ops, ctypes.POINTER(N.gemm_epi_op))
        # Batched: tight packing by default; a stride of 0 shares A or B.
        d.batch = batch
        b_rows = K if b_layout == "kn" else b_cols
        d.batch_stride_a = M * d.lda if batch_stride_a is None else batch_stride_a
        d.batch_stride_b = b_rows * d.ldb if batch_stride_b is None else batch_stride_b
        d.batch_stride_c = M * d.ldc if batch_stride_c is None else batch_stride_c
        d.batch_stride_c8 = M * d.ldc8 if batch_stride_c8 is None else batch_stride_c8
        d.batch_stride_aux = M * d.ld_aux if batch_stride_aux is None else batch_stride_aux
        self.batch = max(1, batch)  # 0 is a single problem too
        d.a_type, d.b_type = OPERAND_TYPES[a_type], OPERAND_TYPES[b_type]
        self.a_type, self.b_type = a_type, b_type
        self.rotary = rotary
        if rotary is not None:
            if head_dim is not None and head_dim != rotary.head_dim:
                raise ValueError("head_dim %d is not the rotary's %d" % (head_dim, rotary.head_dim))
            head_dim = rotary.head_dim
            d.rotary_dim, d.rotary_layout = rotary.rotary_dim, rotary.layout_code
        elif "rotary" in self.program:
            raise ValueError("a program with the rotary op needs rotary=")
        d.head_dim, d.head_cols = head_dim or 0, head_cols
        self.desc = d
        h = N.gemm_epi_handle()
        N.check(self.lib.gemm_epi_create(ctypes.byref(h), ctypes.byref(d)), self.lib)
        self.handle = h
        self.n_out = int(self.lib.gemm_epi_out_cols(h))
        self.workspace_bytes = int(self.lib.gemm_epi_workspace_size(h))
        self._extents = self._operand_extents()

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            self.lib.gemm_epi_destroy(h)
            self.handle = None

    def args(self, A, B, *, alpha=1.0, fp8_scale=1.0, bias=None, row_scale=None, residual=None,
             preact=None, C=None, C8=None, amax=None, row_out=None, col_out=None, workspace=None,
             timeout_ms=0, debug_flags=0, B2=None, a_scale_inv=None, b_scale_inv=None,
             col_scale=None, positions=None, site=0) -> N.gemm_epi_args:
        a = N.gemm_epi_args()
        a.alpha, a.fp8_scale = float(alpha), float(fp8_scale)
        for name, t in (("A", A), ("B", B), ("B2", B2), ("bias", bias), ("row_scale", row_scale),
                        ("residual", residual), ("preact", preact), ("C", C), ("C8", C8), ("amax", amax),
                        ("row_out", row_out), ("col_out", col_out), ("a_scale_inv", a_scale_inv),
                        ("b_scale_inv", b_scale_inv), ("col_scale", col_scale)):
            if t is not None:
                kind, elements, extent = self._extents[name]
                # A contiguous tensor of the right type and size needs no look at its storage.
                if (t.dtype is not _KIND_DTYPE.get(kind) or t.numel() < elements or not t.is_contiguous()):
                    _expect(name, t, kind, *extent)
                setattr(a, name, t.data_ptr())
        if workspace is not None:
            a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        if timeout_ms or debug_flags:
            a.timeout_ms, a.debug_flags = int(timeout_ms), int(debug_flags)
        if self.rotary is not None:
            steps = self.rotary._steps
            index = steps.get_device()
            if A is not None and index != A.get_device():
                raise ValueError("the rotary steps are on %s, A on %s" % (steps.device, A.device))
            if workspace is not None and index != workspace.get_device():
                raise ValueError("the rotary steps are on %s, the workspace on %s" % (steps.device, workspace.device))
            a.rotary_steps, a.rotary_amplitude = steps.data_ptr(), self.rotary.amplitude
            if positions is not None:
                if positions.dtype is not torch.int32 and positions.dtype is not torch.int64:
                    raise TypeError("positions: expected an int32 or int64 tensor, got %s" % positions.dtype)
                if positions.numel() != self.batch * self.M or not positions.is_contiguous():
                    raise ValueError("positions: expected %d contiguous values, got %s"
                                     % (self.batch * self.M, tuple(positions.shape)))
                if positions.get_device() != index:
                    raise ValueError("positions are on %s, the rotary steps on %s"
                                     % (positions.device, steps.device))
                a.positions, a.positions_64 = positions.data_ptr(), 1 if positions.dtype is torch.int64 else 0
        elif positions is not None:
            raise ValueError("positions: the plan has no rotary")
        if self.dropout is not None:
            step = self.dropout._step
            index = step.get_device()
            for name, t in (("A", A), ("the workspace", workspace)):
                if t is not None and index != t.get_device():
                    raise ValueError("the dropout step is on %s, %s on %s" % (step.device, name, t.device))
            if not 0 <= site < 2 ** 32:
                raise ValueError("site must be in [0, 2^32), got %r" % (site,))
            a.dropout_step, a.dropout_seed, a.dropout_site = step.data_ptr(), self.dropout.seed, site
        elif site:
            raise ValueError("site: the plan has no dropout")
        return a

    def _operand_extents(self):
        """What _expect() needs of each tensor, and the elements from its first
        to its last: {name: (kind, elements, (rows, cols, ld, batch, batch_stride))}."""
        d, M, K, Bt = self.desc, self.M, self.K, self.batch
        op_kind = lambda t: "bf16" if t == "bf16" else "byte"  # noqa: E731
        b_cols = self.N // 2 if self.dual else self.N
        b_rows, b_inner = (K, b_cols) if self.b_layout == "kn" else (b_cols, K)
        widths = dict((op, w) for op, w in _width_at(self.program, self.N))
        matrix = {"A": (op_kind(self.a_type), M, K, d.lda, Bt, d.batch_stride_a),
                  "B": (op_kind(self.b_type), b_rows, b_inner, d.ldb, Bt, d.batch_stride_b),
                  "B2": (op_kind(self.b_type), b_rows, b_inner, d.ldb, Bt, d.batch_stride_b),
                  "C": ("bf16", M, self.n_out, d.ldc, Bt, d.batch_stride_c),
                  "C8": ("byte", M, self.n_out, d.ldc8, Bt, d.batch_stride_c8),
                  "residual": ("bf16", M, self.n_out, d.ld_aux, Bt, d.batch_stride_aux),
                  "preact": ("bf16", M, self.n_out, d.ld_aux, Bt, d.batch_stride_aux),
                  "row_scale": ("f32", Bt * M, 1, 1, 1, 0), "row_out": ("f32", Bt * M, 1, 1, 1, 0),
                  "col_out": ("f32", Bt * self.n_out, 1, 1, 1, 0),
                  "bias": ("f32", widths.get("bias", 1), 1, 1, 1, 0),
                  "col_scale": ("f32", widths.get("col_scale", 1), 1, 1, 1, 0)}
        for name in ("amax", "a_scale_inv", "b_scale_inv"):
            matrix[name] = ("f32", 1, 1, 1, 1, 0)
        return {name: (v[0], (v[4] - 1) * v[5] + (v[1] - 1) * v[3] + v[2], v[1:]) for name, v in matrix.items()}

    def run(self, *tensors, stream: Optional[torch.cuda.Stream] = None, **kw):
        """gemm_epi_run on the current (or given) stream of the workspace's device; asynchronous."""
        a = self.args(*tensors, **kw)
        status = _call_on(kw.get("workspace"), stream, lambda s: self.lib.gemm_epi_run(self.handle, ctypes.byref(a), s))
        if status:
            N.check(status, self.lib)

    def run_unfused(self, *tensors, scratch: torch.Tensor, stream=None, **kw):
        a = self.args(*tensors, **kw)
        _expect("scratch", scratch, "bf16", self.M, self.N, scratch.stride(0))
        N.check(_call_on(scratch, stream, lambda s: self.lib.gemm_epi_run_unfused(
            self.handle, ctypes.byref(a), ctypes.c_void_p(scratch.data_ptr()), scratch.stride(0), s)), self.lib)

    def query_status(self, workspace: torch.Tensor, stream=None) -> int:
        return int(_call_on(workspace, stream, lambda s: self.lib.gemm_epi_query_status(
            self.handle, ctypes.c_void_p(workspace.data_ptr()), s)))


@dataclass
class Outputs:
    C: Optional[torch.Tensor] = None
    C8: Optional[torch.Tensor] = None
    amax: Optional[torch.Tensor] = None
    row_out: Optional[torch.Tensor] = None
    col_out: Optional[torch.Tensor] = None
    workspace: Optional[torch.Tensor] = None


def allocate_outputs(plan: Plan, device) -> Outputs:
    """Device buffers for every output the program writes (torch allocates)."""
    prog = [op.partition(":")[0] for op in plan.program]
    o = Outputs()
    lead = (plan.batch,) if plan.batch > 1 else ()
    if "store_bf16" in prog:
        o.C = torch.empty(lead + (plan.M, plan.n_out), dtype=torch.bfloat16, device=device)
    if "store_e4m3" in prog:
        o.C8 = torch.empty(lead + (plan.M, plan.n_out), dtype=torch.uint8, device=device)
    if "amax" in prog:
        o.amax = torch.empty(1, dtype=torch.float32, device=device)
    if any(p.startswith("row_rms") or p == "row_dot" for p in prog):
        o.row_out = torch.empty(lead + (plan.M,), dtype=torch.float32, device=device)
    if "col_sum" in prog:
        o.col_out = torch.empty(lead + (plan.n_out,), dtype=torch.float32, device=device)
    o.workspace = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=device)
    return o


def run_program(plan: Plan, A, B, out: Outputs, *, alpha=1.0, fp8_scale=1.0, bias=None,
                row_scale=None, aux=None, unfused_scratch=None, **kw) -> Outputs:
    """Runs the plan with the auxiliary tensor routed to residual or preact."""
    prog = [op.partition(":")[0] for op in plan.program]
    residual = aux if any(op in RESIDUAL_OPS for op in prog) else None
    preact = aux if any(op in PREACT_OPS for op in prog) else None
    tensors = dict(alpha=alpha, fp8_scale=fp8_scale, bias=bias, row_scale=row_scale,
                   residual=residual, preact=preact, C=out.C, C8=out.C8, amax=out.amax,
                   row_out=out.row_out, col_out=out.col_out, workspace=out.workspace, **kw)
    if unfused_scratch is not None:
        plan.run_unfused(A, B, scratch=unfused_scratch, **tensors)
    else:
        plan.run(A, B, **tensors)
    return out


def rmsnorm_backward(dy, x, s, r, *, w=None, add=None, dx=None, dw=None, stream=None):
    """gemm_epi_rmsnorm_backward: dx = S w dy - x S^3 r / N (+ add) into `dx`
    and dw = sum_m dy x S into `dw` (either may be None); bf16 2-D tensors
    with unit column stride, fp32 vectors.  Asynchronous."""
    lib = N.load()
    a = N.gemm_epi_rmsnorm_bwd_args()
    a.M, a.N = dy.shape
    for name, t in (("dy", dy), ("x", x), ("add", add), ("dx", dx)):
        _expect(name, t, "bf16", a.M, a.N, 1 if t is None else t.stride(0))
    for name, t, n in (("s", s, a.M), ("r", r, a.M), ("w", w, a.N), ("dw", dw, a.N)):
        _expect(name, t, "f32", n)
    a.dy, a.ld_dy = _ptr(dy), dy.stride(0)
    a.x, a.ld_x = _ptr(x), x.stride(0)
    a.add, a.ld_add = _ptr(add), (add.stride(0) if add is not None else 0)
    a.w, a.s, a.r = _ptr(w), _ptr(s), _ptr(r)
    a.dx, a.ld_dx = _ptr(dx), (dx.stride(0) if dx is not None else 0)
    a.dw = _ptr(dw)
    N.check(_call_on(dy, stream, lambda st: lib.gemm_epi_rmsnorm_backward(ctypes.byref(a), st)), lib)


ROTARY_LAYOUTS = {"half": N.GEMM_EPI_ROTARY_HALF, "interleaved": N.GEMM_EPI_ROTARY_INTERLEAVED}
ROTARY_SCALINGS = {"linear": N.GEMM_EPI_ROTARY_LINEAR, "ntk": N.GEMM_EPI_ROTARY_NTK,
                   "by_parts": N.GEMM_EPI_ROTARY_BY_PARTS}
HEAD_TYPES = {torch.bfloat16: N.GEMM_EPI_TYPE_BF16, torch.float32: N.GEMM_EPI_TYPE_F32}


class Rotary:
    """The frequencies of rotary positions (gemm_epi_rotary_steps), copied to
    `device` once and kept for every call.

    The first `rotary_dim` values of a head (all of them by default) are
    rotated in pairs: (i, i + rotary_dim / 2) with layout "half", (2i, 2i + 1)
    with "interleaved".  Pair i turns by base^(-2i / rotary_dim) radians per
    position, or by freqs[i].  `scaling` stretches them for long contexts:
    dict(kind="linear" | "ntk", factor=f) or dict(kind="by_parts", factor=f,
    original_length=n, low=1, high=32), each with an optional amplitude the
    rotated part is multiplied by (default 1).
    """

    def __init__(self, head_dim: int, rotary_dim: Optional[int] = None, base: float = 10000.0, layout: str = "half",
                 scaling: Optional[dict] = None, freqs: Optional[Sequence[float]] = None, device="cuda"):
        if layout not in ROTARY_LAYOUTS:
            raise ValueError("unknown rotary layout %r" % (layout,))
        self.head_dim = int(head_dim)
        self.rotary_dim = self.head_dim if rotary_dim is None else int(rotary_dim)
        if self.rotary_dim > self.head_dim:
            raise ValueError("rotary_dim %d is above head_dim %d" % (self.rotary_dim, self.head_dim))
        self.layout, self.layout_code = layout, ROTARY_LAYOUTS[layout]
        f = N.gemm_epi_rotary_freq()
        f.rotary_dim, f.base = self.rotary_dim, float(base)
        opts = dict(scaling or {})
        kind = opts.pop("kind", None)
        if scaling is not None:
            if kind not in ROTARY_SCALINGS:
                raise ValueError("unknown rotary scaling %r" % (kind,))
            f.scaling, f.factor = ROTARY_SCALINGS[kind], float(opts.pop("factor"))
            if kind == "by_parts":
                f.original_length = float(opts.pop("original_length"))
                f.low, f.high = float(opts.pop("low", 1.0)), float(opts.pop("high", 32.0))
        self.amplitude = float(opts.pop("amplitude", 1.0))
        if opts:
            raise ValueError("unknown options of rotary scaling %r: %s" % (kind, ", ".join(sorted(opts))))
        given = None
        if freqs is not None:
            given = (ctypes.c_double * len(freqs))(*[float(x) for x in freqs])
            if len(freqs) != self.rotary_dim // 2:
                raise ValueError("%d frequencies for %d pairs" % (len(freqs), self.rotary_dim // 2))
            f.freq = ctypes.cast(given, ctypes.POINTER(ctypes.c_double))
        steps = (ctypes.c_uint64 * max(1, self.rotary_dim // 2))()
        lib = N.load()
        N.check(lib.gemm_epi_rotary_steps(ctypes.byref(f), steps), lib)
        # uint64 bits in an int64 tensor: torch has no arithmetic on them here
        self.steps = torch.frombuffer(steps, dtype=torch.int64).clone().to(device)
        self.vector_shape = (self.head_dim,)

    @property
    def steps(self) -> torch.Tensor:
        """The device's rotary_dim / 2 steps (gemm_epi_rotary_steps), as int64;
        others of that type and size may be put in their place."""
        return self._steps

    @steps.setter
    def steps(self, t: torch.Tensor) -> None:
        # checked here, once, so that no call has to: the kernels read this many
        if t.dtype is not torch.int64 or t.shape != (self.rotary_dim // 2,) or not t.is_contiguous():
            raise ValueError("steps: expected %d contiguous int64 values, got %s %s"
                             % (self.rotary_dim // 2, t.dtype, tuple(t.shape)))
        self._steps = t


# gemm_epi_qk_args, packed in one step: filling a ctypes structure field by
# field took 2.4 us of a small call.
_QK_ARGS = struct.Struct("@qqiiiiii24qQQqiiffQQQQQN")
assert _QK_ARGS.size == ctypes.sizeof(N.gemm_epi_qk_args)
_NO_HEADS = (0, 0, 0, 0)
_head_entries: dict = {}


def _head_entry(name: str):
    """The entry point taking a gemm_epi_qk_args as packed bytes."""
    fn = _head_entries.get(name)
    if fn is None:
        fn = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, ctypes.c_void_p)((name, N.load()))
        _head_entries[name] = fn
    return fn


def _heads(name: str, t: torch.Tensor, shape, dtype, index: int):
    """(pointer, batch, token and head strides) of a tensor of q's or k's
    shape, type and device, checked."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError("%s: %s %s does not match %s %s" % (name, t.dtype, tuple(t.shape), dtype, tuple(shape)))
    if t.get_device() != index:
        raise ValueError("%s is on %s, not with the other tensors" % (name, t.device))
    st = t.stride()
    if len(st) == 4:
        sb, ss, sh, sd = st
    else:
        sb, (ss, sh, sd) = 0, st
    if sd != 1 and t.numel():
        raise ValueError("%s: the values of a head must be contiguous" % name)
    return t.data_ptr(), sb, ss, sh


def _head_input(name: str, t: torch.Tensor, shape, head_dim: int):
    """batch, tokens, heads and (pointer, batch, token and head strides) of q or k."""
    batch = dim = 1
    if len(shape) == 4:
        batch, tokens, heads, dim = shape
        sb, ss, sh, sd = t.stride()
    elif len(shape) == 3:
        tokens, heads, dim = shape
        sb, (ss, sh, sd) = 0, t.stride()
    if dim != head_dim:
        raise ValueError("%s: expected (batch, tokens, heads, %d) or (tokens, heads, %d), got %s"
                         % (name, head_dim, head_dim, tuple(shape)))
    if sd != 1 and t.numel():
        raise ValueError("%s: the values of a head must be contiguous" % name)
    return batch, tokens, heads, (t.data_ptr(), sb, ss, sh)


def _vector(name: str, t: torch.Tensor, rope: Rotary, index: int) -> int:
    if t.dtype is not torch.float32:
        raise TypeError("%s: expected a f32 tensor, got %s" % (name, t.dtype))
    if t.shape != rope.vector_shape or not t.is_contiguous():
        raise ValueError("%s: expected %d contiguous values, got %s" % (name, rope.head_dim, tuple(t.shape)))
    if t.get_device() != index:
        raise ValueError("%s is on %s, not with the other tensors" % (name, t.device))
    return t.data_ptr()


def _head_call(entry: str, q, k, rope: Rotary, positions, q_out, k_out, stream, inverse=0, eps=0.0, q_weight=None,
               k_weight=None, backward=False, dyq=None, dyk=None, dwq=None, dwk=None, workspace=None) -> None:
    """Checks the tensors of a gemm_epi_qk_args, packs it and calls `entry` on
    the current (or given) stream of their device."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("q and k are both None")
    shape, dtype, index, head_dim = first.shape, first.dtype, first.get_device(), rope.head_dim
    type_code = HEAD_TYPES.get(dtype)
    if type_code is None:
        raise TypeError("%s: expected a bf16 or fp32 tensor, got %s" % ("q" if q is not None else "k", dtype))
    q_heads = k_heads = 0
    tq = tqo = tdq = tk = tko = tdk = _NO_HEADS
    if q is not None:
        batch, tokens, q_heads, tq = _head_input("q", q, shape, head_dim)
        if q_out is not None:
            tqo = _heads("dq" if backward else "q_out", q_out, shape, dtype, index)
        elif not backward:
            raise ValueError("q_out is missing (pass q itself to work in place)")
        if backward and dyq is not None:
            tdq = _heads("dyq", dyq, shape, dtype, index)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k is not None:
        k_shape = k.shape
        k_batch, k_tokens, k_heads, tk = _head_input("k", k, k_shape, head_dim)
        if q is None:
            batch, tokens = k_batch, k_tokens
        elif k_batch != batch or k_tokens != tokens or len(k_shape) != len(shape) or k.dtype is not dtype:
            raise ValueError("q %s %s and k %s %s do not belong together" % (dtype, tuple(shape), k.dtype, tuple(k_shape)))
        elif k.get_device() != index:
            raise ValueError("k is on %s, not with the other tensors" % k.device)
        if k_out is not None:
            tko = _heads("dk" if backward else "k_out", k_out, k_shape, dtype, index)
        elif not backward:
            raise ValueError("k_out is missing (pass k itself to work in place)")
        if backward and dyk is not None:
            tdk = _heads("dyk", dyk, k_shape, dtype, index)
    elif k_out is not None:
        raise ValueError("k_out without k")
    if backward and ((dyq is None) != (q is None) or (dyk is None) != (k is None)):
        raise ValueError("a gradient and its input (dyq and q, dyk and k) must be given together")
    steps = rope._steps
    if steps.get_device() != index:
        raise ValueError("the rotary steps are on %s, q and k on %s" % (steps.device, first.device))
    at = wide = pos_stride = ws = ws_bytes = wq = wk = dq_at = dk_at = 0
    if positions is not None:
        at, wide, pos_stride = _positions(positions, batch, tokens, index)
    if q_weight is not None:
        wq = _vector("q_weight", q_weight, rope, index)
    if k_weight is not None:
        wk = _vector("k_weight", k_weight, rope, index)
    if backward:
        if dwq is not None:
            dq_at = _vector("dwq", dwq, rope, index)
        if dwk is not None:
            dk_at = _vector("dwk", dwk, rope, index)
        if workspace is not None:
            if workspace.get_device() != index or not workspace.is_contiguous():
                raise ValueError("workspace: expected a contiguous tensor with the others")
            ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    packed = _QK_ARGS.pack(batch, tokens, q_heads, k_heads, head_dim, rope.rotary_dim, rope.layout_code, type_code,
                           *tq, *tk, *tqo, *tko, *tdq, *tdk, steps.data_ptr(), at, pos_stride, wide, inverse,
                           rope.amplitude, eps, wq, wk, dq_at, dk_at, ws, ws_bytes)
    if index < 0:
        raise ValueError("expected CUDA tensors, got %s" % first.device)
    fn = _head_entries.get(entry) or _head_entry(entry)
    if index == _current_device():
        status = fn(packed, _raw_stream(index) if stream is None else stream.cuda_stream)
    else:
        status = _call_on(first, stream, lambda s: fn(packed, s))
    if status:
        N.check(status)


def _positions(p: torch.Tensor, batch: int, tokens: int, index: int):
    """(pointer, 1 if 64-bit, batch stride) of a (tokens,) or (batch, tokens) tensor."""
    dtype, shape, st = p.dtype, p.shape, p.stride()
    if dtype is not torch.int32 and dtype is not torch.int64:
        raise TypeError("positions: expected an int32 or int64 tensor, got %s" % dtype)
    if p.get_device() != index:
        raise ValueError("positions are on %s, not with the other tensors" % p.device)
    if shape == (batch, tokens):
        stride = st[0] if batch > 1 else 0
    elif shape == (tokens,):
        stride = 0
    else:
        raise ValueError("positions: expected (%d,) or (%d, %d), got %s" % (tokens, batch, tokens, tuple(shape)))
    if tokens > 1 and st[-1] != 1:
        raise ValueError("positions: the positions of a sequence must be contiguous")
    return p.data_ptr(), 1 if dtype is torch.int64 else 0, stride


def rotary(q, k, rope: Rotary, positions=None, *, q_out=None, k_out=None, inverse: bool = False, stream=None) -> None:
    """gemm_epi_rotary: q and k (either may be None) rotated by their tokens'
    positions into q_out and k_out, which may be q and k themselves.

    q: (batch, tokens, heads, head_dim) or (tokens, heads, head_dim), bf16 or
    fp32, any strides over contiguous heads (a transposed view where heads are
    outside tokens); k the same with its own number of heads.  positions: int32
    or int64, (tokens,) or (batch, tokens); None counts every sequence from 0.
    inverse=True applies the transpose: the backward pass, from the gradients
    of q_out and k_out to those of q and k.  Asynchronous."""
    _head_call("gemm_epi_rotary", q, k, rope, positions, q_out, k_out, stream, 1 if inverse else 0)


def qk_norm_rotary(q, k, rope: Rotary, positions=None, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                   q_out=None, k_out=None, stream=None) -> None:
    """gemm_epi_qk_norm_rotary: each head of q and k divided by its root mean
    square (plus eps), multiplied by the fp32 weight (None: 1) and rotated, in
    one pass; arguments as for rotary().  Asynchronous."""
    _head_call("gemm_epi_qk_norm_rotary", q, k, rope, positions, q_out, k_out, stream, 0, eps, q_weight, k_weight)


def qk_norm_rotary_workspace(head_dim: int) -> int:
    """Bytes of workspace qk_norm_rotary_backward needs for dwq or dwk."""
    return int(N.load().gemm_epi_qk_norm_rotary_workspace_size(head_dim))


def qk_norm_rotary_backward(dyq, dyk, q, k, rope: Rotary, positions=None, *, q_weight=None, k_weight=None,
                            eps: float = 1e-6, dq=None, dk=None, dwq=None, dwk=None, workspace=None,
                            stream=None) -> None:
    """gemm_epi_qk_norm_rotary_backward: from the gradients dyq and dyk of
    qk_norm_rotary's outputs and its inputs q and k, the gradients of q and k
    into dq and dk (which may be the memory of q or dyq, k or dyk) and those of
    the weights, summed over batch, tokens and heads, into the fp32 dwq and dwk
    (overwritten).  Each of the four may be None; dwq and dwk need a workspace
    of qk_norm_rotary_workspace(head_dim) bytes that no call running at the same
    time (another stream's, another graph's) shares.  Asynchronous."""
    _head_call("gemm_epi_qk_norm_rotary_backward", q, k, rope, positions, dq, dk, stream, 0, eps, q_weight, k_weight,
               True, dyq, dyk, dwq, dwk, workspace)


class Dropout:
    """A dropout probability, the seed its masks are drawn from and the step,
    which lies in device memory.

    p is rounded to a multiple of 2^-16 and cannot be changed later: plans made
    with the object hold it.  What stays is scaled by the inverse of the share
    that stays, so that means are kept.  The mask of a call depends on p, seed,
    step and the call's `site` (and the element's row and column), nothing else: a
    backward pass with the same ones drops what its forward pass dropped.
    advance() counts the step on, on the current stream; captured into a graph,
    each replay draws masks of its own.
    """

    def __init__(self, p: float, seed: int = 0, step: int = 0, device="cuda"):
        if not 0.0 <= p <= 1.0:
            raise ValueError("p must be in [0, 1], got %r" % (p,))
        if not 0 <= seed < 2 ** 64 or not 0 <= step < 2 ** 63:
            raise ValueError("seed must be in [0, 2^64) and step in [0, 2^63), got %r and %r" % (seed, step))
        self._p = float(p)
        self._threshold = round(self._p * 65536)
        self.seed = int(seed)
        self.step = torch.tensor([step], dtype=torch.int64).to(device)

    @property
    def p(self) -> float:
        return self._p

    @property
    def threshold(self) -> int:
        """Of the 65536 values an element's number has, those that drop it."""
        return self._threshold

    @property
    def step(self) -> torch.Tensor:
        """The device's step, one int64, of which the masks take the low 32 bits;
        it may be written to, or another tensor put in its place (one that
        several share, say)."""
        return self._step

    @step.setter
    def step(self, t: torch.Tensor) -> None:
        # checked here, once, so that no call has to: the kernels read it
        if t.dtype is not torch.int64 or t.shape != (1,):
            raise ValueError("step: expected 1 int64 value, got %s %s" % (t.dtype, tuple(t.shape)))
        self._step = t

    def advance(self, steps: int = 1) -> None:
        """The next step's masks: adds to the step in device memory."""
        self._step.add_(steps)


# Packed in one step, as _QK_ARGS.
_DROPOUT_ARGS = struct.Struct("@qqiQQIiQqQqQq")
_LAYER_NORM_ARGS = struct.Struct("@qqifQQIiQqQqQqQqQQQQ")
_LAYER_NORM_BWD_ARGS = struct.Struct("@qqiQQIiQqQqQqQqQqQQQQQQN")
assert _DROPOUT_ARGS.size == ctypes.sizeof(N.gemm_epi_dropout_args)
assert _LAYER_NORM_ARGS.size == ctypes.sizeof(N.gemm_epi_layer_norm_args)
assert _LAYER_NORM_BWD_ARGS.size == ctypes.sizeof(N.gemm_epi_layer_norm_bwd_args)
_NO_ROWS = (0, 0)
_NO_MASK = (0, 0, 0, 0)


def _first_rows(name: str, t: torch.Tensor):
    """(shape, dtype, type code, rows, columns, device index, (pointer, row
    stride)) of the tensor a call's others are checked against."""
    shape, dtype = t.shape, t.dtype
    code = HEAD_TYPES.get(dtype)
    if code is None:
        raise TypeError("%s: expected a bf16 or fp32 tensor, got %s" % (name, dtype))
    if len(shape) == 2:
        rows, cols = shape
    elif shape:
        rows, cols = 1, shape[-1]
        for n in shape[:-1]:
            rows *= n
    else:
        raise ValueError("%s: expected (..., columns), got a scalar" % name)
    at = (t.data_ptr(), cols) if t.is_contiguous() else _row_stride(name, t, shape)
    return shape, dtype, code, rows, cols, t.get_device(), at


def _row_stride(name: str, t: torch.Tensor, shape):
    """(pointer, stride between rows) of a (..., columns) tensor whose rows are
    evenly spaced."""
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1 and t.numel():
        raise ValueError("%s: the values of a row must be contiguous" % name)
    if len(st) == 2:
        return t.data_ptr(), st[0]
    ld, spanned = shape[-1], None  # of the leading dimensions of more than one step, from the last
    for n, s in zip(reversed(shape[:-1]), reversed(st[:-1])):
        if n == 1:
            continue
        if spanned is None:
            ld = s
        elif s != spanned and t.numel():
            raise ValueError("%s: its rows are not evenly spaced (strides %s)" % (name, st))
        spanned = s * n
    return t.data_ptr(), ld


def _rows(name: str, t: torch.Tensor, shape, dtype, index: int):
    """(pointer, row stride) of a tensor of the first one's shape, type and
    device, checked."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError("%s: %s %s does not match %s %s" % (name, t.dtype, tuple(t.shape), dtype, tuple(shape)))
    if t.get_device() != index:
        raise ValueError("%s is on %s, not with the other tensors" % (name, t.device))
    if t.is_contiguous():  # a third of the time that strides take
        return t.data_ptr(), shape[-1]
    return _row_stride(name, t, shape)


def _values(name: str, t: torch.Tensor, n: int, index: int) -> int:
    """Pointer of n contiguous fp32 values on device `index`, checked."""
    if t.dtype is not torch.float32:
        raise TypeError("%s: expected a f32 tensor, got %s" % (name, t.dtype))
    if t.numel() != n or not t.is_contiguous():
        raise ValueError("%s: expected %d contiguous values, got %s" % (name, n, tuple(t.shape)))
    if t.get_device() != index:
        raise ValueError("%s is on %s, not with the other tensors" % (name, t.device))
    return t.data_ptr()


def _mask(rng: Dropout, site: int, index: int):
    """(step, seed, site, threshold) of a gemm_epi_mask."""
    threshold = rng._threshold
    if threshold == 0:
        return _NO_MASK
    step = rng._step
    if step.get_device() != index:
        raise ValueError("the dropout step is on %s, not with the other tensors" % step.device)
    if not 0 <= site < 2 ** 32:
        raise ValueError("site must be in [0, 2^32), got %r" % (site,))
    return step.data_ptr(), rng.seed, site, threshold


def _call_packed(entry: str, packed: bytes, first: torch.Tensor, index: int, stream) -> None:
    if index < 0:
        raise ValueError("expected CUDA tensors, got %s" % first.device)
    fn = _head_entries.get(entry) or _head_entry(entry)
    if index == _current_device():
        status = fn(packed, _raw_stream(index) if stream is None else stream.cuda_stream)
    else:
        status = _call_on(first, stream, lambda s: fn(packed, s))
    if status:
        N.check(status)


def dropout(x, rng: Dropout, *, out, residual=None, site: int = 0, stream=None) -> None:
    """gemm_epi_dropout: x with its elements dropped by rng's mask of `site`, plus
    the residual, into `out`.

    x: (..., columns), bf16 or fp32, rows of contiguous values evenly spaced
    (expanded rows among them); the others the same.  out may be x or residual.
    The backward pass is the same call on out's gradient, without the residual,
    whose own gradient is out's.  Asynchronous."""
    shape, dtype, code, rows, cols, index, tx = _first_rows("x", x)
    _call_packed("gemm_epi_dropout", _DROPOUT_ARGS.pack(
        rows, cols, code, *_mask(rng, site, index), *tx,
        *(_NO_ROWS if residual is None else _rows("residual", residual, shape, dtype, index)),
        *_rows("out", out, shape, dtype, index)), x, index, stream)


def layer_norm(x, *, weight=None, bias=None, eps: float = 1e-5, out, residual=None, dropout: Optional[Dropout] = None,
               site: int = 0, sum_out=None, mean=None, rstd=None, stream=None) -> None:
    """gemm_epi_layer_norm: h = x, dropped by `dropout`'s mask of `site`, plus the
    residual; (h - mean(h)) / sqrt(var(h) + eps) * weight + bias into `out`, each
    row over its columns, in one pass.

    Tensors as for dropout(); weight and bias: fp32, one value per column (None:
    1 and 0).  sum_out takes h, mean and rstd (fp32, one value per row) its
    statistics: what layer_norm_backward reads.  out and sum_out may each be x
    or residual.  Asynchronous."""
    if sum_out is not None and residual is None and dropout is None:
        raise ValueError("sum_out without residual or dropout is x itself")
    shape, dtype, code, rows, cols, index, tx = _first_rows("x", x)
    _call_packed("gemm_epi_layer_norm", _LAYER_NORM_ARGS.pack(
        rows, cols, code, eps, *(_NO_MASK if dropout is None else _mask(dropout, site, index)), *tx,
        *(_NO_ROWS if residual is None else _rows("residual", residual, shape, dtype, index)),
        *_rows("out", out, shape, dtype, index),
        *(_NO_ROWS if sum_out is None else _rows("sum_out", sum_out, shape, dtype, index)),
        0 if weight is None else _values("weight", weight, cols, index),
        0 if bias is None else _values("bias", bias, cols, index),
        0 if mean is None else _values("mean", mean, rows, index),
        0 if rstd is None else _values("rstd", rstd, rows, index)), x, index, stream)


def layer_norm_workspace(cols: int) -> int:
    """Bytes of workspace layer_norm_backward needs for dw or db."""
    return int(N.load().gemm_epi_layer_norm_backward_workspace_size(cols))


def layer_norm_backward(dy, x, mean, rstd, *, weight=None, dx=None, dw=None, db=None, add=None,
                        dropout: Optional[Dropout] = None, site: int = 0, d_residual=None, workspace=None,
                        stream=None) -> None:
    """gemm_epi_layer_norm_backward: from the gradient dy of layer_norm's out, the
    normalised sum x (its sum_out, or its x where nothing was added or dropped)
    and the statistics it gave, the gradient g of that sum, plus `add`, which
    reaches it past the norm: into d_residual as it is and into dx with the
    forward pass's mask applied (`dropout` and `site` as there; None: dx is g).
    dw and db (fp32, overwritten) take the weight's and bias's gradients, summed
    over the rows.  Each of the four may be None; dx and d_residual may be the
    memory of an input.  dw and db need a workspace of layer_norm_workspace(cols)
    bytes that no call running at the same time (another stream's, another
    graph's) shares.  Asynchronous."""
    shape, dtype, code, rows, cols, index, tdy = _first_rows("dy", dy)
    if mean is None or rstd is None:
        raise ValueError("mean and rstd, which the forward pass gave, are needed")
    ws = ws_bytes = 0
    if workspace is not None:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace: expected a contiguous tensor with the others")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call_packed("gemm_epi_layer_norm_backward", _LAYER_NORM_BWD_ARGS.pack(
        rows, cols, code, *(_NO_MASK if dropout is None else _mask(dropout, site, index)), *tdy,
        *_rows("x", x, shape, dtype, index), *(_NO_ROWS if add is None else _rows("add", add, shape, dtype, index)),
        *(_NO_ROWS if dx is None else _rows("dx", dx, shape, dtype, index)),
        *(_NO_ROWS if d_residual is None else _rows("d_residual", d_residual, shape, dtype, index)),
        0 if weight is None else _values("weight", weight, cols, index), _values("mean", mean, rows, index),
        _values("rstd", rstd, rows, index), 0 if dw is None else _values("dw", dw, cols, index),
        0 if db is None else _values("db", db, cols, index), ws, ws_bytes), dy, index, stream)
