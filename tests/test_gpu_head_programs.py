"""Epilogue programs with head_rms and rotary on the GPU, against the formulas
in 64 bits (needs a GB300).

The operands are small integers over powers of two, so the products add up
exactly in fp32 and the bounds of heads_ref hold for the epilogue alone: one
rounding of the stored value, 2^-18 of |a| + |b| of a rotated pair before it
(pointwise ops in front add a few 2^-24 of their result)."""
import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api, native

import heads_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda"
VARIANTS = {"default": 0, "1sm": native.GEMM_EPI_DEBUG_FORCE_1SM, "2sm": native.GEMM_EPI_DEBUG_FORCE_2SM,
            "interp": native.GEMM_EPI_DEBUG_FORCE_INTERPRETER,
            "interp1sm": native.GEMM_EPI_DEBUG_FORCE_INTERPRETER | native.GEMM_EPI_DEBUG_FORCE_1SM}

ROT = ("rotary", "store_bf16")
NORM = ("head_rms:1e-5", "col_scale", "rotary", "store_bf16")


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    assert torch.cuda.is_available()
    return cuda_lib


class Problem:
    """A projection with hq + hk heads of d columns in front of `rest` others."""

    def __init__(self, program, m, k, hq, hk, d, rot, layout, b_layout="nk", rest=None, batch=1, pos="int32",
                 in_type="bf16", seed=1, far=20000, scaling=None):
        g = torch.Generator(device=DEV).manual_seed(seed)
        ints = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device=DEV).float()  # noqa: E731
        self.program, self.m, self.d, self.rot, self.layout, self.batch = list(program), m, d, rot, layout, batch
        self.heads = hq + hk
        self.n = n = self.heads * d + (hk * d if rest is None else rest)
        names = [p.partition(":")[0] for p in program]
        self.names = names
        lead = (batch,) if batch > 1 else ()
        self.A64 = ints(-3, 3, batch, m, k) / 4
        self.B64 = ints(-2, 2, batch, k, n) / 8
        as_op = lambda t: t.bfloat16() if in_type == "bf16" else t.to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        self.A = as_op(self.A64).reshape(lead + (m, k))
        B = self.B64 if b_layout == "kn" else self.B64.transpose(1, 2)
        self.B = as_op(B.contiguous()).reshape(lead + tuple(B.shape[1:]))
        if b_layout == "kn" and n % 8:  # a row stride in whole 16-byte groups
            ldb = (n + 7) // 8 * 8
            wide = torch.zeros(lead + (k, ldb), dtype=torch.bfloat16, device=DEV)
            wide[..., :n] = self.B
            self.B = wide
        self.ldb = self.B.shape[-1]
        vec = lambda size, mean: (mean + torch.randn(size, generator=g, device=DEV) * 0.2)  # noqa: E731
        self.bias = vec(n, 0.0) if "bias" in names else None
        self.col = vec(n, 1.0) if "col_scale" in names else None
        self.row = vec(batch * m, 1.0) if "row_scale" in names else None
        self.alpha = 0.75 if "alpha" in names else 1.0
        self.pos = None
        if pos:
            self.pos = torch.randint(-far, far, (batch, m), generator=g, device=DEV,
                                     dtype=torch.int32 if pos == "int32" else torch.int64).contiguous()
        self.rope = api.Rotary(d, rot, layout=layout, scaling=scaling, device=DEV) if "rotary" in names else None
        ldc = (n + 7) // 8 * 8 + 8
        self.plan = api.Plan(m, n, k, program, b_layout=b_layout, ldb=self.ldb, ldc=ldc, batch=batch,
                             a_type=in_type, b_type=in_type, rotary=self.rope, head_dim=d, head_cols=self.heads * d)
        self.out = api.allocate_outputs(self.plan, DEV)
        if "store_bf16" in names:
            self.out.C = torch.full((batch, m, ldc), 7.0, dtype=torch.bfloat16, device=DEV)
        self.scaling, self.ldc = scaling, ldc

    def run(self, flags=0, **kw):
        o = self.out
        self.plan.run(self.A, self.B, bias=self.bias, col_scale=self.col, row_scale=self.row, alpha=self.alpha,
                      fp8_scale=2.0, C=o.C, C8=o.C8, amax=o.amax, row_out=o.row_out, col_out=o.col_out,
                      positions=self.pos if self.rope else None, workspace=o.workspace, debug_flags=flags, **kw)

    def want(self):
        """(y after the whole program, what its error is measured against), (batch, m, n) fp64."""
        y = torch.matmul(self.A64.double(), self.B64.double()).cpu()
        mag = y.abs()
        d, heads, m = self.d, self.heads, self.m
        for spec in self.program:
            op, _, arg = spec.partition(":")
            split = lambda t: t[..., :heads * d].reshape(self.batch, m, heads, d)  # noqa: E731
            join = lambda h, t: torch.cat([h.reshape(self.batch, m, heads * d), t[..., heads * d:]], -1)  # noqa: E731
            if op == "alpha":
                y, mag = y * self.alpha, mag * self.alpha
            elif op == "bias":
                y, mag = y + self.bias.double().cpu(), mag + self.bias.double().cpu().abs()
            elif op == "row_scale":
                r = self.row.double().cpu().reshape(self.batch, m, 1)
                y, mag = y * r, mag * r.abs()
            elif op == "col_scale":
                y, mag = y * self.col.double().cpu(), mag * self.col.double().cpu().abs()
            elif op == "relu":
                y = y.clamp_min(0)
            elif op == "head_rms":
                h = split(y)
                r = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + float(arg or 1e-6))
                y, mag = join(h * r, y), join(split(mag) * r, mag)
            elif op == "rotary":
                pos = self.pos.cpu() if self.pos is not None else torch.arange(m).expand(self.batch, m)
                ang = R.Angles(pos, self.rot, self.layout, (self.scaling or {}).get("amplitude", 1.0),
                               scaling=self.scaling)
                y, mag = join(ang.rotate(split(y)), y), join(ang.spread(split(mag)), mag)
        return y, mag

    def check(self):
        torch.cuda.synchronize()
        assert self.plan.query_status(self.out.workspace) == native.GEMM_EPI_OK
        y, mag = self.want()
        if "store_bf16" in self.names:
            R.check(self.out.C[..., :self.n], y, mag, torch.bfloat16, 2.0 ** -18)
            assert bool((self.out.C[..., self.n:] == 7.0).all()), "written past the columns"
        return y, mag


# program, m, k, hq, hk, d, rot, layout
CASES = [
    (ROT, 300, 128, 4, 2, 64, 64, "half"),
    (ROT, 1, 64, 1, 1, 128, 128, "half"),
    (ROT, 130, 72, 3, 1, 128, 64, "half"),
    (ROT, 257, 200, 2, 1, 256, 192, "half"),
    (ROT, 64, 64, 3, 2, 64, 32, "half"),
    (ROT, 200, 64, 5, 3, 32, 32, "half"),
    (ROT, 200, 64, 5, 3, 32, 10, "interleaved"),
    (ROT, 129, 136, 3, 1, 128, 128, "interleaved"),
    (ROT, 70, 64, 1, 2, 256, 70, "interleaved"),
    (("bias", "rotary", "store_bf16"), 333, 264, 7, 1, 64, 64, "interleaved"),
    (NORM, 300, 128, 4, 2, 64, 64, "half"),
    (NORM, 64, 512, 6, 2, 128, 128, "half"),
    (NORM, 3, 40, 2, 1, 256, 256, "half"),
    (NORM, 513, 64, 3, 1, 128, 32, "half"),
    (NORM, 100, 64, 3, 3, 32, 32, "interleaved"),
    (("head_rms:1e-3", "store_bf16"), 140, 64, 3, 1, 128, 128, "half"),
    (("head_rms", "rotary", "store_bf16"), 140, 64, 3, 1, 128, 128, "half"),
    (("alpha", "bias", "row_scale", "head_rms:1e-3", "col_scale", "rotary", "store_bf16"), 200, 96, 3, 1, 128, 128, "half"),
    (("row_scale", "relu", "rotary", "col_scale", "store_bf16"), 200, 96, 3, 1, 64, 64, "interleaved"),
]
IDS = ["%s-%dx%d-h%d+%d-d%d-r%d-%s" % ("+".join(p.partition(":")[0] for p in c[0][:-1]), *c[1:7], c[7]) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("b_layout", ["nk", "kn"])
def test_programs(case, b_layout):
    p = Problem(*case, b_layout=b_layout, pos="int32" if b_layout == "nk" else "int64")
    p.run()
    p.check()


@pytest.mark.parametrize("variant", sorted(VARIANTS))
@pytest.mark.parametrize("case", [CASES[0], CASES[9], CASES[10], CASES[11], CASES[17]],
                         ids=[IDS[i] for i in (0, 9, 10, 11, 17)])
def test_kernel_variants(case, variant):
    p = Problem(*case)
    p.run(VARIANTS[variant])
    p.check()


@pytest.mark.parametrize("rest", [0, 24, 100, 333])
def test_columns_past_the_heads(rest):
    """Any number of columns after the heads, none included, ragged last
    16-byte group included; they pass through unrotated."""
    for program in (ROT, NORM):
        p = Problem(program, 150, 64, 2, 1, 128, 128, "half", rest=rest, b_layout="kn" if rest % 8 else "nk")
        p.run()
        p.check()


def test_no_heads_is_the_rest_of_the_program():
    p = Problem(ROT, 100, 64, 0, 0, 64, 64, "half", rest=200)
    p.run()
    p.check()


def test_default_positions_are_the_rows():
    p = Problem(ROT, 300, 64, 2, 1, 64, 64, "half", pos=None)
    p.run()
    p.check()


def test_scaled_frequencies_and_amplitude():
    p = Problem(NORM, 140, 64, 2, 1, 128, 128, "half",
                scaling=dict(kind="by_parts", factor=8.0, original_length=256.0, amplitude=1.25))
    p.run()
    p.check()


@pytest.mark.parametrize("program", [ROT, NORM])
def test_batched(program):
    """Every problem of a batch has positions of its own."""
    p = Problem(program, 200, 64, 2, 1, 128, 128, "half", batch=3)
    p.run()
    p.check()


@pytest.mark.parametrize("m", [40, 300])
@pytest.mark.parametrize("program", [ROT, NORM])
def test_fp8_operands(program, m):
    p = Problem(program, m, 256, 3, 1, 128, 128, "half", in_type="e4m3")
    p.run()
    p.check()


def test_zero_k_rotates_the_bias():
    p = Problem(("bias", "head_rms:1e-4", "rotary", "store_bf16"), 70, 0, 2, 1, 64, 64, "half")
    p.run()
    p.check()


def test_other_outputs_of_the_program():
    """AMAX, e4m3, row statistics and column sums see the rotated values."""
    p = Problem(("head_rms:1e-5", "col_scale", "rotary", "amax", "store_bf16", "store_e4m3", "row_rms", "col_sum"),
                200, 64, 3, 1, 128, 128, "half")
    p.run()
    y, mag = p.check()
    err = 2.0 ** -18 * mag
    assert abs(p.out.amax.item() - y.abs().max().item()) <= 2.0 ** -17 * mag.max().item()
    codes = p.out.C8.view(torch.float8_e4m3fn).double().cpu().reshape(1, 200, p.n) / 2.0
    assert bool(((codes - y).abs() <= y.abs() * 2.0 ** -4 * (1 + 2.0 ** -6) + err + 2.0 ** -11).all())
    # fp32 sums of 200 values, one atomic per 32 rows
    assert bool(((p.out.col_out.double().cpu() - y[0].sum(0)).abs() <= (err + 200 * 2.0 ** -24 * mag)[0].sum(0)).all())
    c = p.out.C[0, :, :p.n].double().cpu()
    want = 1.0 / torch.sqrt((c * c).mean(-1) + 1e-6)
    assert bool(((p.out.row_out.double().cpu() - want).abs() <= (p.n + 8) * 2.0 ** -24 * want).all())


def test_fused_projection_follows_the_separate_passes():
    """One GEMM with head_rms and rotary in its epilogue against the bare GEMM
    and qk_norm_rotary on its stored columns: they differ by the roundings of
    the stored projection (half a bf16 step of each value, through a norm that
    divides by their own root mean square) and of the result."""
    m, hq, hk, d = 500, 6, 2, 128
    p = Problem(NORM, m, 192, hq, hk, d, 128, "half")
    wq, wk = p.col[:d].clone(), p.col[hq * d:hq * d + d].clone()
    p.col[:hq * d], p.col[hq * d:p.heads * d], p.col[p.heads * d:] = wq.repeat(hq), wk.repeat(hk), 1.0
    p.run()
    _, mag = p.check()
    bare = api.Plan(m, p.n, 192, ["store_bf16"], b_layout="nk")
    out = api.allocate_outputs(bare, DEV)
    bare.run(p.A, p.B, C=out.C, workspace=out.workspace)
    heads = out.C.view(m, -1, d)
    q, k = heads[:, :hq], heads[:, hq:hq + hk]
    api.qk_norm_rotary(q, k, p.rope, p.pos[0], q_weight=wq, k_weight=wk, eps=1e-5, q_out=q, k_out=k)
    torch.cuda.synchronize()
    a, b = p.out.C[0, :, :p.n].double().cpu(), out.C.double().cpu()
    # each value of a pair off by 2^-8 and the norm by as much again, then both results' roundings
    assert bool(((a - b).abs() <= 2.0 ** -6 * mag[0] + 2.0 ** -7 * a.abs()).all())
    assert torch.equal(a[:, p.heads * d:], b[:, p.heads * d:])


def test_training_step_of_a_projection():
    """Forward through the bare GEMM, norm and rotation; backward through their
    transposes and the GEMM with the weight: dX against 64 bits."""
    m, k, hq, hk, d = 320, 256, 4, 2, 64
    p = Problem(("store_bf16",), m, k, hq, hk, d, 64, "half")
    rope = api.Rotary(d, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    n = p.n
    plan = api.Plan(m, n, k, ["store_bf16"], b_layout="nk")
    out = api.allocate_outputs(plan, DEV)
    plan.run(p.A, p.B, C=out.C, workspace=out.workspace)
    heads = out.C.view(m, -1, d)
    q, kk, v = heads[:, :hq], heads[:, hq:hq + hk], heads[:, hq + hk:]
    dy = (torch.randn(m, (hq + 2 * hk), d, generator=g, device=DEV)).bfloat16()
    dqkv = dy.clone()  # v's gradient passes through
    dwq, dwk = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    ws = torch.empty(api.qk_norm_rotary_workspace(d), dtype=torch.uint8, device=DEV)
    api.qk_norm_rotary_backward(dy[:, :hq], dy[:, hq:hq + hk], q, kk, rope, dq=dqkv[:, :hq], dk=dqkv[:, hq:hq + hk],
                                dwq=dwq, dwk=dwk, workspace=ws)
    back = api.Plan(m, k, n, ["store_bf16"], b_layout="kn")  # dX = dQKV @ W, W stored n x k
    bo = api.allocate_outputs(back, DEV)
    back.run(dqkv.view(m, n), p.B, C=bo.C, workspace=bo.workspace)
    torch.cuda.synchronize()
    # autograd in 64 bits over the whole chain, from the same stored projection
    x = p.A64[0].double().cpu().requires_grad_()
    W = p.B64[0].double().cpu()
    y = (x @ W).view(m, -1, d)
    ang = R.Angles(torch.arange(m).reshape(1, m), d, "half")
    qk = ang.rotate(R.norm(y[:, :hq + hk].unsqueeze(0), None, 1e-6))[0]
    (torch.cat([qk, y[:, hq + hk:]], 1) * dy.double().cpu()).sum().backward()
    got, want = bo.C.double().cpu(), x.grad
    # dQKV carries two bf16 roundings (the stored projection's through the norm,
    # and its own): 2^-6 of its terms' magnitudes, added over n columns
    step = (dqkv.double().cpu().view(m, n).abs() * 2.0 ** -6) @ W.abs().T
    assert bool(((got - want).abs() <= step + 2.0 ** -7 * want.abs() + 1e-3).all())


def test_captured_projection_replays_on_new_positions():
    p = Problem(NORM, 64, 128, 4, 2, 128, 128, "half")
    p.run()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        p.run()
    p.pos.add_(777)
    torch.cuda.synchronize()
    gr.replay()
    p.check()


def test_allocation_free_run():
    p = Problem(NORM, 200, 64, 2, 1, 128, 128, "half")
    a = p.plan.args(p.A, p.B, col_scale=p.col, C=p.out.C, positions=p.pos, workspace=p.out.workspace)
    import ctypes
    native.check(p.plan.lib.gemm_epi_run_no_alloc(p.plan.handle, ctypes.byref(a),
                                                  torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    y, mag = p.want()
    R.check(p.out.C[..., :p.n], y, mag, torch.bfloat16, 2.0 ** -18)


# Few rows and a long K: a cluster of CTAs shares each tile (K split, partial
# sums exchanged).  m, k, hq, hk, d, rot, layout, batch, b_layout
SPLIT_CASES = [
    (1, 4096, 32, 8, 128, 128, "half", 1, "nk"),
    (64, 2048, 32, 8, 128, 128, "half", 1, "nk"),
    (128, 1032, 6, 2, 128, 64, "half", 1, "kn"),
    (130, 2048, 5, 1, 64, 64, "interleaved", 1, "nk"),
    (300, 1024, 2, 1, 256, 256, "half", 1, "kn"),
    (33, 520, 7, 3, 32, 32, "half", 1, "nk"),
    (96, 2056, 1, 0, 64, 64, "half", 1, "nk"),
    (40, 1024, 2, 1, 128, 128, "half", 3, "nk"),
]


@pytest.mark.parametrize("case", SPLIT_CASES, ids=["%dx%d-h%d+%d-d%d-b%d-%s" % (c[0], c[1], c[2], c[3], c[4], c[7], c[8])
                                                   for c in SPLIT_CASES])
@pytest.mark.parametrize("program", [ROT, NORM, ("bias", "head_rms:1e-4", "col_scale", "rotary", "amax", "store_bf16",
                                                 "store_e4m3", "row_rms", "col_sum")], ids=["rotary", "norm", "all"])
def test_split_k(case, program):
    m, k, hq, hk, d, rot, layout, batch, b_layout = case
    p = Problem(program, m, k, hq, hk, d, rot, layout, batch=batch, b_layout=b_layout)
    p.run()
    p.check()
    got = [t.clone() for t in (p.out.C, p.out.C8, p.out.amax) if t is not None]
    sums = [t.clone() for t in (p.out.row_out, p.out.col_out) if t is not None]
    # the sums are exact, so one loop over all of K gives the same bits; the
    # row and column statistics add in another order
    p.run(VARIANTS["1sm"])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, [t for t in (p.out.C, p.out.C8, p.out.amax) if t is not None]))
    for a, b in zip(sums, [t for t in (p.out.row_out, p.out.col_out) if t is not None]):
        torch.testing.assert_close(a, b, rtol=1e-5, atol=1e-4)


# Growing K: from one CTA to a tile up to eight, so that the heads' pieces are
# dealt out to every number of CTAs for 32, 64 and 128 rows of a slab.
GROWING_K = [(40, k, 8, 2, 64) for k in (72, 136, 392, 640, 2000, 2504, 3000, 4096)] + \
            [(300, k, 5, 2, 128) for k in (264, 776, 1400, 2104, 3000, 4096)] + \
            [(20, k, 3, 1, 32) for k in (136, 200, 1032, 2056, 3400, 4096)] + \
            [(129, k, 2, 1, 256) for k in (1032, 1800, 3000, 4096)]


@pytest.mark.parametrize("m,k,hq,hk,d", GROWING_K)
def test_split_k_over_any_number_of_ctas(m, k, hq, hk, d):
    p = Problem(NORM, m, k, hq, hk, d, d, "half")
    p.run()
    p.check()
    got = p.out.C.clone()
    p.run(VARIANTS["1sm"])
    torch.cuda.synchronize()
    assert torch.equal(got, p.out.C)


def test_split_k_fp8_operands():
    p = Problem(NORM, 48, 2048, 6, 2, 128, 128, "half", in_type="e4m3")
    p.run()
    p.check()


def test_split_k_repeats_bit_for_bit():
    """Values whose sums round: the partial sums are added in a fixed order."""
    p = Problem(NORM, 64, 4096, 32, 8, 128, 128, "half")
    p.A = torch.randn(64, 4096, device=DEV).bfloat16()
    got = []
    for _ in range(5):
        p.run()
        got.append(p.out.C.clone())
    torch.cuda.synchronize()
    assert all(torch.equal(got[0], x) for x in got[1:])


def test_split_k_wait_that_runs_out_is_reported():
    """A first load left out: the first CTA's MMA warp waits in vain, every
    CTA of its cluster still passes the cluster barriers, and the status says
    so; the next run is clean."""
    p = Problem(NORM, 64, 2048, 6, 2, 128, 128, "half")
    p.run(native.GEMM_EPI_DEBUG_SKIP_FIRST_LOAD, timeout_ms=20)
    assert p.plan.query_status(p.out.workspace) == native.GEMM_EPI_ERR_TIMEOUT
    p.run()
    p.check()


@pytest.mark.parametrize("m", [40, 300])
def test_dequantisation_factors(m):
    """Powers of two, so the accumulator stays exact: the head's norm is taken
    after them (split over K at 40 rows, one loop at 300)."""
    p = Problem(("head_rms:1e-2", "col_scale", "rotary", "store_bf16"), m, 2048, 3, 1, 128, 128, "half", in_type="e4m3")
    p.run(a_scale_inv=torch.tensor([0.5], device=DEV), b_scale_inv=torch.tensor([0.0625], device=DEV))
    p.A64, want_b = p.A64 * 0.5, p.B64 * 0.0625
    p.B64 = want_b
    p.check()


def test_interpreted_and_compiled_programs_give_the_same_bits():
    """The interpreter works its angles out eight pairs at a time and stages
    its column vectors alike: every rounding is the same."""
    for program in (ROT, NORM, ("bias", "rotary", "store_bf16"), ("row_scale", "rotary", "store_bf16"),
                    ("bias",) + NORM, ("row_scale",) + NORM):
        for m in (48, 200):
            p = Problem(program, m, 1024, 5, 2, 64, 64, "interleaved")
            p.run()
            got = p.out.C.clone()
            p.run(VARIANTS["interp"])
            torch.cuda.synchronize()
            assert torch.equal(got, p.out.C), program
            p.check()
