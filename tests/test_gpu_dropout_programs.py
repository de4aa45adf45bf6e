"""Epilogue programs with dropout on the GPU, and a block's training step of
these with layer norm (needs a GB300).

With p = 0.5 what stays is doubled, which no rounding disturbs: a program with
dropout gives exactly twice the values of the one without it where the mask
keeps them, whatever else the program does.  Other probabilities are compared
with the formula; the operands are small integers over powers of two, whose
products add up exactly in fp32."""
import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api, native

import residual_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
VARIANTS = {"default": 0, "1sm": native.GEMM_EPI_DEBUG_FORCE_1SM, "2sm": native.GEMM_EPI_DEBUG_FORCE_2SM,
            "interp": native.GEMM_EPI_DEBUG_FORCE_INTERPRETER,
            "interp1sm": native.GEMM_EPI_DEBUG_FORCE_INTERPRETER | native.GEMM_EPI_DEBUG_FORCE_1SM}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    assert torch.cuda.is_available()
    return cuda_lib


class Problem:
    def __init__(self, program, m, n, k, b_layout="nk", batch=1, dual=False, in_type="bf16", p=0.5, seed=1):
        g = torch.Generator(device=DEV).manual_seed(seed)
        ints = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device=DEV).float()  # noqa: E731
        self.names = [s.partition(":")[0] for s in program]
        self.m, self.n, self.batch, self.program = m, n, batch, list(program)
        self.A64, self.B64 = ints(-3, 3, batch, m, k) / 4, ints(-2, 2, batch, k, n) / 8
        as_op = lambda t: t.bfloat16() if in_type == "bf16" else t.to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        lead = (batch,) if batch > 1 else ()
        self.A = as_op(self.A64).reshape(lead + (m, k))
        B = (self.B64 if b_layout == "kn" else self.B64.transpose(1, 2)).contiguous()
        self.B, self.B2 = as_op(B).reshape(lead + tuple(B.shape[1:])), None
        if dual:
            self.B2 = self.B[n // 2:].clone() if b_layout == "nk" else self.B[:, n // 2:].contiguous()
            self.B = self.B[:n // 2].clone() if b_layout == "nk" else self.B[:, :n // 2].contiguous()
        self.n_out = api.out_cols(program, n)
        self.ld = (self.n_out + 15) // 16 * 16
        self.bias = torch.randn(max(n, self.n_out), generator=g, device=DEV) if "bias" in self.names else None
        self.aux = torch.randn(batch, m, self.ld, generator=g, device=DEV).to(BF)
        self.rng = api.Dropout(p, seed=77, step=9, device=DEV)
        self.kw = dict(b_layout=b_layout, batch=batch, dual=dual, a_type=in_type, b_type=in_type, ldc=self.ld,
                       ldc8=self.ld, ld_aux=self.ld)
        self.k = k

    def run(self, program, flags=0, site=3, **kw):
        plan = api.Plan(self.m, self.n, self.k, program, dropout=self.rng, **self.kw)
        o = api.allocate_outputs(plan, DEV)
        o.C = torch.full((self.batch, self.m, self.ld), 7.0, dtype=BF, device=DEV)
        if o.C8 is not None:
            o.C8 = torch.full((self.batch, self.m, self.ld), 7, dtype=torch.uint8, device=DEV)
        aux = {name: self.aux for name, ops in (("residual", api.RESIDUAL_OPS), ("preact", api.PREACT_OPS))
               if any(s.partition(":")[0] in ops for s in program)}
        plan.run(self.A, self.B, B2=self.B2, bias=self.bias, alpha=0.75, fp8_scale=0.25, C=o.C, C8=o.C8, amax=o.amax,
                 row_out=o.row_out, col_out=o.col_out, workspace=o.workspace, debug_flags=flags,
                 site=site if "dropout" in program else 0, **aux, **kw)
        assert plan.query_status(o.workspace) == native.GEMM_EPI_OK
        assert bool((o.C[..., self.n_out:] == 7.0).all())
        return o

    def keep(self, width, site=3):
        """The mask of rows counted through the batch."""
        return R.Mask(self.rng, self.batch * self.m, width, site).keep.view(self.batch, self.m, width).to(DEV)


def expanded(keep, g):
    """The mask of accumulator columns on the gate and up columns of DSWIGLU."""
    m, n = keep.shape[-2:]
    return keep.view(-1, m, n // g, 1, g).expand(-1, m, n // g, 2, g).reshape(-1, m, 2 * n)


# program; m, n, k: single CTAs and pairs, part tiles, ragged last columns, several tiles to a CTA
SHAPES = [(300, 520, 128), (1, 8, 64), (129, 256, 72), (513, 1000, 200)]
PROGRAMS = [
    ("dropout", "store_bf16"),
    ("bias", "gelu_tanh", "dropout", "store_bf16"),
    ("alpha", "bias", "dropout", "relu", "store_bf16"),
    ("dropout", "gelu_tanh_grad", "store_bf16"),
    ("dropout", "gelu_tanh_grad", "store_bf16", "col_sum"),
    ("pair_swiglu", "dropout", "store_bf16"),
    ("pair_mul:4", "dropout", "store_bf16"),
    ("dropout", "dswiglu", "store_bf16"),
    ("alpha", "dropout", "dswiglu:4", "store_bf16"),
    ("silu", "dropout", "store_bf16", "store_e4m3", "amax"),
]


@pytest.mark.parametrize("variant", sorted(VARIANTS))
@pytest.mark.parametrize("program", PROGRAMS, ids="+".join)
def test_programs(program, variant):
    for i, (m, n, k) in enumerate(SHAPES):
        p = Problem(program, m, n, k, b_layout="nk" if i % 2 else "kn")
        got = p.run(program, VARIANTS[variant])
        plain = p.run([s for s in program if s != "dropout"], VARIANTS[variant])
        if "dswiglu" in p.names:
            g = int([s for s in program if s.startswith("dswiglu")][0].partition(":")[2] or 1)
            keep = expanded(p.keep(n), g)
        else:
            keep = p.keep(p.n_out)
        C = plain.C[..., :p.n_out]
        want = torch.where(keep, 2 * C, torch.zeros_like(C))
        assert torch.equal(got.C[..., :p.n_out], want), (m, n, k)
        if got.C8 is not None:  # a saturated value stays one; below that the codes of twice the value
            code = lambda t: t[..., :p.n_out].view(torch.float8_e4m3fn).float()  # noqa: E731
            twice = (2 * code(plain.C8)).clamp(-448, 448)
            mild = code(plain.C8).abs() > 2.0 ** -6  # the steps of subnormal codes are not twice as large
            a, b = code(got.C8), torch.where(keep, twice, torch.zeros_like(twice))
            assert torch.equal(a[mild], b[mild])
            assert bool((a[~keep] == 0).all())
            assert float(got.amax) >= float(want.abs().max()) * (1 - 2.0 ** -8)


@pytest.mark.parametrize("variant", sorted(VARIANTS))
@pytest.mark.parametrize("p", [0.1, 0.9, 1.0, 0.0])
@pytest.mark.parametrize("program", [("bias", "dropout", "residual", "store_bf16"), ("dropout", "residual", "store_bf16"),
                                     ("dropout", "store_bf16", "row_rms:1e-3")], ids="+".join)
def test_probabilities(program, p, variant):
    m, n, k = 333, 776, 136
    q = Problem(program, m, n, k, p=p)
    got = q.run(program, VARIANTS[variant])
    y = torch.matmul(q.A64.double(), q.B64.double()).cpu()[0]
    d = torch.zeros_like(y)
    if "bias" in program:
        y = y + q.bias.cpu().double()
        d = R.U * y.abs()
    mask = R.Mask(q.rng, m, n, 3)
    d, y = mask(d) + 2 * R.U * mask(y).abs(), mask(y)
    if "residual" in program:
        y = y + q.aux[0, :, :n].cpu().double()
        d = d + R.U * y.abs()
    R.close(got.C[0, :, :n], y, d, BF, "C")
    if "row_rms:1e-3" in program:  # of the stored values: n squares one after the other, 4 u for the rest
        C = got.C[0, :, :n].cpu().double()
        r = 1.0 / torch.sqrt((C * C).mean(1) + float(torch.tensor(1e-3)))
        R.close(got.row_out, r, (n + 4) * R.U * r, F32, "row_out")


@pytest.mark.parametrize("variant", sorted(VARIANTS))
def test_column_sums(variant):
    """Sums of eighths well inside fp32's 24 bits: exact in any order."""
    p = Problem(("dropout", "store_bf16", "col_sum"), 700, 520, 64)
    got = p.run(p.program, VARIANTS[variant])
    y = torch.matmul(p.A64.double(), p.B64.double())
    want = torch.where(p.keep(520), 2 * y, torch.zeros_like(y)).sum(1)
    assert torch.equal(got.col_out.double().view(-1), want.view(-1))


def test_same_mask_as_the_stored_matrix():
    p = Problem(("dropout", "store_bf16"), 257, 264, 64)
    plain = p.run(["store_bf16"]).C[0, :, :264]
    got = p.run(p.program, site=2 ** 32 - 1).C[0, :, :264]
    stored = torch.empty_like(plain)
    api.dropout(plain, p.rng, out=stored, site=2 ** 32 - 1)
    assert torch.equal(got, stored)
    other = p.run(p.program, site=5).C[0, :, :264]
    assert not torch.equal(other, got)
    p.rng.advance()
    assert not torch.equal(p.run(p.program, site=5).C[0, :, :264], other)


@pytest.mark.parametrize("m,n", [(200, 264), (5, 40)])
def test_batched(m, n):
    """Every problem of a batch has rows of its own."""
    p = Problem(("bias", "dropout", "store_bf16"), m, n, 64, batch=3)
    C = p.run(["bias", "store_bf16"]).C[..., :n]
    got = p.run(p.program).C[..., :n]
    assert torch.equal(got, torch.where(p.keep(n), 2 * C, torch.zeros_like(C)))


@pytest.mark.parametrize("variant", sorted(VARIANTS))
def test_two_weights(variant):
    p = Problem(("pair_swiglu:128", "dropout", "store_bf16"), 300, 512, 64, dual=True)
    C = p.run(["pair_swiglu:128", "store_bf16"], VARIANTS[variant]).C[..., :256]
    got = p.run(p.program, VARIANTS[variant]).C[..., :256]
    assert torch.equal(got, torch.where(p.keep(256), 2 * C, torch.zeros_like(C)))


@pytest.mark.parametrize("variant", sorted(VARIANTS))
def test_fp8_operands(variant):
    p = Problem(("bias", "dropout", "store_bf16"), 300, 528, 128, in_type="e4m3")
    C = p.run(["bias", "store_bf16"], VARIANTS[variant]).C[..., :528]
    got = p.run(p.program, VARIANTS[variant]).C[..., :528]
    assert torch.equal(got, torch.where(p.keep(528), 2 * C, torch.zeros_like(C)))


def test_nothing_is_dropped_of_what_does_not_matter():
    """NaN and infinity of the accumulator are dropped as any value."""
    p = Problem(("dropout", "store_bf16"), 130, 256, 64)
    want = p.run(p.program).C
    p.A[7] = float("nan")
    p.A[9, 3] = float("inf")
    got = p.run(p.program).C
    keep = p.keep(256)
    assert bool((got[~keep] == 0).all()) and bool(got[0, 7][keep[0, 7]].isnan().all())
    rest = [i for i in range(130) if i not in (7, 9)]
    assert torch.equal(got[0, rest], want[0, rest])


def test_without_a_workspace_of_the_callers(cuda_lib):
    import ctypes
    p = Problem(("dropout", "store_bf16"), 130, 256, 64)
    plan = api.Plan(p.m, p.n, p.k, p.program, dropout=p.rng, **p.kw)
    C = torch.empty(p.m, p.ld, dtype=BF, device=DEV)
    a = plan.args(p.A, p.B, C=C, site=3)
    assert cuda_lib.gemm_epi_run_no_alloc(plan.handle, ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(C, p.run(p.program).C[0])


def test_captured_and_replayed():
    """Each replay draws the mask of its step: the step is read when the kernel runs."""
    p = Problem(("bias", "dropout", "store_bf16"), 200, 264, 64)
    plan = api.Plan(p.m, p.n, p.k, p.program, dropout=p.rng, **p.kw)
    o = api.allocate_outputs(plan, DEV)
    o.C = torch.zeros(p.m, p.ld, dtype=BF, device=DEV)
    call = lambda: plan.run(p.A, p.B, bias=p.bias, C=o.C, workspace=o.workspace, site=3)  # noqa: E731
    want = []
    for _ in range(3):
        call()
        want.append(o.C.clone())
        p.rng.advance()
    p.rng.step[0] = 9
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        p.rng.advance()
    for w in want:
        graph.replay()
        assert torch.equal(o.C, w)


def test_training_step_of_a_block():
    """h = residual + D(x W + b), y = LN(h), z = D(gelu(y U + c)) and its gradients by the package's calls --
    projections with dropout, norm, dropout and GEMMs for the weights -- against the formula in 64 bits with the
    same masks.  Every stored tensor between the calls is rounded to bf16 (2^-8 of it), at most six in a row on the
    way to any result, each scaled on by factors of order one: 2^-5 of a result's root mean square bounds the rounded
    chain, with the sums of independent roundings far below it."""
    m, n, f, eps = 264, 512, 1024, 1e-5
    g = torch.Generator(device=DEV).manual_seed(3)
    normal = lambda *s, std=1.0: torch.randn(s, generator=g, device=DEV) * std  # noqa: E731
    x, residual = normal(m, n).to(BF), normal(m, n).to(BF)
    W, U = normal(n, n, std=n ** -0.5).to(BF), normal(f, n, std=n ** -0.5).to(BF)  # stored N x K
    b, c, w1, b1 = normal(n, std=0.1), normal(f, std=0.1), 1 + normal(n, std=0.1), normal(n, std=0.1)
    dz = normal(m, f).to(BF)
    rng = api.Dropout(0.2, seed=5, step=1, device=DEV)
    empty = lambda *s: torch.empty(s, dtype=BF, device=DEV)  # noqa: E731

    def gemm(A, B, program, mm, nn, kk, b_layout="nk", site=0, **kw):
        plan = api.Plan(mm, nn, kk, program, b_layout=b_layout, dropout=rng if "dropout" in program else None)
        o = api.allocate_outputs(plan, DEV)
        plan.run(A, B, C=o.C, col_out=o.col_out, workspace=o.workspace, **({"site": site} if "dropout" in program else {}), **kw)
        return o

    h = gemm(x, W, ["bias", "dropout", "residual", "store_bf16"], m, n, n, site=1, bias=b, residual=residual).C
    y, mean, rstd = empty(m, n), torch.empty(m, device=DEV), torch.empty(m, device=DEV)
    api.layer_norm(h, weight=w1, bias=b1, eps=eps, out=y, mean=mean, rstd=rstd)
    pre = gemm(y, U, ["bias", "store_bf16"], m, f, n, bias=c).C
    z = gemm(y, U, ["bias", "gelu_tanh", "dropout", "store_bf16"], m, f, n, site=2, bias=c).C
    # back: through dropout and GELU of z (a GEMM with the identity stands for the next layer's), then the norm
    eye = torch.eye(f, device=DEV).to(BF)
    o = gemm(dz, eye, ["dropout", "gelu_tanh_grad", "store_bf16", "col_sum"], m, f, f, site=2, preact=pre)
    dpre, dc = o.C, o.col_out
    dy = gemm(dpre, U, ["store_bf16"], m, n, f, b_layout="kn").C
    dt, dres, dw1, db1 = empty(m, n), empty(m, n), torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    api.layer_norm_backward(dy, h, mean, rstd, weight=w1, dx=dt, d_residual=dres, dw=dw1, db=db1, dropout=rng, site=1,
                            workspace=torch.empty(api.layer_norm_workspace(n), dtype=torch.uint8, device=DEV))
    dx = gemm(dt, W, ["store_bf16"], m, n, n, b_layout="kn").C

    leaf = lambda t: t.detach().cpu().double().requires_grad_(True)  # noqa: E731
    X, RES, WW, UU, B_, C_, W1, B1 = (leaf(t) for t in (x, residual, W, U, b, c, w1, b1))
    m1, m2 = R.Mask(rng, m, n, 1), R.Mask(rng, m, f, 2)
    H = m1(X @ WW.t() + B_) + RES
    mu = H.mean(1, keepdim=True)
    Y = (H - mu) / torch.sqrt(((H - mu) ** 2).mean(1, keepdim=True) + eps) * W1 + B1
    Z = m2(torch.nn.functional.gelu(Y @ UU.t() + C_, approximate="tanh"))
    Z.backward(dz.cpu().double())
    for name, got, want in (("h", h, H), ("y", y, Y), ("z", z, Z), ("dc", dc, C_.grad), ("d residual", dres, RES.grad),
                            ("dx", dx, X.grad), ("dw", dw1, W1.grad), ("db", db1, B1.grad)):
        want = want.detach()
        off = (got.cpu().double() - want).square().mean().sqrt() / want.square().mean().sqrt()
        assert float(off) <= 2.0 ** -5, (name, float(off))
