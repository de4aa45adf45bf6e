"""Dropout at each place of a program, over several tiles to a CTA (needs a GB300).

p = 0.5 doubles what stays, which no rounding disturbs, so that a program is
compared bit for bit with the one without dropout or with a shorter one."""
import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api, native

from test_gpu_dropout_programs import BF, DEV, VARIANTS, Problem, expanded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    assert torch.cuda.is_available()
    return cuda_lib


def dropped(t, keep):
    return torch.where(keep, 2 * t, torch.zeros_like(t))


# 21 x 11 tiles of 128 x 256 on 152 SMs, 11 x 11 of 256 x 256 on 76 pairs: masks of
# a CTA's second tile, drawn ahead and between chunks.
M, N_, K = 2565, 2576, 64


@pytest.mark.parametrize("variant", sorted(VARIANTS))
@pytest.mark.parametrize("program", [
    ("dropout", "store_bf16"),
    ("bias", "gelu_tanh", "dropout", "store_bf16"),
    ("dropout", "gelu_tanh_grad", "store_bf16", "col_sum"),
    ("pair_swiglu", "dropout", "store_bf16"),
    ("dropout", "dswiglu", "store_bf16"),
    ("bias", "dropout", "relu", "store_bf16", "store_e4m3"),
], ids="+".join)
def test_several_tiles_to_a_cta(program, variant):
    p = Problem(program, M, N_, K, b_layout="kn")
    got = p.run(program, VARIANTS[variant])
    plain = p.run([s for s in program if s != "dropout"], VARIANTS[variant])
    keep = expanded(p.keep(N_), 1) if "dswiglu" in program else p.keep(p.n_out)
    assert torch.equal(got.C[..., :p.n_out], dropped(plain.C[..., :p.n_out], keep))


@pytest.mark.parametrize("variant", sorted(VARIANTS))
@pytest.mark.parametrize("program", [("bias", "dropout", "residual", "store_bf16"), ("dropout", "residual", "store_bf16")],
                         ids="+".join)
def test_residual_over_several_tiles(program, variant):
    """The products add up to multiples of 1/32 below 16: with bias and residual of eighths, every sum is exact."""
    p = Problem(program, M, N_, K)
    g = torch.Generator(device=DEV).manual_seed(2)
    eighths = lambda t: torch.randint(-32, 33, t.shape, generator=g, device=DEV) / 8  # noqa: E731
    p.aux = eighths(p.aux).to(BF)
    if p.bias is not None:
        p.bias = eighths(p.bias)
    y = torch.matmul(p.A64.double(), p.B64.double())
    if p.bias is not None:
        y = y + p.bias.double()[:N_]
    want = (dropped(y, p.keep(N_)) + p.aux[..., :N_].double()).float().to(BF)
    assert torch.equal(p.run(program, VARIANTS[variant]).C[..., :N_], want)


@pytest.mark.parametrize("variant", sorted(VARIANTS))
@pytest.mark.parametrize("m,n", [(300, 528), (M, N_)])
def test_outputs_in_front_of_it_and_behind(m, n, variant):
    """What stands in front of the op is not dropped, what stands behind it is: the stored matrix whole, its column
    sums and largest magnitude of what stays.  Multiples of 1/32 below 16, doubled, of 2565 rows: every column sum is
    exact in fp32 in any order."""
    p = Problem(("store_bf16", "dropout", "col_sum", "amax"), m, n, 64)
    got = p.run(p.program, VARIANTS[variant])
    y = torch.matmul(p.A64.double(), p.B64.double())
    d = dropped(y, p.keep(n))
    assert torch.equal(got.C[..., :n], y.float().to(BF))
    assert torch.equal(got.col_out.double().view(-1), d.sum((0, 1)))
    assert float(got.amax) == float(d.abs().max())
    before = Problem(("amax", "col_sum", "dropout", "store_bf16"), m, n, 64)
    got = before.run(before.program, VARIANTS[variant])
    assert float(got.amax) == float(y.abs().max())
    assert torch.equal(got.col_out.double().view(-1), y.sum((0, 1)))
    assert torch.equal(got.C[..., :n], d.float().to(BF))


@pytest.mark.parametrize("variant", sorted(VARIANTS))
def test_row_dot_of_what_stays(variant):
    """Rows' products with small integers: exact sums."""
    m, n = 333, 264
    p = Problem(("dropout", "row_dot", "store_bf16"), m, n, 64)
    p.aux = torch.randint(-2, 3, p.aux.shape, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).to(BF)
    got = p.run(p.program, VARIANTS[variant])
    d = dropped(torch.matmul(p.A64.double(), p.B64.double()), p.keep(n))
    assert torch.equal(got.row_out.double().view(-1), (d * p.aux[..., :n].double()).sum(-1).view(-1))


@pytest.mark.parametrize("variant", sorted(VARIANTS))
def test_no_products(variant):
    """K = 0: the bias alone, dropped."""
    m, n = 200, 264
    rng = api.Dropout(0.5, seed=1, device=DEV)
    plan = api.Plan(m, n, 0, ["bias", "dropout", "store_bf16"], dropout=rng)
    o = api.allocate_outputs(plan, DEV)
    bias = torch.randn(n, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    plan.run(None, None, bias=bias, C=o.C, workspace=o.workspace, site=7, debug_flags=VARIANTS[variant])
    y = bias.to(BF).expand(m, n).contiguous()
    want = torch.empty_like(y)
    api.dropout(y, rng, out=want, site=7)
    assert torch.equal(o.C, want)


@pytest.mark.parametrize("variant", sorted(VARIANTS))
@pytest.mark.parametrize("program", [("bias", "gelu_tanh", "dropout", "store_bf16"), ("pair_swiglu", "dropout", "store_bf16"),
                                     ("dropout", "dswiglu", "store_bf16"), ("dropout", "gelu_tanh_grad", "store_bf16")],
                         ids="+".join)
def test_batches_of_several_tiles(program, variant):
    """Rows are counted through the batch, of more tiles than CTAs."""
    p = Problem(program, 519, 776, 64, batch=13)
    got = p.run(program, VARIANTS[variant])
    plain = p.run([s for s in program if s != "dropout"], VARIANTS[variant])
    keep = expanded(p.keep(776), 1) if "dswiglu" in program else p.keep(p.n_out)
    assert torch.equal(got.C[..., :p.n_out], dropped(plain.C[..., :p.n_out], keep))


@pytest.mark.parametrize("variant", ["default", "1sm"])
@pytest.mark.parametrize("program", [("bias", "dropout", "residual", "store_bf16"), ("dropout", "dswiglu", "store_bf16"),
                                     ("pair_swiglu", "dropout", "store_bf16", "store_e4m3")], ids="+".join)
def test_eight_bit_operands(program, variant):
    p = Problem(program, M, 2592, 128, in_type="e4m3")
    plain = p.run([s for s in program if s not in ("dropout", "residual")], VARIANTS[variant]).C[..., :p.n_out]
    got = p.run([s for s in program if s != "residual"], VARIANTS[variant]).C[..., :p.n_out]
    keep = expanded(p.keep(2592), 1) if "dswiglu" in program else p.keep(p.n_out)
    assert torch.equal(got, dropped(plain, keep))
    if "residual" in program:  # zeros added leave it
        p.aux = torch.zeros_like(p.aux)
        assert torch.equal(p.run(program, VARIANTS[variant]).C[..., :p.n_out], got)


def test_two_plans_at_once():
    """Two streams, each with a plan, outputs and a workspace of its own, and one dropout object between them."""
    problems = [Problem(("bias", "gelu_tanh", "dropout", "store_bf16"), 1000, 1032, 64, seed=s) for s in (1, 2)]
    problems[1].rng = problems[0].rng
    want = [p.run(p.program).C.clone() for p in problems]
    plans = [api.Plan(p.m, p.n, p.k, p.program, dropout=p.rng, **p.kw) for p in problems]
    outs = [api.allocate_outputs(plan, DEV) for plan in plans]
    streams = [torch.cuda.Stream() for _ in plans]
    got = [torch.full_like(w, 7.0) for w in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, plan, o, C, s in zip(problems, plans, outs, got, streams):
            plan.run(p.A, p.B, bias=p.bias, C=C, workspace=o.workspace, site=3, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert all(plan.query_status(o.workspace) == native.GEMM_EPI_OK for plan, o in zip(plans, outs))


@pytest.mark.parametrize("k", [64, 512, 4096])
def test_column_sums_follow_the_accumulator(k):
    """Column sums of one row are the accumulator itself, which keeps fewer bits of K products than fp32 additions
    would.  Sums of many rows add to that no more than their own fp32 additions may: 4 m u of the terms' magnitudes
    (m at most one after the other; the rest for a term's roundings on its way)."""
    m, n = 256, 512
    g = torch.Generator(device=DEV).manual_seed(k)
    A = torch.randn(m, k, generator=g, device=DEV).to(BF)
    B = (torch.randn(n, k, generator=g, device=DEV) * 0.02).to(BF)

    def sums(rows):
        plan = api.Plan(rows.shape[0], n, k, ["col_sum"], b_layout="nk")
        o = api.allocate_outputs(plan, DEV)
        plan.run(rows, B, col_out=o.col_out, workspace=o.workspace)
        return o.col_out.double().view(-1)

    each = torch.stack([sums(A[i:i + 1]) for i in range(m)])
    assert bool(((sums(A) - each.sum(0)).abs() <= 4 * m * 2.0 ** -24 * each.abs().sum(0)).all())
