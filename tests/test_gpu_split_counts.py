"""Projections whose tiles are shared over K by a given number of CTAs, every
number from 2 to 8 for 32, 64 and 128 rows and every head size (needs a GB300).

A forced number of CTAs runs or is refused, so a run that succeeds took the
number under test.  Operands and bounds are test_gpu_head_programs': products
that add up exactly in fp32, so that one loop over all of K gives the same bits."""
import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import native

from test_gpu_head_programs import NORM, ROT, VARIANTS, Problem

pytestmark = pytest.mark.gpu

DEV = "cuda"
SPLIT = native.GEMM_EPI_DEBUG_FORCE_SPLIT
INTERP = native.GEMM_EPI_DEBUG_FORCE_INTERPRETER
# Shared memory under the staging buffers: four stages of a 128 x 64 and a 256 x 64 bf16 block.
RING = 4 * (128 + 256) * 64 * 2


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    assert torch.cuda.is_available()
    return cuda_lib


def has_room(rows, d, n):
    """A CTA receives every other one's sums of its pieces (a head by 32 rows
    each), and keeps 4 KB of squares."""
    pieces = 256 // d * (rows // 32)
    return (n - 1) * -(-pieces // n) * d * 32 * 4 + 4096 <= RING


def run_split(p, n, flags=0):
    p.run(SPLIT(n) | flags)
    assert p.plan.query_status(p.out.workspace) == native.GEMM_EPI_OK
    return p.out.C.clone()


# rows a tile's A box holds: 32, 64, 128 (the last also ragged over three tiles)
ROWS = [(20, 32), (50, 64), (129, 128), (300, 128)]
# head size, q and k heads: four tiles or fewer in a row of them
HEADS = [(32, 20, 4), (64, 8, 2), (128, 5, 2), (256, 2, 1)]


@pytest.mark.parametrize("n", range(2, 9))
@pytest.mark.parametrize("d,hq,hk", HEADS)
@pytest.mark.parametrize("m,rows", ROWS)
def test_every_number_of_ctas(m, rows, d, hq, hk, n):
    p = Problem(NORM, m, 1032, hq, hk, d, d, "half")  # 17 K-blocks: uneven shares for every n
    if not has_room(rows, d, n):
        with pytest.raises(native.GemmEpiError, match="do not fit") as err:
            p.run(SPLIT(n))
        assert err.value.status == native.GEMM_EPI_ERR_UNSUPPORTED
        return
    got = run_split(p, n)
    p.check()
    interpreted = run_split(p, n, INTERP)
    p.run(VARIANTS["1sm"])
    torch.cuda.synchronize()
    assert torch.equal(got, p.out.C) and torch.equal(got, interpreted)


@pytest.mark.parametrize("n", range(2, 9))
@pytest.mark.parametrize("m", [20, 50, 129])
def test_every_output_of_the_program(m, n):
    """Row and column statistics are added up over the cluster's CTAs."""
    program = ("bias", "head_rms:1e-4", "col_scale", "rotary", "amax", "store_bf16", "store_e4m3", "row_rms", "col_sum")
    p = Problem(program, m, 1032, 5, 2, 64, 64, "interleaved")
    got = run_split(p, n)
    p.check()
    c8, amax, row, col = (t.clone() for t in (p.out.C8, p.out.amax, p.out.row_out, p.out.col_out))
    p.run(VARIANTS["1sm"])
    torch.cuda.synchronize()
    assert torch.equal(got, p.out.C) and torch.equal(c8, p.out.C8) and torch.equal(amax, p.out.amax)
    # fp32 atomics in any order: sums of n_out squares, and of m values
    assert bool(((row - p.out.row_out).abs() <= (p.n + 8) * 2.0 ** -23 * p.out.row_out.abs()).all())
    y, mag = p.want()
    assert bool(((col - p.out.col_out).double().cpu().abs() <= m * 2.0 ** -23 * mag[0].sum(0)).all())


@pytest.mark.parametrize("n", range(2, 9))
@pytest.mark.parametrize("m", [20, 50, 129])
def test_every_number_of_ctas_with_8_bit_operands(m, n):
    p = Problem(NORM, m, 2064, 5, 2, 64, 64, "half", in_type="e4m3")  # 17 K-blocks of 128
    got = run_split(p, n)
    p.check()
    p.run(VARIANTS["1sm"])
    torch.cuda.synchronize()
    assert torch.equal(got, p.out.C)


@pytest.mark.parametrize("m", [40, 300])
@pytest.mark.parametrize("form", ["split2", "split4", "1sm", "2sm", "interp1sm", "default"])
def test_dequantisation_factors_on_every_main_loop(m, form):
    """Powers of two, so the accumulator stays exact; the head's norm comes after them."""
    flags = SPLIT(int(form[5:])) if form.startswith("split") else VARIANTS[form]
    p = Problem(("head_rms:1e-2", "col_scale", "rotary", "store_bf16"), m, 2048, 3, 1, 128, 128, "half", in_type="e4m3")
    p.run(flags, a_scale_inv=torch.tensor([0.5], device=DEV), b_scale_inv=torch.tensor([0.0625], device=DEV))
    p.A64, p.B64 = p.A64 * 0.5, p.B64 * 0.0625
    p.check()


def test_the_number_forced_is_the_number_that_runs():
    """Values whose sums round: each number of CTAs adds them in an order of its
    own, the same every time, so some of 230 thousand results differ in a bit."""
    p = Problem(ROT, 128, 2056, 10, 2, 128, 128, "half")
    p.A = torch.randn(128, 2056, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).bfloat16()
    outs = {}
    for n in range(2, 9):
        if has_room(128, 128, n):
            outs[n] = run_split(p, n)
            assert torch.equal(outs[n], run_split(p, n))
    assert len(outs) >= 5
    values = list(outs.values())
    assert not any(torch.equal(a, b) for i, a in enumerate(values) for b in values[:i])


def test_split_refusals():
    p = Problem(ROT, 40, 192, 2, 1, 128, 128, "half")
    run_split(p, 3)
    for flags in (SPLIT(4), SPLIT(3) | native.GEMM_EPI_DEBUG_FORCE_1SM, SPLIT(3) | native.GEMM_EPI_DEBUG_FORCE_2SM):
        with pytest.raises(native.GemmEpiError) as err:
            p.run(flags)
        assert err.value.status == native.GEMM_EPI_ERR_UNSUPPORTED
    for program in (("store_bf16",), ("gelu_tanh", "store_bf16")):
        bare = Problem(program, 40, 1024, 2, 1, 128, 128, "half")
        with pytest.raises(native.GemmEpiError) as err:
            bare.run(SPLIT(2))
        assert err.value.status == native.GEMM_EPI_ERR_UNSUPPORTED
    many = Problem(ROT, 4096, 1024, 6, 2, 128, 128, "half")  # 160 tiles
    with pytest.raises(native.GemmEpiError, match="do not fit"):
        many.run(SPLIT(2))
