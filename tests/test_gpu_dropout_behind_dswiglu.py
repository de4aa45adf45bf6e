"""Programs that drop the output columns of DSWIGLU, twice as many as the tile
has accumulator columns (needs a GB300).

p = 0.5 doubles what stays, which no rounding disturbs: the program gives exactly
twice the values of the one without dropout where the mask of the stored matrix
keeps them."""
import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api

from test_gpu_dropout_programs import DEV, VARIANTS, Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    assert torch.cuda.is_available()
    return cuda_lib


PROGRAMS = [
    ("dswiglu", "dropout", "store_bf16"),
    ("alpha", "dswiglu:4", "dropout", "store_bf16"),
    ("dswiglu:16", "dropout", "relu", "store_bf16"),
    ("dswiglu", "dropout", "store_bf16", "store_e4m3"),
]


# part tiles, one tile, ragged columns, several tiles to a CTA on either main loop
@pytest.mark.parametrize("m,n,k", [(1, 16, 64), (129, 256, 72), (300, 528, 128), (2565, 2576, 64)])
@pytest.mark.parametrize("variant", sorted(VARIANTS))
@pytest.mark.parametrize("program", PROGRAMS, ids="+".join)
def test_output_columns(program, variant, m, n, k):
    p = Problem(program, m, n, k)
    assert p.n_out == 2 * n
    got = p.run(program, VARIANTS[variant]).C[..., :2 * n]
    plain = p.run([s for s in program if s != "dropout"], VARIANTS[variant]).C[..., :2 * n]
    assert torch.equal(got, torch.where(p.keep(2 * n), 2 * plain, torch.zeros_like(plain)))


def test_same_mask_as_the_stored_matrix():
    p = Problem(("dswiglu", "dropout", "store_bf16"), 257, 520, 64)
    plain = p.run(["dswiglu", "store_bf16"]).C[0, :, :1040]
    stored = torch.empty(257, 1040, dtype=torch.bfloat16, device=DEV)
    api.dropout(plain, p.rng, out=stored, site=9)
    assert torch.equal(p.run(p.program, site=9).C[0, :, :1040], stored)


def test_batched():
    p = Problem(("dswiglu", "dropout", "store_bf16"), 200, 264, 64, batch=3)
    plain = p.run(["dswiglu", "store_bf16"]).C[..., :528]
    got = p.run(p.program).C[..., :528]
    assert torch.equal(got, torch.where(p.keep(528), 2 * plain, torch.zeros_like(plain)))
