"""Projections whose heads rotate only in part, with infinities and NaN in the
columns that do not: the other columns have the bits they have without them
(needs a GB300)."""
import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api, native

pytestmark = pytest.mark.gpu

DEV = "cuda"
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    assert torch.cuda.is_available()
    return cuda_lib


# d, rot, layout: the last rotated pair inside a 32-column chunk, or at its end
HEADS = [(32, 10, "interleaved"), (256, 70, "interleaved"), (128, 2, "interleaved"), (64, 32, "interleaved"),
         (128, 64, "half"), (64, 32, "half")]
# m, k, flags: one CTA to a tile, K shared by a cluster, the interpreter
FORMS = {"tile": (300, 64, 0), "pair": (300, 64, native.GEMM_EPI_DEBUG_FORCE_2SM), "split": (40, 1024, 0),
         "interp": (300, 64, native.GEMM_EPI_DEBUG_FORCE_INTERPRETER),
         "interp-split": (40, 1024, native.GEMM_EPI_DEBUG_FORCE_INTERPRETER)}


@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("d,rot,layout", HEADS)
def test_bad_columns_past_the_rotated_part(d, rot, layout, form):
    m, k, flags = FORMS[form]
    heads = 512 // d
    n = heads * d + 40
    g = torch.Generator(device=DEV).manual_seed(1)
    A = torch.randn(m, k, generator=g, device=DEV).bfloat16()
    B = torch.randn(n, k, generator=g, device=DEV).bfloat16()
    bias = torch.randn(n, generator=g, device=DEV)
    bad = bias.clone()
    hit = [rot, rot + 1, (rot + d) // 2, d - 1]
    for i, c in enumerate(hit):
        for h in range(heads):
            bad[h * d + c] = (INF, -INF, NAN)[(i + h) % 3]
    plan = api.Plan(m, n, k, ["bias", "rotary", "store_bf16"], b_layout="nk", head_cols=heads * d,
                    rotary=api.Rotary(d, rot, layout=layout, device=DEV))
    out = api.allocate_outputs(plan, DEV)

    def run(bias):
        plan.run(A, B, bias=bias, C=out.C, workspace=out.workspace, debug_flags=flags)
        assert plan.query_status(out.workspace) == native.GEMM_EPI_OK
        return out.C.clone()

    clean, got = run(bias), run(bad)
    cols = (torch.arange(heads, device=DEV)[:, None] * d + torch.tensor(hit, device=DEV)).flatten()
    want = bad[cols].bfloat16().expand(m, -1)
    assert torch.equal(got[:, cols].nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))
    got[:, cols] = clean[:, cols] = 0.0
    assert torch.equal(got.view(torch.int16), clean.view(torch.int16))
