"""The cos and sin that the epilogue's rotation multiplies by, read in fp32
(needs a GB300).

One row, accumulators (1, 0) in every pair: the rotated pair is (cos, sin), and
with one row the fp32 column sums are those values.  Bound: the phase rounded to
23 bits is off by 2^-24 of a turn, 2 pi 2^-24 = 2^-21.35 radians; its product
with pi, below 4, rounds by 2^-23; __cosf and __sinf are off by at most 2^-21.19
and 2^-21.41 on [-pi, pi].  Together 9.2e-7, below 2^-20 = 9.5e-7."""
import math

import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api

import heads_ref as R

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_cos_and_sin_of_the_epilogue(cuda_lib, layout):
    d, batch, k = 256, 400, 8
    g = torch.Generator().manual_seed(0)
    freqs = (torch.rand(d // 2, generator=g, dtype=torch.float64) * 2 * math.pi).tolist()
    pos = torch.randint(0, 1 << 20, (batch, 1), generator=g)
    A = torch.zeros(batch, 1, k, dtype=torch.bfloat16, device=DEV)
    B = torch.zeros(d, k, dtype=torch.bfloat16, device=DEV)
    first = slice(0, d // 2) if layout == "half" else slice(0, d, 2)
    A[..., 0], B[first, 0] = 1.0, 1.0
    plan = api.Plan(1, d, k, ["rotary", "store_bf16", "col_sum"], b_layout="nk", batch=batch, batch_stride_b=0,
                    rotary=api.Rotary(d, freqs=freqs, layout=layout, device=DEV), head_cols=d)
    out = api.allocate_outputs(plan, DEV)
    plan.run(A, B, positions=pos.to(DEV), C=out.C, col_out=out.col_out, workspace=out.workspace)
    torch.cuda.synchronize()
    got = out.col_out.double().cpu().view(batch, d)
    c, s = (got[:, :d // 2], got[:, d // 2:]) if layout == "half" else (got[:, 0::2], got[:, 1::2])
    angle = R.turns_mod_1(pos, torch.tensor(freqs, dtype=torch.float64)).view(batch, d // 2) * 2 * math.pi
    assert (c - torch.cos(angle)).abs().max().item() <= 2.0 ** -20
    assert (s - torch.sin(angle)).abs().max().item() <= 2.0 ** -20
