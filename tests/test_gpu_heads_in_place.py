"""The head operators over their own inputs, seen through two views (needs a GB300)."""
import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("rot", [64, 32])
def test_views_that_differ_in_single_steps(cuda_lib, rot):
    """A decode step: q read as the transpose of (batch, heads, 1, d), written
    through a (batch, 1, heads, d) view of the same memory."""
    B, H, D = 3, 5, 64
    x = torch.randn(B, H, 1, D, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).bfloat16()
    rope, pos = api.Rotary(D, rot, device=DEV), torch.tensor([[3], [70], [11]], device=DEV, dtype=torch.int32)
    for fn in (api.rotary, api.qk_norm_rotary):
        want, buf = torch.empty(B, 1, H, D, dtype=x.dtype, device=DEV), x.clone()
        fn(x.transpose(1, 2), None, rope, pos, q_out=want)
        q, out = buf.transpose(1, 2), buf.view(B, 1, H, D)
        assert q.stride() != out.stride()
        fn(q, None, rope, pos, q_out=out)
        torch.cuda.synchronize()
        assert torch.equal(buf.view(B, 1, H, D), want)
