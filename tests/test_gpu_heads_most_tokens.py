"""The largest number of tokens the head operators take (needs a GB300 with 10 GB free)."""
import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_two_to_the_31_minus_one_tokens(cuda_lib):
    """Heads of 2 values, every token the same: the last tokens (and some in
    between) are those of a short call at their positions."""
    n, d = 2 ** 31 - 1, 2
    rope = api.Rotary(d, layout="interleaved", base=10000.0, device=DEV)
    one = torch.tensor([0.75, -1.5], device=DEV).bfloat16().reshape(1, 1, d)
    y = torch.empty(n, 1, d, dtype=torch.bfloat16, device=DEV)
    api.rotary(one.expand(n, 1, d), None, rope, q_out=y)
    for first, count in ((0, 1000), (2 ** 30 - 500, 1000), (n - 1000, 1000)):
        pos = torch.arange(first, first + count, device=DEV)
        want = torch.empty(count, 1, d, dtype=torch.bfloat16, device=DEV)
        api.rotary(one.expand(count, 1, d), None, rope, pos, q_out=want)
        torch.cuda.synchronize()
        assert torch.equal(y[first:first + count], want)
