"""What the Python binding of the head operators checks before a pointer crosses
the C ABI, without a GPU."""
import copy

import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api, build, native as N

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    build.build()
    return N.load()


def test_steps_put_in_place_are_checked(lib):
    """The kernels read rotary_dim / 2 steps of 8 bytes, whatever was put there."""
    rope, other = api.Rotary(64, 32, device="cpu"), api.Rotary(64, 32, base=500.0, device="cpu")
    rope.steps = other.steps.clone()
    assert torch.equal(rope.steps, other.steps)
    assert torch.equal(copy.deepcopy(rope).steps, other.steps)
    for bad in (other.steps[:8], torch.cat([other.steps, other.steps]), other.steps.int(), other.steps.double(),
                other.steps.reshape(2, 8), torch.zeros(32, dtype=torch.int64)[::2]):
        with pytest.raises(ValueError, match="16 contiguous int64"):
            rope.steps = bad
    assert torch.equal(rope.steps, other.steps)
