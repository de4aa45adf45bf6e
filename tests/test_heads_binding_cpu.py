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


def test_a_batch_of_zero_is_one_problem_to_the_checks_too(lib):
    """The C ABI runs M rows for batch 0; the binding asked for no positions and
    let operands of any size through."""
    rope = api.Rotary(64, device="cpu")
    plan = api.Plan(64, 256, 64, ["rotary", "store_bf16"], batch=0, rotary=rope, head_cols=128)
    A, B, C = (torch.zeros(64, n, dtype=BF) for n in (64, 256, 256))
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8)
    pos = torch.zeros(64, dtype=torch.int32)
    assert plan.args(A, B, C=C, workspace=ws, positions=pos).positions == pos.data_ptr()
    with pytest.raises(ValueError, match="positions: expected 64"):
        plan.args(A, B, C=C, workspace=ws, positions=pos[:0])
    with pytest.raises(ValueError, match="A: 8192 bytes"):
        plan.args(A[:32].clone(), B, C=C, workspace=ws, positions=pos)
    with pytest.raises(ValueError, match="C: 32768 bytes"):
        plan.args(A, B, C=torch.zeros(64, 128, dtype=BF), workspace=ws, positions=pos)
    assert api.allocate_outputs(plan, "cpu").C.shape == (64, 256)
