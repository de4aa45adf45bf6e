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


class Elsewhere:
    """A tensor that says it is on CUDA device 1."""

    def __init__(self, t):
        self.t = t

    def get_device(self):
        return 1

    device = "cuda:1"

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_plans_run_on_the_device_of_their_tensors(lib, monkeypatch):
    """With device 0 current, tensors on device 1 are launched on with device 1
    current and on its stream."""
    current, calls = [0], []

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(api, "_current_device", lambda: current[0])
    monkeypatch.setattr(api, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(api.torch.cuda, "device", device)

    class Library:
        def __getattr__(self, name):
            def call(*args):
                calls.append((name, current[0], getattr(args[-1], "value", args[-1])))
                return N.GEMM_EPI_OK
            return call

    plan = api.Plan(64, 256, 64, ["store_bf16"])
    A, B, C = (torch.zeros(64, n, dtype=BF) for n in (64, 256, 256))
    ws = Elsewhere(torch.zeros(plan.workspace_bytes, dtype=torch.uint8))
    monkeypatch.setattr(plan, "lib", Library())
    plan.run(A, B, C=C, workspace=ws)
    plan.query_status(ws)
    plan.run_unfused(A, B, C=C, workspace=ws, scratch=Elsewhere(torch.zeros_like(C)))
    current[0] = 1
    plan.run(A, B, C=C, workspace=ws)
    assert calls == [("gemm_epi_run", 1, 1001), ("gemm_epi_query_status", 1, 1001), ("gemm_epi_run_unfused", 1, 1001),
                     ("gemm_epi_run", 1, 1001)]
    monkeypatch.undo()  # the handle is destroyed by the library it is from

    rope = api.Rotary(64, device="cpu")
    heads = api.Plan(64, 256, 64, ["rotary", "store_bf16"], rotary=rope, head_cols=128)
    with pytest.raises(ValueError, match="the workspace on cuda:1"):
        heads.args(None, None, C=C, workspace=ws)


def test_a_forced_split_is_two_to_eight(lib):
    plan = api.Plan(64, 256, 1024, ["rotary", "store_bf16"], rotary=api.Rotary(64, device="cpu"), head_cols=128)
    A, B, C = torch.zeros(64, 1024, dtype=BF), torch.zeros(1024, 256, dtype=BF), torch.zeros(64, 256, dtype=BF)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8)

    class Stream:
        cuda_stream = 0

    for n in (1, 9, 15):
        with pytest.raises(N.GemmEpiError, match="2 to 8") as err:
            plan.run(A, B, C=C, workspace=ws, stream=Stream(), debug_flags=N.GEMM_EPI_DEBUG_FORCE_SPLIT(n))
        assert err.value.status == N.GEMM_EPI_ERR_INVALID_VALUE
