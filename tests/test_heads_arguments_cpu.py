"""Arguments of the head operators that their entry points take or refuse,
without a GPU: an accepted call stops only at the missing device."""
import ctypes

import pytest

from gemm_epilogue_transformer_smem_gb300 import build, native as N

TAKEN = (N.GEMM_EPI_ERR_CUDA, N.GEMM_EPI_ERR_ARCH)  # everything was right but the GPU is missing
REFUSED = (N.GEMM_EPI_ERR_INVALID_VALUE,)
ENTRIES = ["gemm_epi_rotary", "gemm_epi_qk_norm_rotary", "gemm_epi_qk_norm_rotary_backward"]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return N.load()


@pytest.fixture(autouse=True)
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers here are not device memory")


def args(batch, tokens, heads, head_dim=64):
    """q alone, tight (batch, tokens, heads, head_dim); the addresses are never read."""
    buf = (ctypes.c_uint8 * 8192)()
    base = (ctypes.addressof(buf) + 255) // 256 * 256
    a = N.gemm_epi_qk_args()
    a.batch, a.tokens, a.q_heads, a.head_dim, a.rotary_dim = batch, tokens, heads, head_dim, head_dim
    for i, h in enumerate((a.q, a.q_out, a.dy_q)):
        h.data = base + 1024 * i
        h.stride_batch, h.stride_token, h.stride_head = tokens * heads * head_dim, heads * head_dim, head_dim
    a.steps, a.amplitude, a.eps = base + 4096, 1.0, 1e-6
    a._keep = buf
    return a


def strides(h, values):
    h.stride_batch, h.stride_token, h.stride_head = values


# batch, tokens, heads, (batch, token, head strides) of an output of 64 values a head
APART = [
    (2, 5, 3, (960, 192, 64)), (2, 5, 3, (960, 64, 320)), (2, 5, 3, (64, 128, 640)), (2, 5, 3, (-960, 192, -64)),
    (2, 5, 3, (2000, 300, 70)), (1, 5, 3, (0, 192, 64)), (2, 1, 3, (192, 0, 64)), (2, 5, 1, (320, 64, 64)),
    (1, 1, 1, (0, 0, 0)), (1, 5, 1, (64, 64, 64)), (2, 2 ** 30 - 1, 1, (2 ** 39, 64, 0)),
    (2, 3, 2, (2 ** 38, 2 ** 39, 64)), (2, 2 ** 30 - 1, 1, (64, 2 ** 39, 0)),
]
OVERLAPPING = [
    (1, 5, 3, (0, 64, 64)), (2, 5, 1, (64, 64, 0)), (2, 1, 3, (64, 0, 64)), (2, 5, 3, (960, 128, 64)),
    (2, 5, 3, (959, 192, 64)), (2, 5, 3, (960, 191, 64)), (2, 5, 3, (960, -64, 64)), (2, 5, 3, (960, 64, 319)),
    (2, 5, 3, (960, 192, 63)), (2, 5, 3, (0, 192, 64)),
    (2, 5, 3, (-64, 64, 320)), (2, 2 ** 29, 3, (2 ** 38, 2 ** 39, 2 ** 39)),
]


@pytest.mark.parametrize("entry", ENTRIES)
def test_outputs_whose_heads_are_apart(lib, entry):
    for b, t, h, st in APART:
        a = args(b, t, h)
        strides(a.q_out, st)
        assert getattr(lib, entry)(ctypes.byref(a), None) in TAKEN, (b, t, h, st, lib.gemm_epi_last_error())


@pytest.mark.parametrize("entry", ENTRIES)
def test_outputs_whose_heads_overlap(lib, entry):
    """Two heads of an output in the same memory would be a race: refused."""
    for b, t, h, st in OVERLAPPING:
        a = args(b, t, h)
        strides(a.q_out, st)
        assert getattr(lib, entry)(ctypes.byref(a), None) in REFUSED, (b, t, h, st)
        assert b"overlap" in lib.gemm_epi_last_error()


@pytest.mark.parametrize("entry", ENTRIES)
def test_in_place_views_that_differ_in_single_steps(lib, entry):
    """The same memory through two views: the stride of a dimension of one step
    does not matter, another one does."""
    for batch, tokens, heads in ((4, 1, 3), (1, 5, 3), (4, 5, 1), (1, 1, 1)):
        for name in ("stride_batch", "stride_token", "stride_head"):
            a = args(batch, tokens, heads)
            a.q_out.data = a.q.data
            setattr(a.q_out, name, getattr(a.q, name) * 2)
            single = {"stride_batch": batch, "stride_token": tokens, "stride_head": heads}[name] == 1
            got = getattr(lib, entry)(ctypes.byref(a), None)
            assert got in (TAKEN if single else REFUSED), (batch, tokens, heads, name, lib.gemm_epi_last_error())
            a.q_out.data = a.dy_q.data  # over the gradient: any other memory to the forward pass
            got = getattr(lib, entry)(ctypes.byref(a), None)
            if entry.endswith("backward") or single:
                assert got in (TAKEN if single else REFUSED), (batch, tokens, heads, name, lib.gemm_epi_last_error())
