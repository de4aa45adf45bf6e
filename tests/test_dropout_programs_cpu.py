"""Programs with dropout without a GPU: what gemm_epi_create and the binding
take and refuse."""
import ctypes

import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api, build, native as N

DROP = N.GEMM_EPI_OP_DROPOUT


@pytest.fixture(scope="module")
def lib():
    build.build()
    return N.load()


def create(lib, ops, M=64, N_=64, **desc):
    arr = (N.gemm_epi_op * len(ops))(*[N.gemm_epi_op(*(o if isinstance(o, tuple) else (o, 0, 0.0))) for o in ops])
    d = N.gemm_epi_desc()
    d.M, d.N, d.K, d.lda, d.ldb, d.ldc, d.ldc8, d.ld_aux = M, N_, 64, 64, 64, 2 * N_, 2 * N_, 2 * N_
    d.b_layout, d.n_ops, d.ops = N.GEMM_EPI_B_NK, len(ops), ctypes.cast(arr, ctypes.POINTER(N.gemm_epi_op))
    for k, v in desc.items():
        setattr(d, k, v)
    h = N.gemm_epi_handle()
    status = lib.gemm_epi_create(ctypes.byref(h), ctypes.byref(d))
    if status == 0:
        lib.gemm_epi_destroy(h)
    return status


D = (DROP, 6554, 0.0)
STORE = N.GEMM_EPI_OP_STORE_BF16


@pytest.mark.parametrize("ops,desc,want", [
    ([D, STORE], {}, 0), ([(DROP, 0, 0.0), STORE], {}, 0), ([(DROP, 65536, 0.0), STORE], {}, 0),
    ([(DROP, 65537, 0.0), STORE], {}, N.GEMM_EPI_ERR_INVALID_VALUE), ([(DROP, -1, 0.0), STORE], {}, N.GEMM_EPI_ERR_INVALID_VALUE),
    ([D, D, STORE], {}, N.GEMM_EPI_ERR_INVALID_VALUE),
    ([D, N.GEMM_EPI_OP_PAIR_SWIGLU, STORE], {}, N.GEMM_EPI_ERR_UNSUPPORTED),
    ([N.GEMM_EPI_OP_PAIR_SWIGLU, D, STORE], {}, 0), ([D, N.GEMM_EPI_OP_DSWIGLU, STORE], {}, 0),
    ([N.GEMM_EPI_OP_DSWIGLU, D, STORE], {}, 0), ([STORE, D, N.GEMM_EPI_OP_COL_SUM], {}, 0),
    ([D, N.GEMM_EPI_OP_ADD_RESIDUAL, STORE, N.GEMM_EPI_OP_ROW_RMS_RSQRT], {}, 0),
    ([D, N.GEMM_EPI_OP_ROTARY, STORE], dict(head_dim=32, rotary_dim=32), N.GEMM_EPI_ERR_UNSUPPORTED),
    ([N.GEMM_EPI_OP_HEAD_RMS, D, STORE], dict(head_dim=32), N.GEMM_EPI_ERR_UNSUPPORTED),
    ([(22, 0, 0.0)], {}, N.GEMM_EPI_ERR_INVALID_VALUE),
])
def test_create(lib, ops, desc, want):
    assert create(lib, ops, **desc) == want, lib.gemm_epi_last_error()


def test_rows_are_counted_in_32_bits(lib):
    big = dict(M=2 ** 27, N_=8, batch=32, batch_stride_a=2 ** 33, batch_stride_b=0, batch_stride_c=2 ** 31)
    assert create(lib, [D, STORE], **big) == 0
    assert create(lib, [D, STORE], **dict(big, batch=33)) == N.GEMM_EPI_ERR_INVALID_VALUE
    assert create(lib, [STORE], **dict(big, batch=33)) == 0


def plan(p=0.1, program=("dropout", "store_bf16")):
    return api.Plan(64, 64, 64, list(program), b_layout="nk", dropout=api.Dropout(p, device="cpu"))


def test_plan_needs_its_dropout(lib):
    with pytest.raises(ValueError):
        api.Plan(64, 64, 64, ["dropout", "store_bf16"], b_layout="nk")
    assert plan().dropout is not None and plan(program=["store_bf16"]).dropout is None


@pytest.mark.parametrize("site", [-1, 2 ** 32])
def test_site_out_of_range(lib, site):
    with pytest.raises(ValueError):
        plan().args(None, None, site=site)


def test_site_without_dropout(lib):
    with pytest.raises(ValueError):
        plan(program=["store_bf16"]).args(None, None, site=1)


def test_step_must_be_there_and_aligned(lib):
    if torch.cuda.is_available():
        pytest.skip("the pointers here are not device memory")
    buf = torch.zeros(65536, dtype=torch.uint8)
    base = (buf.data_ptr() + 255) // 256 * 256
    p = plan()
    a = p.args(None, None)
    for name in ("A", "B", "C"):
        setattr(a, name, base)
    a.workspace, a.workspace_bytes = base + 16384, 32768
    run = lambda: lib.gemm_epi_run(p.handle, ctypes.byref(a), None)  # noqa: E731
    assert run() in (N.GEMM_EPI_ERR_CUDA, N.GEMM_EPI_ERR_ARCH)
    a.dropout_step += 4
    assert run() == N.GEMM_EPI_ERR_MISALIGNED
    a.dropout_step = None
    assert run() == N.GEMM_EPI_ERR_INVALID_VALUE
    q = plan(0.0)
    assert lib.gemm_epi_run(q.handle, ctypes.byref(a), None) in (N.GEMM_EPI_ERR_CUDA, N.GEMM_EPI_ERR_ARCH)


def test_no_separate_pass(lib):
    p = plan()
    a = p.args(None, None)
    assert lib.gemm_epi_run_unfused(p.handle, ctypes.byref(a), None, 64, None) == N.GEMM_EPI_ERR_UNSUPPORTED
