"""The head operators without a GPU: the steps of a rotary position, what the
entry points refuse, and the 64-bit reference against differences."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api, build, native as N

import heads_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return N.load()


class FakeStream:
    cuda_stream = 0


def test_struct_layouts_match_header(lib, tmp_path):
    structs = [N.gemm_epi_rotary_freq, N.gemm_epi_heads, N.gemm_epi_qk_args]
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "gemm_epi.h"', "int main(void) {"]
    for st in structs:
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (st.__name__, st.__name__))
        for f, _ in st._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (st.__name__, f, st.__name__, f))
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    for st in structs:
        assert int(got[st.__name__]) == ctypes.sizeof(st)
        for f, _ in st._fields_:
            assert int(got["%s.%s" % (st.__name__, f)]) == getattr(st, f).offset, (st.__name__, f)


SCALINGS = [None, dict(kind="linear", factor=4.0), dict(kind="ntk", factor=8.0),
            dict(kind="by_parts", factor=8.0, original_length=8192.0),
            dict(kind="by_parts", factor=4.0, original_length=4096.0, low=1.0, high=4.0, amplitude=1.1)]


@pytest.mark.parametrize("scaling", SCALINGS, ids=[str(s and s["kind"]) for s in SCALINGS])
@pytest.mark.parametrize("rot,base", [(128, 10000.0), (64, 500000.0), (6, 10.0)])
def test_steps_are_the_frequencies(lib, scaling, rot, base):
    """step / 2^64 is the pair's fraction of a turn per position: within the
    rounding of the 64-bit step and of the double arithmetic before it (pow to
    an ulp or two, three products and a quotient: 8 half steps of the value)."""
    rope = api.Rotary(rot, base=base, scaling=scaling, device="cpu")
    want = R.frequencies(rot, base, scaling)
    for step, f in zip(rope.steps.tolist(), want.tolist()):
        turns = (step % 2 ** 64) / 2.0 ** 64
        assert abs(turns - (f / (2 * math.pi)) % 1.0) <= 8 * 2.0 ** -53 * f + 2.0 ** -64
    assert rope.amplitude == (scaling or {}).get("amplitude", 1.0)


def test_given_frequencies_wrap(lib):
    """Negative frequencies and those past a turn per position are taken modulo a turn."""
    freqs = [0.0, -0.25, 2 * math.pi * 3.125, math.pi]
    steps = api.Rotary(8, freqs=freqs, device="cpu").steps.tolist()
    turns = [(s % 2 ** 64) / 2.0 ** 64 for s in steps]
    assert turns[0] == 0.0 and turns[3] == 0.5
    assert abs(turns[1] - (1.0 - 0.25 / (2 * math.pi))) < 2.0 ** -51
    assert abs(turns[2] - 0.125) < 2.0 ** -50
    # a frequency just below zero rounds to a whole turn, which is none
    assert api.Rotary(2, freqs=[-1e-25], layout="interleaved", device="cpu").steps.tolist() == [0]


@pytest.mark.parametrize("kw,match", [
    (dict(head_dim=64, layout="other"), "layout"), (dict(head_dim=64, rotary_dim=66), "above head_dim"),
    (dict(head_dim=64, rotary_dim=0), "rotary_dim"), (dict(head_dim=64, rotary_dim=7), "rotary_dim"),
    (dict(head_dim=1024), "rotary_dim"), (dict(head_dim=64, base=0.0), "base"),
    (dict(head_dim=64, base=float("inf")), "base"), (dict(head_dim=64, base=float("nan")), "base"),
    (dict(head_dim=64, scaling=dict(kind="cubic", factor=2.0)), "scaling"),
    (dict(head_dim=64, scaling=dict(kind="linear", factor=0.0)), "factor"),
    (dict(head_dim=64, scaling=dict(kind="linear", factor=2.0, low=1.0)), "low"),
    (dict(head_dim=2, layout="interleaved", scaling=dict(kind="ntk", factor=2.0)), "NTK"),
    (dict(head_dim=64, base=1e300, scaling=dict(kind="ntk", factor=1e300)), "not finite"),
    (dict(head_dim=64, scaling=dict(kind="by_parts", factor=2.0, original_length=0.0)), "original_length"),
    (dict(head_dim=64, scaling=dict(kind="by_parts", factor=2.0, original_length=8.0, low=4.0, high=4.0)), "low < high"),
    (dict(head_dim=8, freqs=[1.0, 2.0]), "2 frequencies"), (dict(head_dim=4, freqs=[1.0, float("nan")]), "not finite"),
])
def test_rotary_refuses(lib, kw, match):
    with pytest.raises((ValueError, N.GemmEpiError), match=match):
        api.Rotary(device="cpu", **kw)


def base_args():
    buf = (ctypes.c_uint8 * 65536)()
    base = (ctypes.addressof(buf) + 255) // 256 * 256  # never dereferenced on the host
    a = N.gemm_epi_qk_args()
    a.batch, a.tokens, a.q_heads, a.k_heads, a.head_dim, a.rotary_dim = 2, 3, 4, 2, 64, 64
    for i, h in enumerate((a.q, a.k, a.q_out, a.k_out, a.dy_q, a.dy_k)):
        h.data, h.stride_batch, h.stride_token, h.stride_head = base + 4096 * i, 3 * 256, 256, 64
    a.steps, a.amplitude, a.eps = base + 40000, 1.0, 1e-6
    a.dw_q, a.dw_k = base + 48000, base + 52000
    a.workspace, a.workspace_bytes = base, 1 << 30
    return a, buf, base


ENTRIES = ["gemm_epi_rotary", "gemm_epi_qk_norm_rotary", "gemm_epi_qk_norm_rotary_backward"]


def put(a, name, value):
    obj, _, field = name.rpartition(".")
    setattr(getattr(a, obj) if obj else a, field, value)


BAD, MIS, UNS = N.GEMM_EPI_ERR_INVALID_VALUE, N.GEMM_EPI_ERR_MISALIGNED, N.GEMM_EPI_ERR_UNSUPPORTED
REFUSED = [
    ("batch", -1, BAD), ("tokens", 2 ** 31, BAD), ("tokens", 2 ** 30, BAD), ("q_heads", -1, BAD), ("k_heads", 65536, BAD),
    ("head_dim", 0, BAD), ("head_dim", 63, BAD), ("head_dim", 514, BAD), ("rotary_dim", 0, BAD), ("rotary_dim", 66, BAD),
    ("rotary_dim", 7, BAD), ("rotary_dim", 6, UNS), ("layout", 2, BAD), ("type", N.GEMM_EPI_TYPE_E4M3, UNS),
    ("type", 9, UNS), ("amplitude", float("nan"), BAD), ("q.data", None, BAD), ("k.data", None, BAD),
    ("q.stride_token", 2 ** 41, BAD), ("q_out.stride_head", 0, BAD), ("k_out.stride_token", 32, BAD),
    ("q_out.stride_batch", -63, BAD), ("steps", None, BAD), ("position_stride", 2, BAD),
]


@pytest.mark.parametrize("entry", ENTRIES)
def test_entry_points_check_arguments_on_the_host(lib, entry):
    fn = getattr(lib, entry)
    assert fn(None, None) == BAD
    a, keep, base = base_args()
    a.positions = base + 60000
    a.position_stride = 3
    assert fn(ctypes.byref(a), None) in (N.GEMM_EPI_ERR_CUDA, N.GEMM_EPI_ERR_ARCH)  # only the GPU is missing
    bwd = entry.endswith("backward")
    cases = list(REFUSED)
    cases += [("q.data", base + 1, MIS), ("q_out.data", base + 4096 * 2 + 1, MIS), ("steps", base + 4, MIS),
              ("positions", base + 60002, MIS), ("q_weight", base + 2, MIS),
              ("q_out.data", a.k.data, BAD), ("k_out.data", a.q.data, BAD)]
    cases += [("dy_q.data", None, BAD), ("dw_k", base + 2, MIS), ("dw_k", a.dw_q, BAD), ("q_out.data", a.dy_k.data, BAD),
              ("workspace", None, N.GEMM_EPI_ERR_WORKSPACE), ("workspace", base + 8, N.GEMM_EPI_ERR_WORKSPACE),
              ("workspace_bytes", 64, N.GEMM_EPI_ERR_WORKSPACE)] if bwd else \
        [("q_out.data", None, BAD), ("k_out.data", None, BAD)]
    if entry != "gemm_epi_rotary":
        cases += [("eps", -1.0, BAD), ("eps", float("inf"), BAD), ("eps", float("nan"), BAD)]
    for name, value, status in cases:
        a, keep, base2 = base_args()
        a.positions, a.position_stride = base2 + 60000, 3
        if isinstance(value, int) and abs(value - base) < 65536:
            value = value - base + base2
        put(a, name, value)
        got = fn(ctypes.byref(a), None)
        assert got == status, (name, value, got, lib.gemm_epi_last_error())
        assert lib.gemm_epi_last_error()
    # an output on its input's memory with other strides
    a, keep, _ = base_args()
    a.q_out.data, a.q_out.stride_token = a.q.data, 512
    assert fn(ctypes.byref(a), None) == BAD


def test_workspace_size(lib):
    for d in (2, 64, 128, 512):
        assert api.qk_norm_rotary_workspace(d) >= 2 * d * 4
    assert lib.gemm_epi_qk_norm_rotary_workspace_size(0) == 0
    assert lib.gemm_epi_qk_norm_rotary_workspace_size(1024) == 0


def test_binding_checks(lib):
    rope = api.Rotary(64, device="cpu")
    q, k = torch.zeros(2, 5, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16)
    ok = dict(q_out=q, k_out=k)
    pos = torch.zeros(2, 5, dtype=torch.int32)

    def refused(match, q=q, k=k, pos=pos, kind=ValueError, fn=api.rotary, **kw):
        with pytest.raises(kind, match=match):
            fn(q, k, rope, pos, **dict(ok, **kw))

    refused("CUDA tensors")                                   # everything else is right
    refused("both None", q=None, k=None)
    refused("k_out without k", k=None)
    refused("q_out is missing", q_out=None)
    refused("bf16 or fp32", q=q.half(), kind=TypeError)
    refused("expected .batch", q=q[..., :32])
    refused("expected .batch", q=q[0, 0])
    refused("does not match", q_out=q.float())
    refused("does not match", q_out=q[:, :4])
    refused("do not belong", k=k[:, :4], k_out=k[:, :4])
    refused("do not belong", k=k.float(), k_out=k.float())
    refused("contiguous", q=torch.zeros(2, 5, 4, 128, dtype=torch.bfloat16)[..., ::2])
    refused("int32 or int64", pos=pos.float(), kind=TypeError)
    refused("positions: expected", pos=pos[:, :4])
    refused("positions: expected", pos=pos.t())
    refused("contiguous", pos=torch.zeros(2, 10, dtype=torch.int32)[:, ::2])
    refused("f32", fn=api.qk_norm_rotary, q_weight=torch.zeros(64, dtype=torch.float64), kind=TypeError)
    refused("64 contiguous", fn=api.qk_norm_rotary, q_weight=torch.zeros(32))
    with pytest.raises(ValueError, match="given together"):
        api.qk_norm_rotary_backward(None, k, q, k, rope, pos, dk=k)
    with pytest.raises(ValueError, match="does not match"):
        api.qk_norm_rotary_backward(q[:, :, :2], k, q, k, rope, pos, dk=k)
    with pytest.raises(ValueError, match="CUDA tensors"):
        api.qk_norm_rotary_backward(q, k, q, k, rope, pos, dq=q)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_reference_gradients_against_differences(layout):
    """The 64-bit formulas of the backward pass are the derivatives of the
    forward ones (central differences, h = 1e-5: off by h^2 and 2^-53 / h)."""
    g = torch.Generator().manual_seed(3)
    d, rot, eps = 12, 8, 1e-3
    x, dy = torch.randn(2, 3, 2, d, generator=g, dtype=torch.float64), torch.randn(2, 3, 2, d, generator=g, dtype=torch.float64)
    w = 1.0 + 0.3 * torch.randn(d, generator=g, dtype=torch.float64)
    ang = R.Angles(torch.tensor([[0, 5, 9], [2, 3, 4]]), rot, layout, 1.3)
    loss = lambda x, w: (ang.rotate(R.norm(x, w, eps)) * dy).sum().item()  # noqa: E731
    dx, dw, _, _ = R.backward(dy, x, w, eps, ang)
    h = 1e-5
    for i in range(0, x.numel(), 5):
        e = torch.zeros_like(x).view(-1)
        e[i] = h
        e = e.view_as(x)
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx.view(-1)[i].item()) < 1e-7
    for i in range(d):
        e = torch.zeros_like(w)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i].item()) < 1e-7
    # the inverse rotation is the rotation's transpose
    lhs, rhs = (ang.rotate(x) * dy).sum(), (x * ang.rotate(dy, inverse=True)).sum()
    assert abs(lhs - rhs).item() < 1e-12 * x.numel()


def create(lib, program, N_=512, **kw):
    ops = api.encode_program(list(program))
    d = N.gemm_epi_desc(M=64, N=N_, K=64, lda=64, ldb=kw.pop("ldb", 64), ldc=2 * N_, ldc8=2 * N_, ld_aux=2 * N_,
                        b_layout=kw.pop("b_layout", N.GEMM_EPI_B_NK), n_ops=len(program),
                        ops=ctypes.cast(ops, ctypes.POINTER(N.gemm_epi_op)))
    d.head_dim, d.head_cols, d.rotary_dim = 128, 384, 128
    for k, v in kw.items():
        setattr(d, k, v)
    h = N.gemm_epi_handle()
    s = lib.gemm_epi_create(ctypes.byref(h), ctypes.byref(d))
    if s == N.GEMM_EPI_OK:
        lib.gemm_epi_destroy(h)
    return s


NORM = ("head_rms:1e-5", "col_scale", "rotary", "store_bf16")


@pytest.mark.parametrize("program,kw", [
    (NORM, {}), (NORM, dict(head_cols=0)), (NORM, dict(head_cols=512)), (("rotary",), dict(rotary_dim=64)),
    (("rotary", "store_bf16"), dict(rotary_dim=32)), (("rotary", "store_bf16"), dict(rotary_dim=2, rotary_layout=1)),
    (("head_rms", "store_bf16"), dict(rotary_dim=0)), (("bias", "alpha", "gelu_tanh", "rotary", "store_bf16"), {}),
    (("rotary", "amax", "store_bf16", "store_e4m3", "col_sum", "row_rms"), {}),
])
def test_create_accepts_head_programs(lib, program, kw):
    assert create(lib, program, **kw) == N.GEMM_EPI_OK, lib.gemm_epi_last_error()


@pytest.mark.parametrize("program,kw,status", [
    (NORM, dict(head_dim=96, head_cols=96), UNS), (NORM, dict(head_dim=0), UNS), (NORM, dict(head_dim=512, head_cols=512), UNS),
    (NORM, dict(head_cols=100), BAD), (NORM, dict(head_cols=640), BAD), (NORM, dict(head_cols=-128), BAD),
    (NORM, dict(rotary_layout=2), BAD), (NORM, dict(rotary_dim=0), BAD), (NORM, dict(rotary_dim=130), BAD),
    (NORM, dict(rotary_dim=63), BAD), (NORM, dict(rotary_dim=96), UNS), (NORM, dict(rotary_dim=48), UNS),
    (("head_rms:-1", "store_bf16"), {}, BAD), (("head_rms:nan", "store_bf16"), {}, BAD),
    (("head_rms", "head_rms", "store_bf16"), {}, BAD), (("rotary", "rotary", "store_bf16"), {}, BAD),
    (("rotary", "head_rms", "store_bf16"), {}, UNS), (("store_bf16", "rotary"), {}, UNS),
    (("residual", "rotary", "store_bf16"), {}, UNS), (("rotary", "residual", "store_bf16"), {}, UNS),
    (("rotary", "gelu_tanh_grad", "store_bf16"), {}, UNS), (("rotary", "store_bf16", "row_dot"), {}, UNS),
    (("pair_swiglu", "rotary", "store_bf16"), {}, UNS), (("rotary", "pair_swiglu", "store_bf16"), {}, UNS),
    (("rotary", "dswiglu", "store_bf16"), {}, UNS), (("dswiglu", "rotary", "store_bf16"), {}, UNS),
    (NORM, dict(b_layout=N.GEMM_EPI_B_NK | N.GEMM_EPI_B_DUAL), UNS),
])
def test_create_rejects_head_programs(lib, program, kw, status):
    assert create(lib, program, **kw) == status, lib.gemm_epi_last_error()
    assert lib.gemm_epi_last_error()


def test_plan_checks_rotary_and_positions(lib):
    rope = api.Rotary(64, device="cpu")
    with pytest.raises(ValueError, match="needs rotary="):
        api.Plan(64, 256, 64, ["rotary", "store_bf16"], head_dim=64, head_cols=128)
    with pytest.raises(ValueError, match="not the rotary's"):
        api.Plan(64, 256, 64, ["rotary", "store_bf16"], rotary=rope, head_dim=128, head_cols=128)
    plan = api.Plan(64, 256, 64, ["rotary", "store_bf16"], rotary=rope, head_cols=128)
    A, B = torch.zeros(64, 64, dtype=torch.bfloat16), torch.zeros(64, 256, dtype=torch.bfloat16)
    C, ws = torch.zeros(64, 256, dtype=torch.bfloat16), torch.zeros(plan.workspace_bytes, dtype=torch.uint8)
    pos = torch.zeros(64, dtype=torch.int32)
    a = plan.args(A, B, C=C, workspace=ws, positions=pos)
    assert a.positions == pos.data_ptr() and a.positions_64 == 0 and a.rotary_amplitude == 1.0
    for bad, kind in ((pos.float(), TypeError), (pos[:32], ValueError), (torch.zeros(128, dtype=torch.int32)[::2], ValueError)):
        with pytest.raises(kind, match="positions"):
            plan.args(A, B, C=C, workspace=ws, positions=bad)
    bare = api.Plan(64, 256, 64, ["store_bf16"])
    with pytest.raises(ValueError, match="no rotary"):
        bare.args(A, B, C=C, workspace=ws, positions=pos)
    # everything given: stops only at the missing GPU; the separate pass has no such ops
    with pytest.raises(N.GemmEpiError) as err:
        plan.run(A, B, C=C, workspace=ws, positions=pos, stream=FakeStream())
    assert err.value.status in (N.GEMM_EPI_ERR_CUDA, N.GEMM_EPI_ERR_ARCH), str(err.value)
    with pytest.raises(N.GemmEpiError) as err:
        plan.run_unfused(A, B, C=C, workspace=ws, positions=pos, scratch=torch.zeros_like(C), stream=FakeStream())
    assert err.value.status == UNS
    # the C ABI's own checks of the pointers
    for field, value, status in (("rotary_steps", None, BAD), ("rotary_steps", rope.steps.data_ptr() + 4, MIS),
                                 ("positions", pos.data_ptr() + 2, MIS), ("rotary_amplitude", float("inf"), BAD)):
        a = plan.args(A, B, C=C, workspace=ws, positions=pos)
        setattr(a, field, value)
        assert lib.gemm_epi_run(plan.handle, ctypes.byref(a), None) == status, field
