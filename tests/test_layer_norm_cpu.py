"""Dropout, layer norm and its backward pass without a GPU: arguments that the
entry points and the binding take or refuse (an accepted call stops only at the
missing device), and the reference the GPU tests compare with."""
import ctypes
import os
import subprocess

import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api, build, native as N

import residual_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TAKEN = (N.GEMM_EPI_ERR_CUDA, N.GEMM_EPI_ERR_ARCH)  # everything was right but the GPU is missing
INVALID, MISALIGNED = (N.GEMM_EPI_ERR_INVALID_VALUE,), (N.GEMM_EPI_ERR_MISALIGNED,)
UNSUPPORTED, WORKSPACE = (N.GEMM_EPI_ERR_UNSUPPORTED,), (N.GEMM_EPI_ERR_WORKSPACE,)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return N.load()


@pytest.fixture
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("the pointers here are not device memory")


def test_struct_layouts_match_header(lib, tmp_path):
    structs = [N.gemm_epi_mask, N.gemm_epi_dropout_args, N.gemm_epi_layer_norm_args, N.gemm_epi_layer_norm_bwd_args]
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "gemm_epi.h"', "int main(void) {"]
    for st in structs:
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (st.__name__, st.__name__))
        lines += ['printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (st.__name__, f, st.__name__, f) for f, _ in st._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "layout"), str(src)], check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout
    got = dict(line.split() for line in out.splitlines())
    for st in structs:
        assert int(got[st.__name__]) == ctypes.sizeof(st)
        for f, _ in st._fields_:
            assert int(got["%s.%s" % (st.__name__, f)]) == getattr(st, f).offset, (st, f)


@pytest.mark.parametrize("counter,key,words", [
    ((0,) * 4, (0,) * 2, (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_reference_philox(counter, key, words):
    """The generator's published known answers."""
    assert tuple(int(w) for w in R.philox(counter, key)) == words


def test_reference_mask():
    """A mask is a place's own: a part of it is the part's, and its share is the probability's."""
    whole = R.kept(40, 200, 6554, 7, 3, 2)
    assert torch.equal(R.kept(8, 77, 6554, 7, 3, 2, row0=32), whole[32:, :77])
    share = float(R.kept(512, 512, 16384, 1, 0, 0).double().mean())
    assert abs(share - 0.75) < 5 * (0.75 * 0.25) ** 0.5 / 512  # five standard deviations
    assert not torch.equal(whole, R.kept(40, 200, 6554, 7, 4, 2))


def address(shift=0):
    buf = (ctypes.c_uint8 * 16384)()
    base = (ctypes.addressof(buf) + 255) // 256 * 256
    return buf, base + shift


def dropout_args(**kw):
    a = N.gemm_epi_dropout_args()
    buf, at = address()
    a._keep = buf
    a.M, a.N, a.type = 4, 24, N.GEMM_EPI_TYPE_BF16
    a.x, a.ld_x, a.residual, a.ld_residual, a.y, a.ld_y = at, 24, at + 1024, 24, at + 2048, 24
    a.mask.step, a.mask.threshold = at + 4096, 6554
    return fill(a, kw, at)


def norm_args(**kw):
    a = N.gemm_epi_layer_norm_args()
    buf, at = address()
    a._keep = buf
    a.M, a.N, a.type, a.eps = 4, 24, N.GEMM_EPI_TYPE_BF16, 1e-5
    a.x, a.ld_x, a.residual, a.ld_residual, a.y, a.ld_y = at, 24, at + 1024, 24, at + 2048, 24
    a.sum, a.ld_sum, a.w, a.b, a.mean, a.rstd = at + 3008, 24, at + 5000, at + 5200, at + 5400, at + 5600
    a.mask.step, a.mask.threshold = at + 4096, 6554
    return fill(a, kw, at)


def backward_args(**kw):
    a = N.gemm_epi_layer_norm_bwd_args()
    buf, at = address()
    a._keep = buf
    a.M, a.N, a.type = 4, 24, N.GEMM_EPI_TYPE_BF16
    a.dy, a.ld_dy, a.x, a.ld_x, a.add, a.ld_add = at, 24, at + 1024, 24, at + 2048, 24
    a.dx, a.ld_dx, a.d_residual, a.ld_d_residual = at + 3008, 24, at + 6144, 24
    a.w, a.mean, a.rstd, a.dw, a.db = at + 5000, at + 5200, at + 5400, at + 5600, at + 5800
    a.workspace, a.workspace_bytes = at + 8192, N.load().gemm_epi_layer_norm_backward_workspace_size(24)
    a.mask.step, a.mask.threshold = at + 4096, 6554
    return fill(a, kw, at)


def fill(a, kw, at):
    for name, v in kw.items():
        if isinstance(v, str):  # another tensor's address, or one shifted from the tensor's own
            v = getattr(a, name) + int(v) if v[0] in "+-" else getattr(a, v)
        target = a
        if name in ("step", "site", "threshold"):
            target = a.mask
        setattr(target, name, v)
    return a


ENTRIES = {"gemm_epi_dropout": dropout_args, "gemm_epi_layer_norm": norm_args,
           "gemm_epi_layer_norm_backward": backward_args}
BOTH = [
    (dict(), TAKEN), (dict(M=0), TAKEN), (dict(M=-1), INVALID), (dict(M=2 ** 31), INVALID), (dict(N=0), INVALID),
    (dict(N=2 ** 31 - 4095), INVALID), (dict(N=-5), INVALID), (dict(type=N.GEMM_EPI_TYPE_E4M3), UNSUPPORTED),
    (dict(threshold=0, step=None), TAKEN), (dict(threshold=65536), TAKEN), (dict(threshold=65537), INVALID),
    (dict(threshold=-1), INVALID), (dict(step=None), INVALID), (dict(x=None), INVALID), (dict(x="+1"), MISALIGNED),
    (dict(x="+2"), TAKEN), (dict(ld_x=0), TAKEN), (dict(ld_x=1), TAKEN), (dict(ld_x=-24), INVALID),
    (dict(ld_x=2 ** 40 + 1), INVALID),
]
FORWARD = [
    (dict(residual=None), TAKEN), (dict(ld_residual=0), TAKEN), (dict(y=None), INVALID), (dict(ld_y=23), INVALID),
    (dict(ld_y=23, M=1), TAKEN), (dict(ld_y=25), TAKEN), (dict(y="x"), TAKEN), (dict(y="x", ld_x=32), INVALID),
    (dict(y="residual"), TAKEN), (dict(y="residual", ld_y=32), INVALID),
]
CALLS = [(e, kw, want) for e in ENTRIES for kw, want in BOTH]
CALLS += [(e, kw, want) for e in ("gemm_epi_dropout", "gemm_epi_layer_norm") for kw, want in FORWARD]
CALLS += [("gemm_epi_layer_norm", kw, want) for kw, want in [
    (dict(eps=-1e-5), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=0.0), TAKEN), (dict(sum=None), TAKEN),
    (dict(sum="x"), TAKEN), (dict(sum="y"), INVALID), (dict(ld_sum=8), INVALID), (dict(sum="residual", ld_sum=32), INVALID),
    (dict(w=None, b=None, mean=None, rstd=None), TAKEN), (dict(w="+2"), MISALIGNED), (dict(w="+4"), TAKEN),
    (dict(rstd="+1"), MISALIGNED), (dict(mean="rstd"), INVALID),
]]
CALLS += [("gemm_epi_layer_norm_backward", kw, want) for kw, want in [
    (dict(dy=None), INVALID), (dict(add=None), TAKEN), (dict(dx=None), TAKEN), (dict(d_residual=None), TAKEN),
    (dict(dx="dy"), TAKEN), (dict(dx="x", d_residual="dy"), TAKEN), (dict(d_residual="add"), TAKEN),
    (dict(dx="dy", ld_dx=32), INVALID), (dict(d_residual="dx"), INVALID), (dict(ld_dx=23), INVALID),
    (dict(mean=None), INVALID), (dict(rstd=None), INVALID), (dict(w=None), TAKEN), (dict(dw="+1"), MISALIGNED),
    (dict(dw="db"), INVALID), (dict(workspace=None), WORKSPACE), (dict(workspace="+8"), WORKSPACE),
    (dict(workspace_bytes=100), WORKSPACE), (dict(workspace=None, dw=None, db=None), TAKEN),
    (dict(workspace=None, dw=None), WORKSPACE), (dict(dx=None, d_residual=None, dw=None, db=None, dy=None), TAKEN),
    (dict(M=0, workspace=None), TAKEN),
]]


@pytest.mark.parametrize("entry,kw,want", CALLS, ids=lambda v: str(v).replace("gemm_epi_", "") if isinstance(v, (str, dict)) else "")
def test_arguments(lib, no_gpu, entry, kw, want):
    a = ENTRIES[entry](**kw)
    assert getattr(lib, entry)(ctypes.byref(a), None) in want, lib.gemm_epi_last_error()
    assert lib.gemm_epi_last_error()


@pytest.mark.parametrize("entry", list(ENTRIES))
def test_null_arguments(lib, entry):
    assert getattr(lib, entry)(None, None) == N.GEMM_EPI_ERR_INVALID_VALUE


def test_workspace_size(lib):
    size = lib.gemm_epi_layer_norm_backward_workspace_size
    assert size(0) == size(-1) == size(2 ** 31 - 4095) == 0
    assert size(1) % 16 == 0 and 0 < size(1) <= size(24) < size(257) < size(2048)
    assert 1 <= size(2 ** 31 - 4096) / (304 * 2 * (2 ** 31 - 4096) * 4) < 1.001  # no overflow


# ---------------------------------------------------------------- the binding

def host(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def rng():
    return api.Dropout(0.5, device="cpu")


@pytest.mark.parametrize("kw", [dict(p=-0.1), dict(p=1.5), dict(p=float("nan")), dict(p=0.5, seed=-1),
                                dict(p=0.5, seed=2 ** 64), dict(p=0.5, step=-1)])
def test_dropout_object_refuses(kw):
    with pytest.raises(ValueError):
        api.Dropout(device="cpu", **kw)


def test_dropout_object():
    d = api.Dropout(0.1, seed=2 ** 64 - 1, step=2 ** 40, device="cpu")
    assert d.threshold == 6554 and d.seed == 2 ** 64 - 1 and int(d.step) == 2 ** 40
    d.advance()
    d.advance(3)
    assert int(d.step) == 2 ** 40 + 4
    d.step = torch.tensor([1])
    for bad in (torch.zeros(1), torch.zeros(2, dtype=torch.int64), torch.zeros((), dtype=torch.int64)):
        with pytest.raises(ValueError):
            d.step = bad
    assert api.Dropout(1e-6, device="cpu").threshold == 0 and api.Dropout(1.0, device="cpu").threshold == 65536


BINDING = [
    (lambda: api.dropout(host(4, 8), rng(), out=host(4, 8)), ValueError),                       # host memory
    (lambda: api.dropout(host(4, 8, dtype=torch.float16), rng(), out=host(4, 8)), TypeError),
    (lambda: api.dropout(host(4, 8), rng(), out=host(4, 8, dtype=torch.float32)), ValueError),
    (lambda: api.dropout(host(4, 8), rng(), out=host(4, 9)), ValueError),
    (lambda: api.dropout(host(8, 4).t(), rng(), out=host(4, 8)), ValueError),                   # strided columns
    (lambda: api.dropout(host(4, 8), rng(), out=host(4, 8), site=-1), ValueError),
    (lambda: api.dropout(host(4, 8), rng(), out=host(4, 8), site=2 ** 32), ValueError),
    (lambda: api.dropout(host(3, 4, 8).transpose(0, 1), rng(), out=host(4, 3, 8)), ValueError),  # uneven rows
    (lambda: api.dropout(torch.zeros(()), rng(), out=torch.zeros(())), ValueError),
    (lambda: api.layer_norm(host(4, 8), out=host(4, 8), sum_out=host(4, 8)), ValueError),
    (lambda: api.layer_norm(host(4, 8), out=host(4, 8), weight=host(8)), TypeError),
    (lambda: api.layer_norm(host(4, 8), out=host(4, 8), weight=torch.zeros(7)), ValueError),
    (lambda: api.layer_norm(host(4, 8), out=host(4, 8), bias=torch.zeros(16)[::2]), ValueError),
    (lambda: api.layer_norm(host(4, 8), out=host(4, 8), mean=torch.zeros(5)), ValueError),
    (lambda: api.layer_norm_backward(host(4, 8), host(4, 9), torch.zeros(4), torch.zeros(4)), ValueError),
    (lambda: api.layer_norm_backward(host(4, 8), host(4, 8), torch.zeros(3), torch.zeros(4)), ValueError),
    (lambda: api.layer_norm_backward(host(4, 8), host(4, 8), torch.zeros(4), torch.zeros(4).double()), TypeError),
    (lambda: api.layer_norm_backward(host(4, 8), host(4, 8), torch.zeros(4), torch.zeros(4), add=host(4)), ValueError),
    (lambda: api.layer_norm_backward(host(4, 8), host(4, 8), torch.zeros(4), torch.zeros(4), dw=torch.zeros(9)), ValueError),
]


@pytest.mark.parametrize("i", range(len(BINDING)))
def test_binding_refuses(lib, i):
    call, error = BINDING[i]
    with pytest.raises(error):
        call()


def test_row_strides():
    even = host(2, 3, 5, 16)[..., :8]
    assert api._row_stride("t", even, even.shape)[1] == 16
    one = host(2, 1, 5, 8).transpose(0, 1)
    assert api._row_stride("t", one, one.shape)[1] == 8
    same = host(1, 8).expand(6, 8)
    assert api._row_stride("t", same, same.shape)[1] == 0
    assert api._row_stride("t", host(8), (8,))[1] == 8
    with pytest.raises(ValueError):
        api._row_stride("t", host(2, 4, 8)[:, :3], (2, 3, 8))
