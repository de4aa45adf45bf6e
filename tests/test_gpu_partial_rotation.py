"""Heads that rotate only in part, with infinities, NaN and negative zeros in
them: the values past the rotated part are not touched by the rotation, and a
value of the rotated part reaches its own pair only (needs a GB300).

What a bad value may not reach has the bits it has without it, so nothing here
has a tolerance."""
import pytest
import torch

from gemm_epilogue_transformer_smem_gb300 import api

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    assert torch.cuda.is_available()
    return cuda_lib


def bits(t):
    """The bits of a tensor; every NaN is one value (a conversion keeps no payload)."""
    t = torch.where(torch.isnan(t), torch.full_like(t, NAN), t).contiguous()
    return t.view(torch.int16 if t.dtype is BF else torch.int32)


def same(a, b):
    return torch.equal(bits(a), bits(b))


# type, d, rot, layout, step: heads at a 16-byte aligned stride of d values, or
# one value further (single-element accesses)
CASES = [
    (BF, 128, 64, "half", 0), (BF, 128, 64, "interleaved", 0), (BF, 128, 64, "half", 1),
    (BF, 256, 64, "interleaved", 0), (BF, 96, 48, "half", 0), (BF, 512, 128, "half", 0),
    (BF, 80, 20, "interleaved", 0), (BF, 80, 20, "half", 0), (BF, 64, 6, "interleaved", 0), (BF, 64, 6, "interleaved", 1),
    (F32, 80, 32, "half", 0), (F32, 128, 8, "half", 0), (F32, 256, 30, "interleaved", 0), (F32, 64, 2, "interleaved", 0),
    (F32, 88, 24, "half", 1), (F32, 40, 14, "interleaved", 1), (BF, 4, 2, "interleaved", 1),
]
IDS = ["%s-d%d-r%d-%s-%d" % (str(c[0])[6:], *c[1:]) for c in CASES]

B, S, H = 2, 11, 5


def heads(case, seed):
    dtype, d, _, _, step = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = torch.randn(B, S, H, d + step, generator=g, device=DEV).to(dtype)
    return t[..., step:]


def copy_of(x):
    """A copy with x's strides, gaps included."""
    return torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=DEV).copy_(x)


def spoiled(x, places):
    """x with bad values, one in each of some heads, and where they are."""
    bad, at = copy_of(x), []
    for i, d in enumerate(places):
        for j, v in enumerate((INF, -INF, NAN, -0.0)):
            b, s, h = (i + j) % B, (3 * i + 2 * j + 1) % S, (i + 2 * j) % H
            bad[b, s, h, d] = v
            at.append((b, s, h, d))
    return bad, at


def unrotated_places(case):
    _, d, rot, _, _ = case
    return sorted({rot, rot + 1, (rot + d) // 2, d - 1})


def partner(case, i):
    _, _, rot, layout, _ = case
    return (i + rot // 2) % rot if layout == "half" else i ^ 1


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_rotary_leaves_the_rest_of_a_head_alone(case, inverse):
    dtype, d, rot, layout, _ = case
    x = heads(case, 1)
    bad, _ = spoiled(x, unrotated_places(case))
    rope = api.Rotary(d, rot, layout=layout, scaling=dict(kind="linear", factor=2.0, amplitude=1.5), device=DEV)
    clean, got = torch.empty(B, S, H, d, dtype=dtype, device=DEV), torch.empty(B, S, H, d, dtype=dtype, device=DEV)
    api.rotary(x, None, rope, q_out=clean, inverse=inverse)
    api.rotary(bad, None, rope, q_out=got, inverse=inverse)
    in_place = copy_of(bad)
    api.rotary(in_place, None, rope, q_out=in_place, inverse=inverse)
    torch.cuda.synchronize()
    assert same(got[..., :rot], clean[..., :rot])
    assert same(got[..., rot:], bad[..., rot:])
    assert same(got, in_place)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_rotated_values_reach_their_own_pair(case):
    dtype, d, rot, layout, _ = case
    x = heads(case, 2)
    bad, at = spoiled(x, sorted({0, rot // 2, rot - 1}))
    rope = api.Rotary(d, rot, layout=layout, device=DEV)
    clean, got = torch.empty(B, S, H, d, dtype=dtype, device=DEV), torch.empty(B, S, H, d, dtype=dtype, device=DEV)
    api.rotary(x, None, rope, q_out=clean)
    api.rotary(bad, None, rope, q_out=got)
    torch.cuda.synchronize()
    for b, s, h, i in at:
        for j in (i, partner(case, i)):
            clean[b, s, h, j] = got[b, s, h, j]
    assert same(got, clean)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_norm_with_infinities_past_the_rotated_part(case):
    """1 / rms of a head with an infinity is zero: zeros, and NaN where the
    infinity was."""
    dtype, d, rot, layout, _ = case
    x = heads(case, 3)
    rope = api.Rotary(d, rot, layout=layout, device=DEV)
    clean, got = torch.empty(B, S, H, d, dtype=dtype, device=DEV), torch.empty(B, S, H, d, dtype=dtype, device=DEV)
    api.qk_norm_rotary(x, None, rope, q_out=clean)
    for i in unrotated_places(case):
        bad = copy_of(x)
        bad[1, 3, 2, i] = INF
        api.qk_norm_rotary(bad, None, rope, q_out=got)
        torch.cuda.synchronize()
        want = clean.clone()
        want[1, 3, 2], want[1, 3, 2, i] = 0.0, NAN
        assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward_with_bad_gradients_past_the_rotated_part(case):
    """dw of the place alone sees them, dx of the head alone."""
    dtype, d, rot, layout, _ = case
    x, dy = heads(case, 4), heads(case, 5)
    rope = api.Rotary(d, rot, layout=layout, device=DEV)
    ws = torch.empty(api.qk_norm_rotary_workspace(d), dtype=torch.uint8, device=DEV)

    def run(dy):
        dx, dw = torch.empty(B, S, H, d, dtype=dtype, device=DEV), torch.empty(d, device=DEV)
        api.qk_norm_rotary_backward(dy, None, x, None, rope, dq=dx, dwq=dw, workspace=ws)
        torch.cuda.synchronize()
        return dx, dw

    clean, clean_dw = run(dy)
    for i in unrotated_places(case):
        for v in (INF, NAN):
            bad = copy_of(dy)
            bad[0, 7, 1, i] = v
            dx, dw = run(bad)
            assert not torch.isfinite(dw[i]) and not torch.isfinite(dx[0, 7, 1]).any()
            dx[0, 7, 1], dw[i] = clean[0, 7, 1], clean_dw[i]
            assert same(dx, clean) and same(dw, clean_dw)
